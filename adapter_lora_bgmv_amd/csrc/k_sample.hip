// k_sample.hip -- one token of every row of logits, drawn under temperature, top-k, top-p and min-p from a given number.
//
// For a row x with maximum m and temperature T, token t has the weight
//     W_t = rint(2^43 exp((x_t - m) / T)),
// a whole number of at most 2^43, so that a vocabulary of 2^20 sums below
// 2^63.  Sums of whole numbers do not depend on their order: however a row is
// cut into threads and workgroups, and whatever batch it stands in, its token
// is the same.  2^-43 of the largest weight is what a weight is rounded to;
// the exponential runs in 64 bits.
//
// All filters keep a prefix of one order, by value, equal values by the lower
// index first: top-k the first k, top-p the fewest whose weights reach p of
// what top-k kept, min-p those of at least that part of the largest weight.
// So a row needs one cut in that order, a value's key with the last index that
// is kept among its equals.  Tokens are then run through by index, and the
// first at which the running sum exceeds floor(u sum) is the row's.
//
// The exponent's whole steps, n = rint(256 log2(e) (x - m) / T), serve twice:
// they pick 2^(n/256) from a table, and some of them are a bin: 1 up to 512, 2
// up to 1536, 4 up to 3584 and so on, as a flat row's tokens lie in the first
// powers of two.  (16 throughout: 131071 normally distributed logits put 2300 into
// top-p's bin, more than a list holds, and the draw took 328 us.)  Rows go by
// what they ask for:
//   top-k up to 512: the row's maximum comes with those of its parts, 32
//     logits each.  The bin that k of these maxima reach bounds the k-th
//     largest logit from below, so the few logits from there up are listed
//     and everything else happens among them.
//   top-p: the weights of every bin are summed, the bin in which the cut lies
//     follows, its logits are listed, and the cut among them by their
//     finer bins and then one by one.
//   neither: the weights are summed.
// Sums are kept for each segment of 2048 logits, a wave's 32 a lane.  The
// segment that holds the number drawn is read again by the whole workgroup.
// Where a list overflows (many equal logits), the cut is found by histograms
// over the key's bits, 11, 11 and 10 of them, and a count in order of index.
//
// Few rows are spread over workgroups by kernels that each end where all of a
// row is needed: maxima, sums and lists, lists of top-p's bin, the drawing.
//
// Vector instructions bound many rows, 64-bit ones above all: 4096 rows of
// 32000 in bf16 take 148 us without a cut (a weight is 14 f64 instructions; one
// reading at HBM's rate would take 50, and a row is read twice), 262 with
// top-p, which goes through the row once more, 119 with top-k.  Of settings of
// all kinds, 187 us, vector instructions take 65 %; 2.1 readings come from HBM,
// and registers that spill write 112 MB.  Chains of launches, round trips and
// barriers bound few: 64 such rows take 17, 33 and 24 us, one of 131071 in f32
// with top-p 32.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "common.hpp"
#include "verify.hpp"

namespace lora {

typedef unsigned long long u64;
constexpr int kRadixBins = 2048;
constexpr int kBins = 2274;          // of 44 powers of two and the step below, beyond which weights are 0
constexpr int kSteps = 44 * 256 + 32;
constexpr int kLowest = kBins - 1;   // holds weights of 0 only: its first step is 11280, 2^(43 - 44.06)
constexpr int kBinsEach = (kBins + kSampleThreads - 1) / kSampleThreads;  // of a thread
constexpr int kMostListedK = 512;    // top-k that goes by the parts' maxima
constexpr int kParts = 4096;         // maxima that a row keeps at most
constexpr int kWaves = kSampleThreads / 64;
constexpr double kUnit = 8796093022208.0;  // 2^43

__device__ __forceinline__ uint32_t sample_key(float x) {  // unsigned order is the value's; the zeros are equal
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) { return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key); }
// Larger values first, equal ones by the lower index.
__device__ __forceinline__ u64 place_of(float x, int index) { return (u64)sample_key(x) << 32 | (uint32_t)~index; }
__device__ __forceinline__ int index_of(u64 place) { return (int)~(uint32_t)place; }

// The same value in every lane, to be held in scalar registers.
__device__ __forceinline__ float uniform(float v) { return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(v))); }
__device__ __forceinline__ u64 uniform(u64 v) {
  return (u64)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32)) << 32 |
         (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
}
__device__ __forceinline__ double uniform(double v) { return __longlong_as_double((long long)uniform((u64)__double_as_longlong(v))); }

template <typename T>
struct Logits;
template <>
struct Logits<float> {
  static constexpr int N = 4;
  static __device__ float at(const uint4 &v, int e) {
    return __uint_as_float(e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w);
  }
};
template <>
struct Logits<u16> {
  static constexpr int N = 8;
  static __device__ float at(const uint4 &v, int e) {
    const uint32_t w = e < 2 ? v.x : e < 4 ? v.y : e < 6 ? v.z : v.w;
    return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
  }
};

// Sum over the lanes up to and including this one, in registers (as wave_incl_scan, 64 bits).
template <int CTRL, int ROWS>
__device__ __forceinline__ u64 dpp_step64(u64 v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROWS, 0xf, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, ROWS, 0xf, false);
  return v + ((u64)hi << 32 | lo);
}
__device__ __forceinline__ u64 wave_scan64(u64 v) {
  v = dpp_step64<0x111, 0xf>(v);
  v = dpp_step64<0x112, 0xf>(v);
  v = dpp_step64<0x114, 0xf>(v);
  v = dpp_step64<0x118, 0xf>(v);
  v = dpp_step64<0x142, 0xa>(v);
  return dpp_step64<0x143, 0xc>(v);
}
__device__ __forceinline__ u64 lane_of64(u64 v, int lane) {
  return (u64)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
}
__device__ __forceinline__ u64 wave_sum64(u64 v) { return lane_of64(wave_scan64(v), 63); }

struct alignas(16) SampleLds {
  double table[256];  // 2^43 2^(j/256)
  union {
    u64 bins[kBins];
    ulonglong2 picks[kSampleList];  // of a list: place and measure
  };
  u64 seg[kSampleMaxSegs];
  union {
    struct {
      u64 list[kSampleList], w[kSampleList];
    };
    float parts[kParts];
    u64 radix[kRadixBins];
  };
  u64 scan[kWaves];
  u64 found_above;
  float m[kWaves];
  int found, index, count, picked, bad;
};

// A row and its settings.  cut: what is kept so far, places from `cut` up.
template <typename T>
struct Row {
  static constexpr int VE = Logits<T>::N, NV = kSampleSeg / 64 / VE;
  const T *x;
  int V, skew, segs;
  float m;
  double steps;  // 256 log2(e) / T
  u64 cut, least;
  int top_k;
  float temp, top_p, min_p, u;
  bool greedy;

  __device__ __forceinline__ void begin(const SampleArgs &a, int r) {
    x = (const T *)a.logits + (long long)r * a.stride;
    V = a.n_vocab;
    skew = (int)(((uintptr_t)x & 15) / sizeof(T));
    segs = (V + skew + kSampleSeg - 1) / kSampleSeg;
    temp = a.temperature ? a.temperature[r] : 1.f;
    top_p = a.top_p ? a.top_p[r] : 1.f;
    min_p = a.min_p ? a.min_p[r] : 0.f;
    top_k = a.top_k ? a.top_k[r] : 0;
    u = a.uniform[r];
    greedy = temp == 0.f;
    if (greedy || min_p > 1.f) top_k = 1;
    if (top_k >= V || top_k < 0) top_k = 0;
    if (top_k == 1 && top_p == top_p) top_p = 1.f;  // a NaN stays for set_max to find
    cut = 0;
    least = uniform(min_p > 0.f && min_p <= 1.f ? (u64)ceil((double)min_p * kUnit) : 0);
  }
  // False for a row without a distribution; max is NaN where the row holds one.
  __device__ __forceinline__ bool set_max(float max) {
    m = uniform(max);
    steps = uniform(369.32993046757463228 / (greedy ? 1.0 : (double)temp));
    return fabsf(max) < INFINITY && temp >= 0.f && temp < INFINITY && top_p == top_p && min_p == min_p && u == u;
  }
  __device__ bool by_list() const { return top_k > 0 && top_k <= kMostListedK; }

  __device__ __forceinline__ uint4 load(int at) const {  // elements outside the row: -inf
    constexpr uint32_t kNegInf = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
    if (at >= 0 && at + VE <= V) return ldg16(x + at);
    uint32_t w[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
    if (at + VE > 0 && at < V) {
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (at + e >= 0 && at + e < V) {
          if constexpr (sizeof(T) == 4) w[e] = __float_as_uint(x[at + e]);
          else w[e / 2] = e & 1 ? (w[e / 2] & 0xffffu) | (uint32_t)x[at + e] << 16 : (w[e / 2] & 0xffff0000u) | x[at + e];
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // f(segment, first index of vector i's elements, the vectors) for the wave's segments of [s0, s1), the next one's loads in flight.
  template <typename F>
  __device__ __forceinline__ void segments(int s0, int s1, F f) const {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int s = s0 + wave;
    if (s >= s1) return;
    auto first = [&](int seg, int i) { return seg * kSampleSeg - skew + (i * 64 + lane) * VE; };
    uint4 next[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) next[i] = load(first(s, i));
    for (; s < s1; s += kWaves) {
      uint4 v[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = next[i];
      if (s + kWaves < s1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) next[i] = load(first(s + kWaves, i));
      }
      f(s, first(s, 0), v);
    }
  }
  static __device__ int index(int first, int i, int e) { return first + i * 64 * VE + e; }

  // 256 log2 of the weight's share, at least 1 - kSteps: from there on weights are 0.
  __device__ double exponent(float v) const { return fmax(((double)v - (double)m) * steps, (double)(1 - kSteps)); }
  static __device__ int whole(double t) { return (int)(uint32_t)__double_as_longlong(t + 6755399441055744.0); }  // + 1.5 2^52
  // 512 bins for every doubling of 512 - n: nine digits of it as a float
  static constexpr int kBinBits = 14, kBin0 = (127 + 9) << (23 - kBinBits);
  static __device__ int bin_of(int n) { return (int)(__float_as_uint((float)(512 - n)) >> kBinBits) - kBin0; }
  static __device__ int first_step(int b) { return (int)__uint_as_float((uint32_t)(b + kBin0) << kBinBits) - 512; }
  __device__ int bin(float v) const { return bin_of(whole(exponent(v))); }
  // No logit below it lies in bin b or above: b's own floor less a step, and the next lower float.
  __device__ float floor_of_bin(int b) const {
    const float f = (float)((double)m - (first_step(b + 1) + 1) / steps);
    return uniform(f > -INFINITY ? value_of(sample_key(f) - 1) : f);
  }
  // The place within its bin, in 256 parts: larger weights first.
  __device__ int fine_bin(float v, int b) const {
    const int first = first_step(b);
    return min(max((int)((-exponent(v) - first + 0.5) * (256.0 / (first_step(b + 1) - first))), 0), 255);
  }
  // 2^(n/256) from the table, times 2^(h/256) for what is left, |h| <= 1/2: its
  // series in h, in which a^2 h^2 stands for the fourth term's h^4 at the end
  // a = 1/2 and leaves 3.5e-14 at most.  Adding 2^52 rounds to nearest even
  // and leaves the number in the low bits, above which 2^52's own bits are
  // taken off a sum.
  static constexpr u64 kMagicBits = 0x4330000000000000ull;
  __device__ __forceinline__ u64 magic_weight(double t, const double *table) const {
    const double z = t + 6755399441055744.0;
    const int n = (int)(uint32_t)__double_as_longlong(z);
    const double h = t - (z - 6755399441055744.0);
    constexpr double c = 0.0027076061740622862, c4 = c * c * c * c / 24.0;  // c = ln(2) / 256
    double p = fma(h, c * c * c / 6.0, c * c / 2.0 + c4 / 4.0);
    p = fma(p, h, c) * h;
    const double w = table[n & 255], r = fma(w, p, w);
    const u64 bits = (u64)__double_as_longlong(r) + ((u64)((uint32_t)(n >> 8) << 20) << 32);
    return (u64)__double_as_longlong(__longlong_as_double((long long)bits) + 4503599627370496.0);
  }
  __device__ u64 weight(float v, const double *table) const { return magic_weight(exponent(v), table) - kMagicBits; }
  __device__ bool keeps(u64 place) const { return place >= cut; }
};

__device__ __forceinline__ void fill_table(SampleLds &lds) {
  for (int j = threadIdx.x; j < 256; j += kSampleThreads) {
    const double f = j * 0.0027076061740622862;  // ln(2) / 256
    double p = 1.0;
#pragma unroll
    for (int i = 18; i > 0; --i) p = fma(p, f * (1.0 / i), 1.0);  // f below 0.7: the 19th term is under 1e-19
    lds.table[j] = p * kUnit;
  }
}

__device__ __forceinline__ u64 block_sum64(u64 v, SampleLds &lds) {
  v = wave_sum64(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds.scan[threadIdx.x >> 6] = v;
  __syncthreads();
  u64 s = lds.scan[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) s += lds.scan[w];
  return s;
}

// The first of n entries at which the running sum reaches goal >= 1 into
// lds.found, the sum before it into lds.found_above; n where none does.  at(i)
// gives entry i < n.  Called after a barrier, ends with one.
template <typename N, typename At>
__device__ __forceinline__ void find_reach(N n, u64 goal, At at, SampleLds &lds) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int per = (n + kSampleThreads - 1) / kSampleThreads | 1, first = per * tid;  // odd: distinct banks
  u64 sum = 0;
#pragma unroll
  for (int i = 0; i < per; ++i) sum += first + i < n ? at(first + i) : 0;
  u64 incl = wave_scan64(sum);
  if (lane == 63) lds.scan[wave] = incl;
  if (tid == 0) lds.found = n;
  __syncthreads();
  for (int w = 0; w < wave; ++w) incl += lds.scan[w];
  u64 before = incl - sum;
  if (goal > before && goal <= incl) {
    for (int i = 0; i < per; ++i) {
      const u64 w = at(first + i);
      if (goal <= before + w) {
        lds.found = first + i;
        lds.found_above = before;
        break;
      }
      before += w;
    }
  }
  __syncthreads();
}
// As many entries as are known when this is compiled: their reads go out together.
template <int N>
using Bins = std::integral_constant<int, N>;

template <typename N>
__device__ __forceinline__ void clear_bins(SampleLds &lds, N n) {
#pragma unroll
  for (int e = 0; e < (n + kSampleThreads - 1) / kSampleThreads; ++e)
    if (threadIdx.x + e * kSampleThreads < n) lds.bins[threadIdx.x + e * kSampleThreads] = 0;
}
__device__ __forceinline__ void put(SampleLds &lds, u64 place) {
  const int at = atomicAdd(&lds.count, 1);
  if (at < kSampleList) lds.list[at] = place;
}

// ---------------------------------------------------------------- the passes over a row's segments [s0, s1)
// Maximum, NaN where there is one, and the maxima of the parts to part(segment, lane value).
template <typename T, typename Part>
__device__ __forceinline__ float max_pass(const Row<T> &row, int s0, int s1, SampleLds &lds, Part part) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (tid == 0) lds.bad = 0;
  __syncthreads();
  float m = -INFINITY;
  uint32_t largest = 0;  // of the magnitudes' bits: above infinity's there is a NaN
  row.segments(s0, s1, [&](int s, int, const uint4 *v) {
    float mine = -INFINITY;
#pragma unroll
    for (int i = 0; i < Row<T>::NV; ++i)
#pragma unroll
      for (int e = 0; e < Row<T>::VE; ++e) {
        const float x = Logits<T>::at(v[i], e);
        mine = fmaxf(mine, x);
        largest = max(largest, __float_as_uint(x) & 0x7fffffffu);
      }
    part(s, mine);
    m = fmaxf(m, mine);
  });
  m = __int_as_float(wave_reduce(__float_as_int(m), (int)0xff800000u,
                                 [](int a, int b) { return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b))); }));
  if (lane == 0) lds.m[wave] = m;
  if (largest > 0x7f800000u) lds.bad = 1;
  __syncthreads();
  m = lds.m[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) m = fmaxf(m, lds.m[w]);
  return lds.bad ? __uint_as_float(0x7fc00000u) : m;
}

// Eight logits of a lane at a time: enough of their chains side by side, and
// branches for eight together, so that the chains are not cut.
template <typename T, typename F>
__device__ __forceinline__ void eights(const Row<T> &row, int first, const uint4 *v, F f) {
  constexpr int kVectors = 8 / Row<T>::VE;
#pragma unroll
  for (int i = 0; i < Row<T>::NV; i += kVectors) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = Logits<T>::at(v[i + e / Row<T>::VE], e % Row<T>::VE);
    f(x, [&](int e) { return Row<T>::index(first, i + e / Row<T>::VE, e % Row<T>::VE); });
    __builtin_amdgcn_sched_barrier(0);  // more side by side spill more than the 6 to 42 registers of sample_kernel and sample_draw_kernel
  }
}

// The weights of each segment's tokens that the cut keeps and that are `least` or more, by seg(segment, sum).
template <typename T, typename Seg>
__device__ __forceinline__ void mass_pass(const Row<T> &row, int s0, int s1, u64 least, SampleLds &lds, Seg seg) {
  const bool all = row.cut == 0 && least == 0;
  row.segments(s0, s1, [&](int s, int first, const uint4 *v) {
    u64 sum = 0;
    eights(row, first, v, [&](const float *x, auto index) {
      if (all) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += row.magic_weight(row.exponent(x[e]), lds.table);
        sum -= 8 * Row<T>::kMagicBits;
      } else {
        u64 places[8];
        bool some = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          places[e] = place_of(x[e], index(e));
          some |= row.keeps(places[e]);
        }
        if (!__any(some)) return;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const u64 w = row.weight(x[e], lds.table);
          sum += w >= least && row.keeps(places[e]) ? w : 0;
        }
      }
    });
    sum = wave_sum64(sum);
    if ((threadIdx.x & 63) == 0) seg(s, sum);
  });
}

// The measure of every bin into lds.bins, which are clear: weights or counts of what is kept.
template <typename T>
__device__ __forceinline__ void bin_pass(const Row<T> &row, int s0, int s1, bool counts, SampleLds &lds) {
  row.segments(s0, s1, [&](int, int first, const uint4 *v) {
    eights(row, first, v, [&](const float *x, auto index) {
      int b[8];
      u64 w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const double t = row.exponent(x[e]);
        b[e] = Row<T>::bin_of(Row<T>::whole(t));
        w[e] = row.magic_weight(t, lds.table) - Row<T>::kMagicBits;
      }
      if (counts) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = b[e] < kLowest;  // the lowest bin's logits may lie outside the row
      }
      if (row.cut) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = row.keeps(place_of(x[e], index(e))) ? w[e] : 0;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) atomicAdd(&lds.bins[b[e]], w[e]);
    });
  });
}

// put(value, index) for the row's logits from `floor` up, above -infinity.
template <typename T, typename Put>
__device__ __forceinline__ void list_pass(const Row<T> &row, int s0, int s1, float floor, Put put) {
  row.segments(s0, s1, [&](int, int first, const uint4 *v) {
#pragma unroll
    for (int i = 0; i < Row<T>::NV; ++i) {
      float most = Logits<T>::at(v[i], 0);
#pragma unroll
      for (int e = 1; e < Row<T>::VE; ++e) most = fmaxf(most, Logits<T>::at(v[i], e));
      if (!__any(most >= floor)) continue;
#pragma unroll
      for (int e = 0; e < Row<T>::VE; ++e) {
        const float x = Logits<T>::at(v[i], e);
        if (x >= floor && x > -INFINITY) put(x, Row<T>::index(first, i, e));
      }
    }
  });
}

// put(place) for what the row keeps of bin b, and the weights of each segment's tokens in the bins above it.
template <typename T, typename Put, typename Seg>
__device__ __forceinline__ void list_and_mass_pass(const Row<T> &row, int s0, int s1, int b, SampleLds &lds, Put put, Seg seg) {
  const float floor = row.floor_of_bin(b);
  row.segments(s0, s1, [&](int s, int first, const uint4 *v) {
    u64 sum = 0;
    eights(row, first, v, [&](const float *x, auto index) {
      float most = x[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) most = fmaxf(most, x[e]);
      if (!__any(most >= floor)) return;
      int its[8];
      u64 w[8];
      bool here = false;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const double t = row.exponent(x[e]);
        its[e] = Row<T>::bin_of(Row<T>::whole(t));
        w[e] = row.magic_weight(t, lds.table) - Row<T>::kMagicBits;
        here |= its[e] == b;
      }
      if (row.cut | row.least) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = w[e] >= row.least && row.keeps(place_of(x[e], index(e))) ? w[e] : 0;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += its[e] < b ? w[e] : 0;
      if (__any(here)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const u64 place = place_of(x[e], index(e));
          if (its[e] == b && row.keeps(place)) put(place);
        }
      }
    });
    sum = wave_sum64(sum);
    if ((threadIdx.x & 63) == 0) seg(s, sum);
  });
}

// ---------------------------------------------------------------- cuts
// The smallest prefix of what the row keeps whose measure reaches goal >= 1,
// which it does, by histograms over the key's bits: one workgroup, any row.
template <typename T>
__device__ __forceinline__ void cut_by_bits(Row<T> &row, u64 goal, bool counts, SampleLds &lds) {
  constexpr int VE = Row<T>::VE, kTile = kSampleThreads * VE;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, tiles = (row.V + row.skew + kTile - 1) / kTile;
  auto measure = [&](float v) -> u64 { return counts ? 1 : row.weight(v, lds.table); };
  uint32_t prefix = 0;
  int shift = 32;
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass < 2 ? 11 : 10, top = shift, size = 1 << bits;
    shift -= bits;
    __syncthreads();
    for (int i = tid; i < size; i += kSampleThreads) lds.radix[i] = 0;
    __syncthreads();
    for (int i = 0; i < tiles; ++i) {
      const int at = (i * kSampleThreads + tid) * VE - row.skew;
      const uint4 w = row.load(at);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float v = Logits<T>::at(w, e);
        const uint32_t k = sample_key(v);
        if (at + e >= 0 && at + e < row.V && (pass == 0 || k >> top == prefix) && row.keeps(place_of(v, at + e)))
          atomicAdd(&lds.radix[size - 1 - ((k >> shift) & (size - 1))], measure(v));  // the largest values' bin is the first
      }
    }
    __syncthreads();
    const int per = size / kSampleThreads;
    u64 sum = 0;
    for (int i = 0; i < per; ++i) sum += lds.radix[per * tid + i];
    u64 incl = wave_scan64(sum);
    if (lane == 63) lds.scan[wave] = incl;
    __syncthreads();
    for (int w = 0; w < wave; ++w) incl += lds.scan[w];
    u64 before = incl - sum;
    if (goal > before && goal <= incl) {
      for (int i = 0; i < per; ++i) {
        const u64 w = lds.radix[per * tid + i];
        if (goal <= before + w) {
          lds.found = per * tid + i;
          lds.found_above = before;
          break;
        }
        before += w;
      }
    }
    __syncthreads();
    prefix = prefix << bits | (uint32_t)(size - 1 - lds.found);
    goal -= lds.found_above;
  }
  // `goal` of the tokens of value `prefix`, each of the same measure: so many of them, in order of index
  const u64 one = measure(value_of(prefix));
  int left = (int)((goal + one - 1) / one);
  __syncthreads();
  for (int i = 0; i < tiles; ++i) {
    const int at = (i * kSampleThreads + tid) * VE - row.skew;
    const uint4 w = row.load(at);
    auto counts_one = [&](int e) {
      const float v = Logits<T>::at(w, e);
      return at + e >= 0 && at + e < row.V && sample_key(v) == prefix && row.keeps(place_of(v, at + e));
    };
    int mine = 0;
#pragma unroll
    for (int e = 0; e < VE; ++e) mine += counts_one(e);
    int incl = wave_incl_scan(mine);
    __syncthreads();
    if (lane == 63) lds.scan[wave] = incl;
    __syncthreads();
    int all = 0;
    for (int v = 0; v < kWaves; ++v) {
      if (v < wave) incl += (int)lds.scan[v];
      all += (int)lds.scan[v];
    }
    if (left <= incl && left > incl - mine) {
      int n = incl - mine;
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (counts_one(e) && ++n == left) lds.index = at + e;
    }
    left -= all;
    if (left <= 0) break;
  }
  __syncthreads();
  row.cut = uniform((u64)prefix << 32 | (uint32_t)~lds.index);
  __syncthreads();
}

// The weights of the listed places into lds.w.
template <typename T>
__device__ __forceinline__ void weigh_list(const Row<T> &row, SampleLds &lds) {
  for (int i = threadIdx.x; i < lds.count; i += kSampleThreads) lds.w[i] = row.weight(value_of((uint32_t)(lds.list[i] >> 32)), lds.table);
  __syncthreads();
}
// The listed places for which in(i) holds, each with its measure(i), side by
// side into lds.picks.  Called after a barrier, ends with one.
template <typename In, typename Measure>
__device__ __forceinline__ void pick_from_list(In in, Measure measure, SampleLds &lds) {
  if (threadIdx.x == 0) lds.picked = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < lds.count; i += kSampleThreads)
    if (in(i)) lds.picks[atomicAdd(&lds.picked, 1)] = ulonglong2{lds.list[i], measure(i)};
  __syncthreads();
}
// Among the picked places, the one at which the running measure reaches goal;
// over(a, b): place a comes before b.  Ends with a barrier.
template <typename Over, typename Found>
__device__ __forceinline__ void reach_in_picks(u64 goal, Over over, Found found, SampleLds &lds) {
  const int c = lds.picked;
  for (int i = threadIdx.x; i < c; i += kSampleThreads) {
    const ulonglong2 me = lds.picks[i];
    u64 before = 0;
#pragma unroll 8
    for (int j = 0; j < c; ++j) {
      const ulonglong2 other = lds.picks[j];
      before += over(other.x, me.x) ? other.y : 0;
    }
    if (goal > before && goal <= before + me.y) found(me.x);
  }
  __syncthreads();
}
// The cut among the lds.count <= kSampleList listed places that the row
// keeps, of bin b or, for b < 0, of any: the smallest prefix of them whose
// measure reaches goal, which it does.  lds.w holds their weights.
template <typename T>
__device__ __forceinline__ u64 cut_in_list(const Row<T> &row, int b, u64 goal, bool counts, SampleLds &lds) {
  const int tid = threadIdx.x, n = lds.count;
  auto value = [&](int i) { return value_of((uint32_t)(lds.list[i] >> 32)); };
  auto measure = [&](int i) -> u64 { return counts ? 1 : lds.w[i]; };
  if (b < 0) {
    clear_bins(lds, Bins<kBins>());
    __syncthreads();
    for (int i = tid; i < n; i += kSampleThreads)
      if (row.keeps(lds.list[i])) atomicAdd(&lds.bins[row.bin(value(i))], measure(i));
    __syncthreads();
    find_reach(Bins<kBins>(), goal, [&](int i) { return lds.bins[i]; }, lds);
    b = lds.found;
    goal -= lds.found_above;
    __syncthreads();
  }
  auto fine = [&](int i) { return row.keeps(lds.list[i]) && row.bin(value(i)) == b ? row.fine_bin(value(i), b) : -1; };
  clear_bins(lds, Bins<256>());
  __syncthreads();
  for (int i = tid; i < n; i += kSampleThreads) {
    const int f = fine(i);
    if (f >= 0) atomicAdd(&lds.bins[f], measure(i));
  }
  __syncthreads();
  find_reach(Bins<256>(), goal, [&](int i) { return lds.bins[i]; }, lds);
  const int f = lds.found;
  goal -= lds.found_above;
  __syncthreads();
  pick_from_list([&](int i) { return fine(i) == f; }, measure, lds);
  reach_in_picks(goal, [](u64 a, u64 b) { return a > b; }, [&](u64 place) { lds.found_above = place; }, lds);
  const u64 cut = uniform(lds.found_above);
  __syncthreads();
  return cut;
}

// ---------------------------------------------------------------- the drawing
// The weight that top-p wants of a sum.
__device__ __forceinline__ u64 wanted(float top_p, u64 mass) {
  const double goal = ceil((double)top_p * (double)mass);
  return goal >= 1.0 ? (u64)goal : 1;
}
__device__ __forceinline__ u64 goal_of(float u, u64 total) {
  const double g = floor((double)u * (double)total);
  return g > 0.0 ? (g < (double)total ? min((u64)g, total - 1) : total - 1) : 0;
}
template <typename T>
__device__ __forceinline__ void write_result(const SampleArgs &a, const Row<T> &row, int r, int id, float v, u64 total) {
  a.ids[r] = id;
  if (a.logp)
    a.logp[r] = row.greedy ? 0.f : (float)(((double)v - (double)row.m) / (double)row.temp - log((double)total * (1.0 / kUnit)));
}
__device__ __forceinline__ void write_none(const SampleArgs &a, int r) {
  if (threadIdx.x == 0) {
    a.ids[r] = -1;
    if (a.logp) a.logp[r] = __uint_as_float(0x7fc00000u);
  }
}

// By the sums of the row's segments, lds.seg, of what it keeps.
template <typename T>
__device__ __forceinline__ void draw_from_segments(const SampleArgs &a, const Row<T> &row, int r, SampleLds &lds) {
  constexpr int kPer = std::max(kSampleSeg / kSampleThreads, Row<T>::VE);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  u64 total = 0;
  for (int i = tid; i < row.segs; i += kSampleThreads) total += lds.seg[i];
  total = block_sum64(total, lds);
  const u64 goal = goal_of(row.u, total);
  __syncthreads();
  find_reach(row.segs, goal + 1, [&](int i) { return lds.seg[i]; }, lds);
  u64 before = lds.found_above;
  const int at = lds.found * kSampleSeg - row.skew + tid * kPer;
  __syncthreads();
  uint4 v[kPer / Row<T>::VE];
#pragma unroll
  for (int i = 0; i < kPer / Row<T>::VE; ++i) v[i] = row.load(tid * kPer < kSampleSeg ? at + i * Row<T>::VE : INT_MIN);
  u64 w[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const float x = Logits<T>::at(v[i / Row<T>::VE], i % Row<T>::VE);
    w[i] = 0;
    if (row.keeps(place_of(x, at + i))) {
      w[i] = row.weight(x, lds.table);
      if (w[i] < row.least) w[i] = 0;
    }
    sum += w[i];
  }
  u64 incl = wave_scan64(sum);
  if (lane == 63) lds.scan[wave] = incl;
  __syncthreads();
  for (int i = 0; i < wave; ++i) incl += lds.scan[i];
  before += incl - sum;
  if (goal >= before && goal < before + sum) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (goal >= before && goal < before + w[i])
        write_result(a, row, r, at + i, Logits<T>::at(v[i / Row<T>::VE], i % Row<T>::VE), total);
      before += w[i];
    }
  }
}

// Among the lds.count <= kSampleList listed places, which hold at least the
// row's first top_k or all that have a weight.
template <typename T>
__device__ __forceinline__ void draw_from_list(const SampleArgs &a, Row<T> row, int r, SampleLds &lds) {
  const int tid = threadIdx.x, n = lds.count;
  weigh_list(row, lds);
  if (row.top_k < n) row.cut = cut_in_list(row, -1, (u64)row.top_k, true, lds);
  if (row.top_p < 1.f) {
    u64 mass = 0;
    for (int i = tid; i < n; i += kSampleThreads) mass += row.keeps(lds.list[i]) ? lds.w[i] : 0;
    mass = block_sum64(mass, lds);
    __syncthreads();
    row.cut = cut_in_list(row, -1, wanted(row.top_p, mass), false, lds);
  }
  // by index: bins of 2^shift of them
  const int shift = max(0, 32 - __clz(row.V) - 9);
  static_assert(kBins >= 512, "a bin for every 2^shift indexes");
  clear_bins(lds, Bins<512>());
  __syncthreads();
  u64 total = 0;
  auto stays = [&](int i) { return row.keeps(lds.list[i]) && lds.w[i] >= row.least; };
  for (int i = tid; i < n; i += kSampleThreads)
    if (stays(i)) {
      total += lds.w[i];
      atomicAdd(&lds.bins[index_of(lds.list[i]) >> shift], lds.w[i]);
    }
  total = block_sum64(total, lds);
  u64 goal = goal_of(row.u, total) + 1;
  __syncthreads();
  find_reach(Bins<512>(), goal, [&](int i) { return lds.bins[i]; }, lds);
  const int b = lds.found;
  goal -= lds.found_above;
  __syncthreads();
  pick_from_list([&](int i) { return stays(i) && index_of(lds.list[i]) >> shift == b; }, [&](int i) { return lds.w[i]; }, lds);
  reach_in_picks(goal, [](u64 a, u64 b) { return (uint32_t)a > (uint32_t)b; },  // the index's complement
                 [&](u64 place) { write_result(a, row, r, index_of(place), value_of((uint32_t)(place >> 32)), total); }, lds);
}

// ---------------------------------------------------------------- one workgroup's way through a row
// The maxima of a row's parts: 32 logits each, neighbouring lanes' together where a row has more than kParts.
__device__ __forceinline__ int part_shift(int segs) {
  int shift = 0;
  while (segs << (6 - shift) > kParts) ++shift;
  return shift;
}
__device__ __forceinline__ void store_part(float *parts, int shift, int seg, float mine) {
  const int lane = threadIdx.x & 63;
  for (int i = 0; i < shift; ++i) mine = fmaxf(mine, __shfl_xor(mine, 1 << i, 64));
  if ((lane & ((1 << shift) - 1)) == 0) parts[(seg << (6 - shift)) + (lane >> shift)] = mine;
}
// A value that at least top_k of the row's logits reach, or all that have a
// weight: the smallest of the parts' maxima in the bins that top_k of them reach.
template <typename T>
__device__ __forceinline__ float list_floor(const Row<T> &row, const float *parts, SampleLds &lds) {
  const int tid = threadIdx.x, n = row.segs << (6 - part_shift(row.segs));
  clear_bins(lds, Bins<kBins>());
  __syncthreads();
  for (int i = tid; i < n; i += kSampleThreads) {
    const int b = row.bin(parts[i]);
    if (b < kLowest) atomicAdd(&lds.bins[b], 1ull);
  }
  __syncthreads();
  find_reach(Bins<kBins>(), (u64)row.top_k, [&](int i) { return lds.bins[i]; }, lds);
  const int b = __builtin_amdgcn_readfirstlane(lds.found);
  if (b == kBins) return row.floor_of_bin(kLowest - 1);
  float f = INFINITY;
  for (int i = tid; i < n; i += kSampleThreads)
    if (row.bin(parts[i]) <= b) f = fminf(f, parts[i]);
  f = __int_as_float(wave_reduce(__float_as_int(f), 0x7f800000,
                                 [](int a, int b) { return __float_as_int(fminf(__int_as_float(a), __int_as_float(b))); }));
  if ((tid & 63) == 0) lds.m[tid >> 6] = f;
  __syncthreads();
  f = lds.m[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) f = fminf(f, lds.m[w]);
  return uniform(f);
}
// lds.bins' sum, the bin in which top-p's cut lies and what the cut wants of it.
template <typename T>
__device__ __forceinline__ int top_p_bin(const Row<T> &row, u64 *wants, SampleLds &lds) {
  u64 mass = 0;
#pragma unroll
  for (int e = 0; e < kBinsEach; ++e) {
    const int i = threadIdx.x + e * kSampleThreads;
    mass += i < kBins ? lds.bins[i] : 0;
  }
  mass = block_sum64(mass, lds);
  const u64 goal = wanted(row.top_p, mass);
  __syncthreads();
  find_reach(Bins<kBins>(), goal, [&](int i) { return lds.bins[i]; }, lds);
  *wants = goal - lds.found_above;
  return __builtin_amdgcn_readfirstlane(lds.found);
}
// Top-p's cut among the listed places of its bin; those that it keeps join their segments' sums.
template <typename T>
__device__ __forceinline__ void cut_and_add(Row<T> &row, int b, u64 wants, SampleLds &lds) {
  weigh_list(row, lds);
  row.cut = cut_in_list(row, b, wants, false, lds);
  for (int i = threadIdx.x; i < lds.count; i += kSampleThreads)
    if (row.keeps(lds.list[i]) && lds.w[i] >= row.least)
      atomicAdd(&lds.seg[(index_of(lds.list[i]) + row.skew) / kSampleSeg], lds.w[i]);
  __syncthreads();
}

// Whatever a list could not hold.  Begins with a barrier: a caller may have
// filled the table and come straight here, and every wave reads what all of
// them wrote.
template <typename T>
__device__ __attribute__((noinline)) void draw_by_bits(const SampleArgs &a, int r, float m, SampleLds &lds) {
  Row<T> row;
  row.begin(a, r);
  row.set_max(m);
  __syncthreads();
  auto to_seg = [&](int s, u64 sum) { lds.seg[s] = sum; };
  row.cut = 0;
  if (row.top_k > 0) cut_by_bits(row, (u64)row.top_k, true, lds);
  if (row.top_p < 1.f) {
    mass_pass(row, 0, row.segs, 0, lds, to_seg);
    __syncthreads();
    u64 mass = 0;
    for (int i = threadIdx.x; i < row.segs; i += kSampleThreads) mass += lds.seg[i];
    mass = block_sum64(mass, lds);
    cut_by_bits(row, wanted(row.top_p, mass), false, lds);
  }
  mass_pass(row, 0, row.segs, row.least, lds, to_seg);
  __syncthreads();
  draw_from_segments(a, row, r, lds);
}

// A row that does not go by a list of its first top_k; false where a list overflows.
template <typename T>
__device__ __forceinline__ bool draw_by_bins(const SampleArgs &a, Row<T> row, int r, SampleLds &lds) {
  const int tid = threadIdx.x;
  auto to_list = [&](u64 place) { put(lds, place); };
  auto to_seg = [&](int s, u64 sum) { lds.seg[s] = sum; };
  if (row.top_k > 0) {
    clear_bins(lds, Bins<kBins>());
    if (tid == 0) lds.count = 0;
    __syncthreads();
    bin_pass(row, 0, row.segs, true, lds);
    __syncthreads();
    find_reach(Bins<kBins>(), (u64)row.top_k, [&](int i) { return lds.bins[i]; }, lds);
    if (lds.found < kBins) {  // else fewer have a weight
      const int b = lds.found;
      const u64 wants = (u64)row.top_k - lds.found_above;
      list_and_mass_pass(row, 0, row.segs, b, lds, to_list, [](int, u64) {});
      __syncthreads();
      if (lds.count > kSampleList) return false;
      row.cut = cut_in_list(row, b, wants, true, lds);
    }
    __syncthreads();
  }
  if (row.top_p < 1.f) {
    clear_bins(lds, Bins<kBins>());
    if (tid == 0) lds.count = 0;
    __syncthreads();
    bin_pass(row, 0, row.segs, false, lds);
    __syncthreads();
    u64 wants;
    const int b = top_p_bin(row, &wants, lds);
    list_and_mass_pass(row, 0, row.segs, b, lds, to_list, to_seg);
    __syncthreads();
    if (lds.count > kSampleList) return false;
    cut_and_add(row, b, wants, lds);
  } else {
    mass_pass(row, 0, row.segs, row.least, lds, to_seg);
    __syncthreads();
  }
  draw_from_segments(a, row, r, lds);
  return true;
}

// Grid: rows.
template <typename T>
__global__ __launch_bounds__(kSampleThreads, 4) void sample_kernel(SampleArgs a) {
  __shared__ SampleLds lds;
  const int r = blockIdx.x;
  Row<T> row;
  row.begin(a, r);
  fill_table(lds);
  const bool by_list = row.by_list();
  const int shift = part_shift(row.segs);
  const float m = max_pass(row, 0, row.segs, lds, [&](int s, float mine) {
    if (by_list) store_part(lds.parts, shift, s, mine);
  });
  if (!row.set_max(m)) {
    write_none(a, r);
    return;
  }
  bool done;
  if (by_list) {
    const float floor = list_floor(row, lds.parts, lds);
    if (threadIdx.x == 0) lds.count = 0;
    __syncthreads();
    list_pass(row, 0, row.segs, floor, [&](float v, int i) { put(lds, place_of(v, i)); });
    __syncthreads();
    done = lds.count <= kSampleList;
    if (done) draw_from_list(a, row, r, lds);
  } else {
    done = draw_by_bins(a, row, r, lds);
  }
  if (!done) draw_by_bits<T>(a, r, m, lds);
}

// ---------------------------------------------------------------- few rows: a row on several workgroups
// What the workgroups of a row leave each other; nothing of it is read before it is written.
struct SampleRow {
  float max[kSampleMaxChunks];
  int count, bin;
  u64 wants;
  float parts[kParts];
  u64 list[kSampleList];
  u64 seg[kSampleMaxSegs];
  u64 bins[1][kBins];  // a chunk's each
};
size_t sample_row_bytes(int chunks) { return sizeof(SampleRow) + (chunks - 1) * kBins * sizeof(u64); }
__device__ __forceinline__ SampleRow &row_record(const SampleArgs &a, int r) {
  return *(SampleRow *)((char *)a.rows + r * (sizeof(SampleRow) + (a.chunks - 1) * kBins * sizeof(u64)));
}

struct Chunk {
  int r, c, s0, s1;
  __device__ Chunk(const SampleArgs &a, int segs) {
    r = blockIdx.x / a.chunks;
    c = blockIdx.x - r * a.chunks;
    const int per = (segs + a.chunks - 1) / a.chunks;
    s0 = min(c * per, segs);
    s1 = min(s0 + per, segs);
  }
};
template <typename T>
__device__ __forceinline__ bool max_of_chunks(const SampleArgs &a, const SampleRow &w, Row<T> &row) {
  const int lane = threadIdx.x & 63;
  static_assert(kSampleMaxChunks <= 64, "a lane for every chunk");
  const float mine = lane < a.chunks ? w.max[lane] : -INFINITY;
  const float m = __int_as_float(wave_reduce(__float_as_int(mine), (int)0xff800000u,
                                             [](int a, int b) { return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b))); }));
  return row.set_max(__any(mine != mine) ? __uint_as_float(0x7fc00000u) : m);
}
// The workgroup's list joins the row's: one reservation, as every trip to
// memory's counter is a microsecond.  Called after a barrier.
__device__ __forceinline__ void join_list(SampleRow &w, SampleLds &lds) {
  const int n = lds.count;
  if (n == 0) return;
  if (threadIdx.x == 0) lds.index = __hip_atomic_fetch_add(&w.count, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  for (int i = threadIdx.x; i < min(n, kSampleList); i += kSampleThreads)
    if (lds.index + i < kSampleList) w.list[lds.index + i] = lds.list[i];
}

// Grid of these three: rows x chunks.  Maxima.
template <typename T>
__global__ __launch_bounds__(kSampleThreads, 4) void sample_max_kernel(SampleArgs a) {
  __shared__ SampleLds lds;
  Row<T> row;
  row.begin(a, blockIdx.x / a.chunks);
  const Chunk k(a, row.segs);
  SampleRow &w = row_record(a, k.r);
  const bool by_list = row.by_list();
  const int shift = part_shift(row.segs);
  const float m = max_pass(row, k.s0, k.s1, lds, [&](int s, float mine) {
    if (by_list) store_part(w.parts, shift, s, mine);
  });
  if (threadIdx.x == 0) {
    w.max[k.c] = m;
    if (k.c == 0) w.count = 0;
  }
}

// The lists of rows that go by one, top-p's bins, the sums of rows without a cut.
template <typename T>
__global__ __launch_bounds__(kSampleThreads, 4) void sample_sum_kernel(SampleArgs a) {
  __shared__ SampleLds lds;
  Row<T> row;
  row.begin(a, blockIdx.x / a.chunks);
  const Chunk k(a, row.segs);
  SampleRow &w = row_record(a, k.r);
  if (!max_of_chunks(a, w, row)) return;
  if (row.by_list()) {
    const float floor = list_floor(row, w.parts, lds);
    if (threadIdx.x == 0) lds.count = 0;
    __syncthreads();
    list_pass(row, k.s0, k.s1, floor, [&](float v, int i) { put(lds, place_of(v, i)); });
    __syncthreads();
    join_list(w, lds);
  } else if (row.top_k == 0) {
    fill_table(lds);
    if (row.top_p < 1.f) {
      clear_bins(lds, Bins<kBins>());
      __syncthreads();
      bin_pass(row, k.s0, k.s1, false, lds);
      __syncthreads();
      for (int i = threadIdx.x; i < kBins; i += kSampleThreads) w.bins[k.c][i] = lds.bins[i];
    } else {
      __syncthreads();
      mass_pass(row, k.s0, k.s1, row.least, lds, [&](int s, u64 sum) { w.seg[s] = sum; });
    }
  }
}

// Top-p: the bin of the cut from all chunks' bins, its list, the sums above it.
template <typename T>
__global__ __launch_bounds__(kSampleThreads, 4) void sample_list_kernel(SampleArgs a) {
  __shared__ SampleLds lds;
  Row<T> row;
  row.begin(a, blockIdx.x / a.chunks);
  if (!(row.top_p < 1.f) || row.top_k > 0) return;
  const Chunk k(a, row.segs);
  SampleRow &w = row_record(a, k.r);
  if (!max_of_chunks(a, w, row)) return;
  fill_table(lds);
  u64 sums[kBinsEach] = {};
#pragma unroll 3
  for (int c = 0; c < a.chunks; ++c)
#pragma unroll
    for (int e = 0; e < kBinsEach; ++e) sums[e] += w.bins[c][min((int)threadIdx.x + e * kSampleThreads, kBins - 1)];
#pragma unroll
  for (int e = 0; e < kBinsEach; ++e)
    if (threadIdx.x + e * kSampleThreads < kBins) lds.bins[threadIdx.x + e * kSampleThreads] = sums[e];
  __syncthreads();
  u64 wants;
  const int b = top_p_bin(row, &wants, lds);
  if (k.c == 0 && threadIdx.x == 0) {
    w.bin = b;
    w.wants = wants;
  }
  if (threadIdx.x == 0) lds.count = 0;
  __syncthreads();
  list_and_mass_pass(row, k.s0, k.s1, b, lds, [&](u64 place) { put(lds, place); }, [&](int s, u64 sum) { w.seg[s] = sum; });
  __syncthreads();
  join_list(w, lds);
}

// Grid: rows.  The drawing.
template <typename T>
__global__ __launch_bounds__(kSampleThreads, 4) void sample_draw_kernel(SampleArgs a) {
  __shared__ SampleLds lds;
  const int r = blockIdx.x, tid = threadIdx.x;
  Row<T> row;
  row.begin(a, r);
  const SampleRow &w = row_record(a, r);
  if (!max_of_chunks(a, w, row)) {
    write_none(a, r);
    return;
  }
  fill_table(lds);
  const bool by_list = row.by_list(), listed = by_list || row.top_p < 1.f;
  const int n = listed && (by_list || row.top_k == 0) ? w.count : 0;
  if (tid == 0) lds.count = n;
  bool done = n <= kSampleList;
  if (row.top_k > 0 && !by_list) {
    __syncthreads();
    done = draw_by_bins(a, row, r, lds);
  } else if (done) {
    for (int i = tid; i < n; i += kSampleThreads) lds.list[i] = w.list[i];
    if (!by_list)
      for (int i = tid; i < row.segs; i += kSampleThreads) lds.seg[i] = w.seg[i];
    __syncthreads();
    if (by_list) {
      draw_from_list(a, row, r, lds);
    } else {
      if (listed) cut_and_add(row, w.bin, w.wants, lds);
      draw_from_segments(a, row, r, lds);
    }
  }
  if (!done) draw_by_bits<T>(a, r, row.m, lds);
}

// ---------------------------------------------------------------- launcher
// Workgroups of a row: one where the rows alone fill the card, otherwise
// enough of them that every wave has a segment.  With one and with more, us:
// top-p of 64 rows of 32000 37 30, of 128 37 35, of 200 38 42, without a cut 17
// 17, 17 19, 17 22, top-p of one row of 131071 152 31.  A second workgroup of a
// row is worth its launches up to 256 rows where rows are long.
int sample_chunks(int n, int n_vocab, int dtype) {
  const int ve = dtype == 0 ? 4 : 8;
  const int segs = (n_vocab + ve - 1 + kSampleSeg - 1) / kSampleSeg;  // a row may begin up to ve - 1 elements into its first vector
  const int fill = n_vocab <= 65536 ? 256 : 512;
  return std::max(1, std::min({(segs + kWaves - 1) / kWaves, fill / n, kSampleMaxChunks}));
}

template <typename T>
static hipError_t launch(const SampleArgs &a, hipStream_t st) {
  const dim3 block(kSampleThreads), rows(a.n), parts(a.n * a.chunks);
  if (a.chunks == 1) {
    hipLaunchKernelGGL((sample_kernel<T>), rows, block, 0, st, a);
  } else {
    hipLaunchKernelGGL((sample_max_kernel<T>), parts, block, 0, st, a);
    hipLaunchKernelGGL((sample_sum_kernel<T>), parts, block, 0, st, a);
    if (a.top_p) hipLaunchKernelGGL((sample_list_kernel<T>), parts, block, 0, st, a);
    hipLaunchKernelGGL((sample_draw_kernel<T>), rows, block, 0, st, a);
  }
  return hipGetLastError();
}
hipError_t launch_sample(const SampleArgs &a, int dtype, hipStream_t st) { return dtype == 0 ? launch<float>(a, st) : launch<u16>(a, st); }

}  // namespace lora
