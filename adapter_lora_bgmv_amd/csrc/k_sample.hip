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
// So a row needs one cut in that order: a value's key and the last index that
// is kept among its equals.  Tokens are then run through by index, and the
// first at which the running sum exceeds floor(u sum) is the row's.
//
// A cut is found by three histograms over the key's bits (11, 11 and 10), each
// over the tokens of the bin that the one before found, counts for top-k and
// weights for top-p, and the cut among equals by a count in order of index.
#include <climits>

#include "common.hpp"
#include "verify.hpp"

namespace lora {

typedef unsigned long long u64;
constexpr int kSampleBins = 2048;

__device__ __forceinline__ uint32_t sample_key(float x) {  // unsigned order is the value's; the zeros are equal
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

template <typename T>
struct Logits;
template <>
struct Logits<float> {
  static constexpr int N = 4;
  static __device__ float at(const uint4 &v, int e) {
    return __uint_as_float(e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w);
  }
  static __device__ float one(const float *p) { return *p; }
};
template <>
struct Logits<u16> {
  static constexpr int N = 8;
  static __device__ float at(const uint4 &v, int e) {
    const uint32_t w = e < 2 ? v.x : e < 4 ? v.y : e < 6 ? v.z : v.w;
    return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
  }
  static __device__ float one(const u16 *p) { return bf2f(*p); }
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

// 2^43 2^t rounded to a whole number, for t <= 0.  Taylor's series of 2^f on
// [-1/2, 1/2], to 1e-14; adding 2^52 rounds to nearest even and leaves the
// number in the low bits.
__device__ __forceinline__ u64 weight_of(double t) {
  t = fmax(t, -64.0);  // rounds to 0 from -44 on; NaN is kept out by the callers
  const double n = rint(t), f = (t - n) * 0.69314718055994530942;
  double p = 1.0 / 479001600.0;
  p = fma(p, f, 1.0 / 39916800.0);
  p = fma(p, f, 1.0 / 3628800.0);
  p = fma(p, f, 1.0 / 362880.0);
  p = fma(p, f, 1.0 / 40320.0);
  p = fma(p, f, 1.0 / 5040.0);
  p = fma(p, f, 1.0 / 720.0);
  p = fma(p, f, 1.0 / 120.0);
  p = fma(p, f, 1.0 / 24.0);
  p = fma(p, f, 1.0 / 6.0);
  p = fma(p, f, 0.5);
  p = fma(p, f, 1.0);
  p = fma(p, f, 1.0);
  const double w = ldexp(p, (int)n + 43) + 4503599627370496.0;
  return (u64)__double_as_longlong(w) & 0xfffffffffffffull;
}

struct SampleLds {
  u64 bins[kSampleBins];

  u64 scan[4];
  u64 found_above;
  int found, index;
  float m[4];
  int bad;
};

// The row, as the kernel's phases see it.
template <typename T>
struct Row {
  static constexpr int VE = Logits<T>::N;
  const T *x;
  int V, skew, tiles;  // a tile: VE logits of every thread
  float m;
  double per;  // log2(e) / T

  __device__ uint4 load(int at) const {  // elements outside the row: -inf
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
  __device__ int first(int tile) const { return (tile * kSampleThreads + (int)threadIdx.x) * VE - skew; }
  __device__ u64 weight(float v) const { return weight_of(((double)v - (double)m) * per); }
  // f(value, index) for every logit of the thread's
  template <typename F>
  __device__ void each(F f) const {
    for (int i = 0; i < tiles; ++i) {
      const int at = first(i);
      const uint4 w = load(at);
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (at + e >= 0 && at + e < V) f(Logits<T>::at(w, e), at + e);
    }
  }
};

// What is kept so far: tokens above `key`, and equal ones up to `index`.
struct Cut {
  uint32_t key;
  int index;
  __device__ bool keeps(uint32_t k, int i) const { return k > key || (k == key && i <= index); }
};

__device__ __forceinline__ u64 block_sum64(u64 v, SampleLds &lds) {
  v = lane_of64(wave_scan64(v), 63);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds.scan[threadIdx.x >> 6] = v;
  __syncthreads();
  return lds.scan[0] + lds.scan[1] + lds.scan[2] + lds.scan[3];
}

// The smallest prefix of what `cut` keeps whose measure reaches goal >= 1, as
// a cut; the whole measure reaches it.  measure(value) is the same for equal values.
template <typename T, typename M>
__device__ Cut cut_at(const Row<T> &row, const Cut &cut, u64 goal, M measure, SampleLds &lds) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int kPer = kSampleBins / kSampleThreads;
  uint32_t prefix = 0;  // of the key looked for, the bits above `shift + bits`
  int shift = 32;
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass < 2 ? 11 : 10, top = shift;
    shift -= bits;
    for (int i = tid; i < kSampleBins; i += kSampleThreads) lds.bins[i] = 0;
    __syncthreads();
    row.each([&](float v, int i) {
      const uint32_t k = sample_key(v);
      if ((pass == 0 || k >> top == prefix) && cut.keeps(k, i)) atomicAdd(&lds.bins[(k >> shift) & ((1u << bits) - 1)], measure(v));
    });
    __syncthreads();
    // from the largest bin down: thread t has bins n - 1 - kPer t and the ones below
    u64 sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += lds.bins[kSampleBins - 1 - (kPer * tid + i)];
    u64 incl = wave_scan64(sum);
    if (lane == 63) lds.scan[wave] = incl;
    __syncthreads();
    for (int w = 0; w < wave; ++w) incl += lds.scan[w];
    u64 at = incl - sum;
    if (goal > at && goal <= incl) {
      for (int i = 0; i < kPer; ++i) {
        const int b = kSampleBins - 1 - (kPer * tid + i);
        const u64 w = lds.bins[b];
        if (goal <= at + w) {
          lds.found = b;
          lds.found_above = at;
          break;
        }
        at += w;
      }
    }
    __syncthreads();
    prefix = prefix << bits | (uint32_t)lds.found;
    goal -= lds.found_above;
    __syncthreads();
  }
  // `goal` of the tokens of value `prefix`, each of the same measure: so many of them, in order of index
  const uint32_t key = prefix;
  const uint32_t b = key & 0x80000000u ? key ^ 0x80000000u : ~key;
  const u64 one = measure(__uint_as_float(b));
  int left = (int)((goal + one - 1) / one);
  if (tid == 0) lds.index = INT_MAX;
  for (int i = 0; i < row.tiles; ++i) {
    const int at = row.first(i);
    const uint4 w = row.load(at);
    int mine = 0;
#pragma unroll
    for (int e = 0; e < Row<T>::VE; ++e)
      if (at + e >= 0 && at + e < row.V) mine += sample_key(Logits<T>::at(w, e)) == key && cut.keeps(key, at + e);
    int incl = wave_incl_scan(mine);
    __syncthreads();
    if (lane == 63) lds.scan[wave] = incl;
    __syncthreads();
    for (int v = 0; v < wave; ++v) incl += (int)lds.scan[v];
    const int all = (int)(lds.scan[0] + lds.scan[1] + lds.scan[2] + lds.scan[3]);
    if (left <= incl && left > incl - mine) {
      int n = incl - mine;
#pragma unroll
      for (int e = 0; e < Row<T>::VE; ++e)
        if (at + e >= 0 && at + e < row.V && sample_key(Logits<T>::at(w, e)) == key && cut.keeps(key, at + e) && ++n == left)
          lds.index = at + e;
    }
    left -= all;
    if (left <= 0) break;
  }
  __syncthreads();
  const Cut got = {key, lds.index};
  __syncthreads();
  return got;
}

template <typename T>
__global__ __launch_bounds__(kSampleThreads) void sample_kernel(SampleArgs a) {
  constexpr int VE = Logits<T>::N;
  __shared__ SampleLds lds;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = blockIdx.x;
  Row<T> row;
  row.x = (const T *)a.logits + (long long)r * a.stride;
  row.V = a.n_vocab;
  row.skew = (int)(((uintptr_t)row.x & 15) / sizeof(T));
  row.tiles = (a.n_vocab + row.skew + VE * kSampleThreads - 1) / (VE * kSampleThreads);
  const float temp = a.temperature ? a.temperature[r] : 1.f;
  const float top_p = a.top_p ? a.top_p[r] : 1.f, min_p = a.min_p ? a.min_p[r] : 0.f, u = a.uniform[r];
  int top_k = a.top_k ? a.top_k[r] : 0;

  float m = -INFINITY;
  bool nan = false;
  row.each([&](float v, int) {
    m = fmaxf(m, v);
    nan |= v != v;
  });
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  if (tid == 0) lds.bad = 0;
  __syncthreads();
  if (lane == 0) lds.m[wave] = m;
  if (nan) lds.bad = 1;
  __syncthreads();
  m = fmaxf(fmaxf(lds.m[0], lds.m[1]), fmaxf(lds.m[2], lds.m[3]));
  const bool none = lds.bad || !(fabsf(m) < INFINITY) || !(temp >= 0.f && temp < INFINITY) || top_p != top_p || min_p != min_p || u != u;
  if (none) {
    if (tid == 0) {
      a.ids[r] = -1;
      if (a.logp) a.logp[r] = __uint_as_float(0x7fc00000u);
    }
    return;
  }
  const bool greedy = temp == 0.f;
  row.m = m;
  row.per = 1.4426950408889634 / (greedy ? 1.0 : (double)temp);
  if (greedy || min_p > 1.f) top_k = 1;

  Cut cut = {0, INT_MAX};
  if (top_k > 0 && top_k < a.n_vocab) cut = cut_at(row, cut, (u64)top_k, [](float) -> u64 { return 1; }, lds);
  if (top_p < 1.f && top_k != 1) {
    u64 mass = 0;
    row.each([&](float v, int i) {
      if (cut.keeps(sample_key(v), i)) mass += row.weight(v);
    });
    mass = block_sum64(mass, lds);
    const double goal = ceil((double)top_p * (double)mass);
    cut = cut_at(row, cut, goal >= 1.0 ? (u64)goal : 1, [&](float v) { return row.weight(v); }, lds);
  }
  const u64 least = min_p > 0.f && min_p <= 1.f ? (u64)ceil((double)min_p * 8796093022208.0) : 0;
  auto kept = [&](float v, int i) -> u64 {
    const uint32_t k = sample_key(v);
    if (!cut.keeps(k, i)) return 0;
    const u64 w = row.weight(v);
    return w >= least ? w : 0;
  };

  u64 total = 0;
  row.each([&](float v, int i) { total += kept(v, i); });
  total = block_sum64(total, lds);
  const double g = floor((double)u * (double)total);
  const u64 goal = g > 0.0 ? (g < (double)total ? (u64)g : total - 1) : 0;

  // by index: the first token at which the running sum exceeds the goal
  u64 before = 0;
  for (int i = 0; i < row.tiles; ++i) {
    const int at = row.first(i);
    const uint4 w = row.load(at);
    u64 mine = 0;
#pragma unroll
    for (int e = 0; e < VE; ++e)
      if (at + e >= 0 && at + e < a.n_vocab) mine += kept(Logits<T>::at(w, e), at + e);
    u64 incl = wave_scan64(mine);
    __syncthreads();
    if (lane == 63) lds.scan[wave] = incl;
    __syncthreads();
    u64 base = before;
    for (int v = 0; v < wave; ++v) base += lds.scan[v];
    incl += base;
    const u64 all = lds.scan[0] + lds.scan[1] + lds.scan[2] + lds.scan[3];
    if (goal < incl && goal >= incl - mine) {
      u64 n = incl - mine;
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (at + e >= 0 && at + e < a.n_vocab) {
          const float v = Logits<T>::at(w, e);
          const u64 one = kept(v, at + e);
          if (goal >= n && goal < n + one) {
            a.ids[r] = at + e;
            if (a.logp)
              a.logp[r] = greedy ? 0.f : (float)(((double)v - (double)m) / (double)temp - log((double)total * (1.0 / 8796093022208.0)));
          }
          n += one;
        }
    }
    before += all;
    if (goal < before) break;
  }
}

hipError_t launch_sample(const SampleArgs &a, int dtype, hipStream_t st) {
  const dim3 grid(a.n), block(kSampleThreads);
  if (dtype == 0) hipLaunchKernelGGL((sample_kernel<float>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((sample_kernel<u16>), grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace lora
