// k_score.hip -- log probabilities of given tokens, with entropy, rank and the top alternatives.
//
// For a row x of n_vocab logits, m its maximum and s = sum exp(x - m):
//     logp   = x[id] - m - log s,
//     entropy = log s - sum exp(x - m) (x - m) / s,
//     rank   = 1 + the number of logits above x[id],
//     top    = the `top` largest by (value, lower index first).
// One pass over the logits: a workgroup of 256 threads streams a row (or a
// chunk of it, where rows are few), a batch of 32 logits a thread at a time
// with the next batch's loads in flight, and every thread keeps its own
// running maximum, sums and count; they meet once at the end.  The
// exponentials run in base 2, t = (x - m) log2(e): the difference first, so
// that rows of the type's lowest value stay finite.
//
// Top: the order is that of 64-bit keys, the value's bits in unsigned order
// above the complement of the index, all of them different.  Of the 64
// lanes' maxima a wave finds (by ballots, bit after bit) a value that `top`
// of them reach: no smaller logit can be among the `top`.  A lane whose batch
// reaches it puts the batch's maximum and number on a list in LDS, and the
// wave's value is found anew; after a few batches that is rare.  At the end
// the batches on the list whose maximum reaches the largest of the four
// waves' values are read again (they are few: 32 logits each), and an entry's
// place among what reaches it is the number of larger keys.  Where a list
// overflows (equal or rising logits) the whole chunk is read again for what
// reaches the final value, and where even that is too much, once for every
// place.
//
// A row of several chunks leaves a record of each in the workspace; the last
// chunk to arrive joins them, the lists by the same selection.
//
// HBM bounds large calls (4096 rows of 32000 bf16 logits: 58 us, 4.5 TB/s) and
// the exponentials and compares follow closely, 14 vector instructions a
// logit; latency bounds small ones (36 rows of 131071: 17 us).
#include <algorithm>

#include "common.hpp"
#include "verify.hpp"

namespace lora {

constexpr int kScoreList = 1024;  // entries of the LDS list
typedef unsigned long long u64;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// Unsigned order of an f32's bits is its value's order; the zeros are equal (-0 + 0 is 0).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
// NaN of either sign is above everything, so that the keys of a row reach what its maximum reaches.
__device__ __forceinline__ u64 key_of(float x, uint32_t index) {
  return (u64)(x == x ? ordered(x) : ~0u) << 32 | (uint32_t)~index;
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ float at(const uint4 &v, int e) {
    return __uint_as_float(e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w);
  }
  static __device__ float one(const float *p) { return *p; }
};
template <>
struct Vec<u16> {
  static constexpr int N = 8;
  static __device__ float at(const uint4 &v, int e) {
    const uint32_t w = e < 2 ? v.x : e < 4 ? v.y : e < 6 ? v.z : v.w;
    return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
  }
  static __device__ float one(const u16 *p) { return bf2f(*p); }
};

__device__ __forceinline__ float wave_sum(float v) {
  return __int_as_float(wave_reduce(__float_as_int(v), 0, [](int a, int b) { return __float_as_int(__int_as_float(a) + __int_as_float(b)); }));
}
__device__ __forceinline__ float wave_max(float v) {
  return __int_as_float(wave_reduce(__float_as_int(v), (int)0xff800000u,
                                    [](int a, int b) { return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b))); }));
}

// A lower bound of the k-th largest of the wave's 64 keys: its upper 16 bits.
__device__ __forceinline__ uint32_t kth_floor(uint32_t key, int k) {
  uint32_t t = 0;
#pragma unroll
  for (int bit = 31; bit >= 16; --bit) {
    const uint32_t c = t | 1u << bit;
    if (__popcll(__ballot(key >= c)) >= k) t = c;
  }
  return t;
}

struct ScoreLds {
  u64 list[kScoreList], kept[kScoreList];
  uint32_t pick[kScoreList];
  u64 top[kScoreMaxTop];
  u64 red[4];
  float m[4], s[4], sx[4];
  uint32_t floor[4];
  int above[4];
  int count, kept_count, picks;
  unsigned arrived;
};

// Puts a key on a list in LDS; what no longer fits is only counted.
__device__ __forceinline__ void put(u64 *list, int *count, u64 key) {
  const int at = atomicAdd(count, 1);
  if (at < kScoreList) list[at] = key;
}

// The `k` largest keys into lds.top, in order (0 where there are fewer).
// `floor`: a value (upper half) that at least k of the keys reach, if there
// are k.  lds.kept holds the lds.kept_count keys that reach it, unless `all`:
// then each(f) calls f(key) for all of the thread's keys.  Called by the
// whole workgroup after a barrier; ends with one.
template <typename Each>
__device__ __forceinline__ void rank_top(int k, uint32_t floor, bool all, Each each, ScoreLds &lds) {
  const int tid = threadIdx.x;
  if (tid < k) lds.top[tid] = 0;
  if (all) {
    if (tid == 0) lds.kept_count = 0;
    __syncthreads();
    each([&](u64 key) {
      if ((uint32_t)(key >> 32) >= floor) put(lds.kept, &lds.kept_count, key);
    });
  }
  __syncthreads();
  const int kept = lds.kept_count;
  if (kept <= kScoreList) {
    for (int c = tid; c < kept; c += kScoreThreads) {
      const u64 mine = lds.kept[c];
      int above = 0;
#pragma unroll 4
      for (int i = 0; i < kept; ++i) above += lds.kept[i] > mine;
      if (above < k) lds.top[above] = mine;
    }
    __syncthreads();
    return;
  }
  u64 last = ~0ull;
  for (int r = 0; r < k; ++r) {
    u64 best = 0;
    each([&](u64 key) {
      if (key < last && key > best) best = key;
    });
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
      const u64 o = __shfl_xor(best, off, 64);
      best = o > best ? o : best;
    }
    if ((tid & 63) == 0) lds.red[tid >> 6] = best;
    __syncthreads();
    best = lds.red[0];
#pragma unroll
    for (int w = 1; w < 4; ++w) best = lds.red[w] > best ? lds.red[w] : best;
    if (tid == 0) lds.top[r] = best;
    last = best;
    __syncthreads();
  }
}

// The results of a row from its maximum, sums, count and lds.top.
__device__ __forceinline__ void finish(const ScoreArgs &a, int row, int id, float xt, float m, float s, float sx, int above,
                                       const ScoreLds &lds) {
  const int tid = threadIdx.x;
  const float ls = s == 0.f ? 0.f : __builtin_amdgcn_logf(s);  // log2; s is 0 where every logit is -inf
  const bool there = (unsigned)id < (unsigned)a.n_vocab;
  if (tid == 0) {
    // NaN or +inf in the row makes s NaN, and with it these
    if (a.logp) a.logp[row] = there ? (xt - m) - kLn2 * ls : s == s ? -INFINITY : s;
    if (a.entropy) a.entropy[row] = s == 0.f ? 0.f : kLn2 * (ls - sx / s);
    if (a.rank) a.rank[row] = there ? above + 1 : 0;
  }
  if (tid < a.top) {
    const u64 key = lds.top[tid];
    a.top_ids[(size_t)row * a.top + tid] = (int32_t)~(uint32_t)key;
    a.top_logp[(size_t)row * a.top + tid] = (from_ordered((uint32_t)(key >> 32)) - m) - kLn2 * ls;
  }
}

template <typename T>
__global__ __launch_bounds__(kScoreThreads) void score_kernel(ScoreArgs a) {
  constexpr int VE = Vec<T>::N, NV = kScoreBatch / VE, kStride = kScoreThreads * VE;
  __shared__ ScoreLds lds;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row = blockIdx.x / a.chunks, chunk = blockIdx.x - row * a.chunks;
  const T *x = (const T *)a.logits + (long long)row * a.stride;
  // the grid of vectors begins at the 16-byte line that holds the row's first element
  const int skew = (int)(((uintptr_t)x & 15) / sizeof(T));
  const int begin = chunk * a.batches * (NV * kStride) - skew + tid * VE;  // index of the thread's first element
  const int id = a.ids[row];
  if (tid == 0) lds.count = lds.kept_count = lds.picks = 0;
  __syncthreads();

  constexpr uint32_t kNegInf = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
  auto load = [&](int at) -> uint4 {  // elements outside the row: -inf
    if (at >= 0 && at + VE <= a.n_vocab) return ldg16(x + at);
    uint32_t w[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
    if (at + VE > 0 && at < a.n_vocab) {
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (at + e >= 0 && at + e < a.n_vocab) {
          if constexpr (sizeof(T) == 4) w[e] = __float_as_uint(x[at + e]);
          else w[e / 2] = e & 1 ? (w[e / 2] & 0xffffu) | (uint32_t)x[at + e] << 16 : (w[e / 2] & 0xffff0000u) | x[at + e];
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  };
  uint4 next[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) next[i] = load(begin + i * kStride);
  const bool there = (unsigned)id < (unsigned)a.n_vocab;
  const float xt = there ? Vec<T>::one(x + id) : INFINITY;  // nothing is above +inf

  float m = -INFINITY, s = 0.f, sx = 0.f;  // the thread's maximum, and its sums against it
  int above = 0;                           // the wave's
  uint32_t floor = 0;                      // `top` of the wave's lanes reach it
  for (int b = 0; b < a.batches; ++b) {
    const int first = begin + b * (NV * kStride);
    if (b * (NV * kStride) + begin - tid * VE >= a.n_vocab) break;  // the last chunk may hold fewer
    uint4 v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = next[i];
    if (b + 1 < a.batches) {
#pragma unroll
      for (int i = 0; i < NV; ++i) next[i] = load(first + (NV + i) * kStride);
    }
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VE; ++e) mx = fmaxf(mx, Vec<T>::at(v[i], e));
    if (__any(mx > m)) {
      const float mn = fmaxf(m, mx);
      const float by = m == -INFINITY ? 0.f : (m - mn) * kLog2e;  // with no maximum yet the sums are 0
      const float f = __builtin_amdgcn_exp2f(by);
      sx = (sx + (f == 0.f ? 0.f : s * by)) * f;
      s *= f;
      m = mn;
    }
    const bool holds = first < a.n_vocab;  // the lane has an element of the row in this batch
    if (a.top && __any(holds && ordered(mx) >= floor)) {
      // lanes without elements count as lower than any
      floor = max(floor, kth_floor(begin < a.n_vocab ? ordered(m) : 0u, a.top));
      if (holds && ordered(mx) >= floor) put(lds.list, &lds.count, (u64)ordered(mx) << 32 | (uint32_t)(b * kScoreThreads + tid));
    }
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float y = Vec<T>::at(v[i], e);
        const float t = (y - base) * kLog2e, p = __builtin_amdgcn_exp2f(t);
        s += p;
        sx = fmaf(p, fmaxf(t, -1e4f), sx);  // p is 0 far below; the bound keeps 0 x inf out
        above += __popcll(__ballot(y > xt));
      }
  }
  const float wm = wave_max(m);
  if (lane == 0) {
    lds.m[wave] = wm;
    lds.floor[wave] = floor;
  }
  __syncthreads();
  const float m_raw = fmaxf(fmaxf(lds.m[0], lds.m[1]), fmaxf(lds.m[2], lds.m[3]));
  {
    const float by = m == -INFINITY ? 0.f : (m - m_raw) * kLog2e;
    const float f = __builtin_amdgcn_exp2f(by);
    sx = wave_sum((sx + (f == 0.f ? 0.f : s * by)) * f);
    s = wave_sum(s * f);
  }
  m = m_raw == -INFINITY ? 0.f : m_raw;
  if (lane == 0) {
    lds.s[wave] = s;
    lds.sx[wave] = sx;
    lds.above[wave] = above;
  }
  if (a.top) {
    const uint32_t f = max(max(lds.floor[0], lds.floor[1]), max(lds.floor[2], lds.floor[3]));
    auto each = [&](auto &&use) {
      for (int i = 0; i < a.batches * NV; ++i) {
        const uint4 w = load(begin + i * kStride);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const int at = begin + i * kStride + e;
          if (at >= 0 && at < a.n_vocab) use(key_of(Vec<T>::at(w, e), (uint32_t)at));
        }
      }
    };
    __syncthreads();
    const int listed = lds.count;
    for (int c = tid; c < min(listed, kScoreList); c += kScoreThreads)
      if ((uint32_t)(lds.list[c] >> 32) >= f) lds.pick[atomicAdd(&lds.picks, 1)] = (uint32_t)lds.list[c];
    __syncthreads();
    const int picks = lds.picks;
    for (int c = tid / kScoreBatch; c < picks; c += kScoreThreads / kScoreBatch) {
      const int who = lds.pick[c], i = tid % kScoreBatch;
      const int at = (chunk * a.batches + who / kScoreThreads) * (NV * kStride) - skew + who % kScoreThreads * VE +
                     i / VE * kStride + i % VE;
      if (at >= 0 && at < a.n_vocab) {
        const u64 key = key_of(Vec<T>::one(x + at), (uint32_t)at);
        if ((uint32_t)(key >> 32) >= f) put(lds.kept, &lds.kept_count, key);
      }
    }
    __syncthreads();
    const bool all = listed > kScoreList || lds.kept_count > kScoreList;
    __syncthreads();  // everybody has read the count before it may be cleared
    rank_top(a.top, f, all, each, lds);
  } else {
    __syncthreads();
  }
  s = (lds.s[0] + lds.s[1]) + (lds.s[2] + lds.s[3]);
  sx = (lds.sx[0] + lds.sx[1]) + (lds.sx[2] + lds.sx[3]);
  above = (lds.above[0] + lds.above[1]) + (lds.above[2] + lds.above[3]);
  if (a.chunks == 1) {
    finish(a, row, id, xt, m, s, sx, above, lds);
    return;
  }

  // the chunk's record: {m, s, sx, above}, then the keys
  const size_t rec = score_record_bytes(a.top);
  char *base = (char *)a.part + (size_t)row * a.chunks * rec;
  const __amdgpu_buffer_rsrc_t mine = coherent_rsrc(base + chunk * rec, (uint32_t)rec);
  if (tid == 0) st16_coherent(mine, 0, 0, f32x4{m_raw, s, sx, __int_as_float(above)});
  if (2 * tid < a.top) {
    const u64 k0 = lds.top[2 * tid], k1 = 2 * tid + 1 < a.top ? lds.top[2 * tid + 1] : 0;
    st16_coherent(mine, 16 + 16 * tid, 0, f32x4{__uint_as_float((uint32_t)k0), __uint_as_float((uint32_t)(k0 >> 32)),
                                                __uint_as_float((uint32_t)k1), __uint_as_float((uint32_t)(k1 >> 32))});
  }
  wait_vmcnt<0>();
  asm volatile("" ::: "memory");
  __syncthreads();
  if (tid == 0) {
    const unsigned got = __hip_atomic_fetch_add(a.cnt + row, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (got == (unsigned)a.chunks - 1) __hip_atomic_store(a.cnt + row, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    lds.arrived = got;
  }
  __syncthreads();
  if (lds.arrived != (unsigned)a.chunks - 1) return;

  // join, a chunk's numbers on each of the first threads
  static_assert(kScoreMaxChunks <= kScoreThreads, "a thread for every chunk");
  f32x4 r = {-INFINITY, 0.f, 0.f, 0.f};
  const __amdgpu_buffer_rsrc_t all = coherent_rsrc(base, (uint32_t)(rec * a.chunks));
  if (tid < a.chunks) r = ld16_coherent(all, (uint32_t)(tid * rec), 0);
  // pairs of keys: pair p of chunk c on thread c pairs + p, `rounds` of them
  const int pairs = (a.top + 1) / 2;
  constexpr int kRounds = kScoreMaxChunks * (kScoreMaxTop / 2) / kScoreThreads;
  static_assert(kRounds * kScoreThreads == kScoreMaxChunks * (kScoreMaxTop / 2), "every pair has its place");
  u64 keys[2 * kRounds];
  uint32_t best = 0;
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int at = tid + i * kScoreThreads;
    keys[2 * i] = keys[2 * i + 1] = 0;
    if (at < a.chunks * pairs) {
      const int c = at / pairs, p = at - c * pairs;
      const f32x4 w = ld16_coherent(all, (uint32_t)(c * rec + 16 + 16 * p), 0);
      keys[2 * i] = (u64)__float_as_uint(w[1]) << 32 | __float_as_uint(w[0]);
      keys[2 * i + 1] = (u64)__float_as_uint(w[3]) << 32 | __float_as_uint(w[2]);
      best = max(best, __float_as_uint(w[1]));  // a record's keys come in order: the pair's first is the larger
    }
  }
  const float wmx = wave_max(r[0]);
  if (lane == 0) lds.m[wave] = wmx;
  if (a.top) {
    const uint32_t f = kth_floor(best, a.top);
    if (lane == 0) lds.floor[wave] = f;
  }
  if (tid == 0) lds.kept_count = 0;
  __syncthreads();
  const float M_raw = fmaxf(fmaxf(lds.m[0], lds.m[1]), fmaxf(lds.m[2], lds.m[3]));
  const float M = M_raw == -INFINITY ? 0.f : M_raw;
  // a chunk's terms move to the common maximum: t + (its m - M) log2(e)
  const float by = r[0] == -INFINITY ? 0.f : (r[0] - M) * kLog2e;
  const float f2 = r[0] == -INFINITY && r[1] == 0.f ? 0.f : __builtin_amdgcn_exp2f(by);
  s = wave_sum(r[1] * f2);
  sx = wave_sum((r[2] + (f2 == 0.f ? 0.f : r[1] * by)) * f2);
  above = wave_reduce(__float_as_int(r[3]), 0, [](int a, int b) { return a + b; });
  __syncthreads();
  if (lane == 0) {
    lds.s[wave] = s;
    lds.sx[wave] = sx;
    lds.above[wave] = above;
  }
  if (a.top) {
    const uint32_t f = max(max(lds.floor[0], lds.floor[1]), max(lds.floor[2], lds.floor[3]));
    auto each = [&](auto &&use) {
#pragma unroll
      for (int i = 0; i < 2 * kRounds; ++i)
        if (keys[i]) use(keys[i]);
    };
    if (best >= f)
      each([&](u64 key) {
        if ((uint32_t)(key >> 32) >= f) put(lds.kept, &lds.kept_count, key);
      });
    __syncthreads();
    rank_top(a.top, f, false, each, lds);
  } else {
    __syncthreads();
  }
  s = (lds.s[0] + lds.s[1]) + (lds.s[2] + lds.s[3]);
  sx = (lds.sx[0] + lds.sx[1]) + (lds.sx[2] + lds.sx[3]);
  above = (lds.above[0] + lds.above[1]) + (lds.above[2] + lds.above[3]);
  finish(a, row, id, xt, M, s, sx, above, lds);
}

// ---------------------------------------------------------------- launcher
// Workgroups of a row, and the batches each takes: one where the rows alone
// make two workgroups a CU, otherwise as many as make that, down to a batch
// each.  Four a CU fit and do not pay, as each has a selection and a share of
// the join: 64 rows of 128256 13.8 us for 16.2 with four, 700 of 32000 15.9
// for 24.3, 1000 of 128256 52.7 for 60.2, 36 of 131071 17.4 for 18.1; the
// other way round 200 of 128256 27.7 for 26.9 and 600 43.8 for 42.0.
ScoreSplit score_split(int n, int n_vocab, int dtype) {
  const int ve = dtype == 0 ? 4 : 8, batch = kScoreThreads * kScoreBatch;
  const int all = (n_vocab + ve - 1 + batch - 1) / batch;  // a row may begin up to ve - 1 elements into its first vector
  // a vocabulary of 2^20 whose rows may begin inside a vector has one batch more than the join takes chunks
  const int want = std::min({all, (512 + n - 1) / n, kScoreMaxChunks});
  ScoreSplit r;
  r.batches = (all + want - 1) / want;
  r.chunks = (all + r.batches - 1) / r.batches;
  return r;
}

hipError_t launch_score(const ScoreArgs &a, int dtype, hipStream_t st) {
  const dim3 grid(a.n * a.chunks), block(kScoreThreads);
  if (dtype == 0) hipLaunchKernelGGL((score_kernel<float>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((score_kernel<u16>), grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace lora
