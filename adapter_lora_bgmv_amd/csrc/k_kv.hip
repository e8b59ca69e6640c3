// k_kv.hip -- the 8-bit paged KV cache: rows quantised into pages, and pages read back to rows.
//
// A page's head holds P x D e4m3 codes of K, as many of V, and one exponent
// byte e for each: a code c stands for c 2^(e - 127).  For the largest finite
// |x| among a page's values the scale is the smallest power of two s with
// |x| <= 448 s, so codes never overflow; being a power of two, it divides
// without rounding, and moving old codes to a larger scale is exact while
// they stay normal.  One workgroup owns one (page, head) of K or of V for the
// call, so that nothing is shared between workgroups and no atomics are used:
// load the page's new rows once, reduce the largest magnitude, then convert
// from registers and store.
//
// The order of codes is the order in which the attention reads them
// (k_attend.hip).  K: [P/16][4][D/16][4][16] = (16-token group, quad, 16-dim
// chunk, token of the quad, dim): 16 bytes of one token side by side with the
// same chunk of its three neighbours.  V: [P/16][D][16] = (group, dim,
// token): a dim's 16 tokens side by side.
//
// Both kernels move bytes only, so HBM bounds large calls (4 x 4096 tokens of
// 8 heads x 128 back to bf16 rows: 24 us, 4.3 TB/s, two thirds of it writes)
// and latency small ones (64 rows joining their pages: 5.7 us, four dependent
// round trips).  A K item is one token's 16 dims: 32 bytes of bf16 row, 16 bytes of
// code.  A V item is four tokens by four dims, transposed in registers by
// byte permutes (the two layouts differ by exactly that transpose), the
// quad's index fastest over the lanes so that four lanes store 16 bytes side
// by side.
#include "common.hpp"
#include "verify.hpp"

namespace lora {

constexpr int kKvThreads = 256;
constexpr int kExpMin = 10, kExpMax = 247;  // 2^-117 .. 2^120

// The pages that a sequence's rows touch: logical pages [p0, p0 + count).
__device__ __forceinline__ int touched(const KvDev &a, const SeqDev &s, int *p0) {
  const int first = max(s.start, 0), last = min(s.len, kv_cap(a)) - 1;
  *p0 = first >> a.page_shift;
  return s.rows > 0 && last >= first ? (last >> a.page_shift) - *p0 + 1 : 0;
}

// Work item u of the call's touched pages: its sequence and logical page, or
// false past the last.  Every wave finds it by itself: lane l counts the
// pages of `per` sequences, one scan over the lanes, and the lane whose share
// holds u walks it.
__device__ __forceinline__ bool find_page(const KvDev &a, int u, int lane, SeqDev *s, int *seq, int *page) {
  const int per = (a.n_seqs + 63) >> 6, i0 = lane * per, i1 = min(i0 + per, a.n_seqs);
  SeqDev its = {0, 0, 0, 0};  // the lane's first sequence, later the one that holds u
  if (i0 < i1) its = load_seq(a, i0);
  int p0, sum = i0 < i1 ? touched(a, its, &p0) : 0;
  for (int i = i0 + 1; i < i1; ++i) sum += touched(a, load_seq(a, i), &p0);
  const int incl = wave_incl_scan(sum);
  int found = -1, where = 0;
  if (u < incl && u >= incl - sum) {
    int at = incl - sum;
    for (int i = i0; i < i1; ++i) {
      if (i > i0) its = load_seq(a, i);
      const int c = touched(a, its, &p0);
      if (u < at + c) {
        found = i;
        where = p0 + u - at;
        break;
      }
      at += c;
    }
  }
  const unsigned long long who = __ballot(found >= 0);
  if (!who) return false;
  const int src = __ffsll(who) - 1;
  *seq = __builtin_amdgcn_readlane(found, src);
  *page = __builtin_amdgcn_readlane(where, src);
  *s = seq_of_lane(its, src);
  return true;
}

// 4 x 4 bytes: w[i] holds row i's columns 0..3; on return w[c] holds column c's rows 0..3.
__device__ __forceinline__ void transpose4(uint32_t w[4]) {
  const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400);  // r0c0 r1c0 r0c1 r1c1
  const uint32_t b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602);  // r0c2 r1c2 r0c3 r1c3
  const uint32_t c = __builtin_amdgcn_perm(w[3], w[2], 0x05010400);
  const uint32_t d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602);
  w[0] = __builtin_amdgcn_perm(c, a, 0x05040100);
  w[1] = __builtin_amdgcn_perm(c, a, 0x07060302);
  w[2] = __builtin_amdgcn_perm(d, b, 0x05040100);
  w[3] = __builtin_amdgcn_perm(d, b, 0x07060302);
}

// Four values of a row as f32, from registers.
template <typename T>
struct Raw4;
template <>
struct Raw4<float> {
  uint4 r;
  __device__ void load(const float *p) { r = ldg16(p); }
  __device__ void zero() { r = z4(); }
  __device__ float at(int i) const { return __uint_as_float(i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w); }
};
template <>
struct Raw4<u16> {
  uint2 r;
  __device__ void load(const u16 *p) {
    typedef unsigned u32x2n __attribute__((ext_vector_type(2)));
    const u32x2n v = *(const __attribute__((address_space(1))) u32x2n *)(uintptr_t)p;
    r = make_uint2(v.x, v.y);
  }
  __device__ void zero() { r = make_uint2(0u, 0u); }
  __device__ float at(int i) const {
    const uint32_t w = i < 2 ? r.x : r.y;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
};

// |x|'s bits where x is finite, 0 elsewhere: unsigned order is magnitude order.
__device__ __forceinline__ uint32_t finite_bits(float x) {
  const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}

// The exponent byte for a largest magnitude m 2^(E - 127), 1 <= m < 2: 448 is
// 1.75 2^8, so 2^(E - 135) does where m <= 1.75 and twice that elsewhere.
__device__ __forceinline__ int exp_for(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u);
  return min(max(e, kExpMin), kExpMax);
}

// Four scaled values as codes; infinities and NaN become NaN, so that they
// show in what reads them.  The conversion rounds to nearest, ties to even,
// and nothing exceeds 448.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float inv) {
  const float qnan = __uint_as_float(0x7fc00000u);
  a = finite_bits(a) || a == 0.f ? a * inv : qnan;
  b = finite_bits(b) || b == 0.f ? b * inv : qnan;
  c = finite_bits(c) || c == 0.f ? c * inv : qnan;
  d = finite_bits(d) || d == 0.f ? d * inv : qnan;
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// Four codes moved by a power of two: exact while normal, rounded to nearest even below.
__device__ __forceinline__ uint32_t moved4(uint32_t w, int by) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(ldexpf(a[0], by), ldexpf(a[1], by), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(ldexpf(b[0], by), ldexpf(b[1], by), r, true);
}

// Bytes of a quad's dword whose token is in [lo, hi), for the quad that begins at t0.
__device__ __forceinline__ uint32_t byte_mask(int t0, int lo, int hi) {
  const int a = min(max(lo - t0, 0), 4), b = min(max(hi - t0, 0), 4);
  return b > a ? (uint32_t)((1ull << (8 * b)) - (1ull << (8 * a))) : 0u;
}

__device__ __forceinline__ void st4(uint32_t *p, uint32_t v) { *p = v; }

// ---------------------------------------------------------------- write
// Grid: touched pages x heads x {K, V}.  IT items of 16 values per thread
// cover the page (P D = 16 IT 256 at most).
template <typename T, int D, int IT>
__global__ __launch_bounds__(kKvThreads) void kv_write_kernel(KvDev a, const T *krows, int k_stride, const T *vrows,
                                                              int v_stride) {
  __shared__ uint32_t wave_max[kKvThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63;
  SeqDev s;
  int seq, lp;
  if (!find_page(a, blockIdx.x, lane, &s, &seq, &lp)) return;
  const int page = page_of(a, seq, lp);
  if (page < 0) return;
  const int h = blockIdx.y, P = 1 << a.page_shift, t_page = lp << a.page_shift;
  const bool is_v = blockIdx.z != 0;
  // new tokens of the page [t0, t1), and the first's row
  const int t0 = max(s.start - t_page, 0), t1 = min(s.len - t_page, P);
  const long long row0 = (long long)s.row0 + (t_page - s.start);  // row of the page's token 0, were it new
  uint8_t *codes = (is_v ? a.v : a.k) + ((size_t)page * a.H + h) * ((size_t)P * D);
  uint8_t *ep = (is_v ? a.ve : a.ke) + (size_t)page * a.H + h;
  const int before = t0 > 0 ? *ep : 0;
  const T *src = (is_v ? vrows : krows) + (size_t)h * D;
  const int stride = is_v ? v_stride : k_stride;
  const int items = P * D / 16;

  Raw4<T> x[IT][4];
  uint32_t big = 0;
#pragma unroll
  for (int j = 0; j < IT; ++j) {
    const int it = tid + j * kKvThreads;
    if (!is_v) {
      const int t = it / (D / 16), c = it % (D / 16);
      const bool live = it < items && t >= t0 && t < t1;
      const T *p = src + (size_t)(live ? row0 + t : 0) * stride + c * 16;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (live) x[j][i].load(p + 4 * i);
        else x[j][i].zero();
      }
    } else {
      const int q = (it & 3) + 4 * (it / D), db = (it >> 2) % (D / 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 4 * q + i;
        const bool live = it < items && t >= t0 && t < t1;
        if (live) x[j][i].load(src + (size_t)(row0 + t) * stride + db * 4);
        else x[j][i].zero();
      }
    }
  }
#pragma unroll
  for (int j = 0; j < IT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) big = max(big, finite_bits(x[j][i].at(e)));
  big = (uint32_t)wave_reduce((int)big, 0, [](int a, int b) { return max(a, b); });  // bits of finite numbers: no sign
  if (lane == 0) wave_max[tid >> 6] = big;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kKvThreads / 64; ++w) big = max(big, wave_max[w]);
  const int need = exp_for(big);
  const int e = min(max(before, need), kExpMax);
  const int by = before - e;  // old tokens move by 2^by
  const bool move = t0 > 0 && by != 0;
  const float inv = __uint_as_float((uint32_t)(254 - e) << 23);
  if (tid == 0) *ep = (uint8_t)e;

#pragma unroll
  for (int j = 0; j < IT; ++j) {
    const int it = tid + j * kKvThreads;
    if (it >= items) continue;
    if (!is_v) {
      const int t = it / (D / 16), c = it % (D / 16);
      uint4 *p = (uint4 *)(codes + (t >> 4) * (16 * D) + ((t >> 2) & 3) * (4 * D) + c * 64 + (t & 3) * 16);
      if (t >= t0 && t < t1) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = codes4(x[j][i].at(0), x[j][i].at(1), x[j][i].at(2), x[j][i].at(3), inv);
        *p = make_uint4(w[0], w[1], w[2], w[3]);
      } else if (move && t < t0) {
        const uint4 o = *p;
        *p = make_uint4(moved4(o.x, by), moved4(o.y, by), moved4(o.z, by), moved4(o.w, by));
      }
    } else {
      const int q = (it & 3) + 4 * (it / D), db = (it >> 2) % (D / 4);
      const uint32_t fresh = byte_mask(4 * q, t0, t1), old = move ? byte_mask(4 * q, 0, t0) : 0u;
      if (!(fresh | old)) continue;
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = codes4(x[j][i].at(0), x[j][i].at(1), x[j][i].at(2), x[j][i].at(3), inv);
      transpose4(w);
      uint32_t *p = (uint32_t *)(codes + (q >> 2) * (16 * D) + db * 64 + (q & 3) * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (fresh != 0xffffffffu) {
          const uint32_t o = p[4 * i];
          w[i] = (w[i] & fresh) | (moved4(o, by) & old) | (o & ~(fresh | old));
        }
        st4(p + 4 * i, w[i]);
      }
    }
  }
}

// ---------------------------------------------------------------- read
template <typename T>
__device__ __forceinline__ void store_row4(T *p, uint32_t codes, float scale);
template <>
__device__ __forceinline__ void store_row4<u16>(u16 *p, uint32_t w, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true);
  *(uint2 *)p = make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
}
template <>
__device__ __forceinline__ void store_row4<float>(float *p, uint32_t w, float scale) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  *(float4 *)p = make_float4(a[0] * scale, a[1] * scale, b[0] * scale, b[1] * scale);
}

// Sixteen values of a row, 16 bytes at a time.
template <typename T>
__device__ __forceinline__ void store_row16(T *p, const uint32_t w[4], float scale) {
  if constexpr (sizeof(T) == 2) {
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = __builtin_bit_cast(uint32_t, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], scale, false));
      o[2 * i + 1] = __builtin_bit_cast(uint32_t, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], scale, true));
    }
    ((uint4 *)p)[0] = make_uint4(o[0], o[1], o[2], o[3]);
    ((uint4 *)p)[1] = make_uint4(o[4], o[5], o[6], o[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) store_row4<T>(p + 4 * i, w[i], scale);
  }
}

// Grid as in the write, but the heads of a page come one after the other, so
// that the parts of a row are stored close together in time (4 x 4096 tokens,
// 8 heads x 128: 25.1 -> 23.6 us, f32 47.8 -> 44.2); a call's rows are few
// enough for pages to be a grid's second dimension.  Every product is exact:
// e4m3 times a power of two in the range of the exponent bytes is a bf16
// number, but for 256 2^120 and above, which become infinities.
template <typename T, int D, int IT>
__global__ __launch_bounds__(kKvThreads) void kv_read_kernel(KvDev a, T *krows, int k_stride, T *vrows, int v_stride) {
  const int tid = threadIdx.x, lane = tid & 63;
  SeqDev s;
  int seq, lp;
  if (!find_page(a, blockIdx.y, lane, &s, &seq, &lp)) return;
  const int page = page_of(a, seq, lp);
  if (page < 0) return;
  const int h = blockIdx.x, P = 1 << a.page_shift, t_page = lp << a.page_shift;
  const bool is_v = blockIdx.z != 0;
  const int t0 = max(s.start - t_page, 0), t1 = min(s.len - t_page, P);
  const long long row0 = (long long)s.row0 + (t_page - s.start);
  const uint8_t *codes = (is_v ? a.v : a.k) + ((size_t)page * a.H + h) * ((size_t)P * D);
  const float scale = __uint_as_float((uint32_t)(is_v ? a.ve : a.ke)[(size_t)page * a.H + h] << 23);
  T *dst = (is_v ? vrows : krows) + (size_t)h * D;
  const int stride = is_v ? v_stride : k_stride;
  const int items = P * D / 16;
  uint4 w[IT];
#pragma unroll
  for (int j = 0; j < IT; ++j) {
    const int it = tid + j * kKvThreads;
    if (it >= items) continue;
    if (!is_v) {
      const int t = it / (D / 16), c = it % (D / 16);
      w[j] = ldg16(codes + (t >> 4) * (16 * D) + ((t >> 2) & 3) * (4 * D) + c * 64 + (t & 3) * 16);
    } else {
      const int q = (it & 3) + 4 * (it / D), db = (it >> 2) % (D / 4);
      const uint32_t *p = (const uint32_t *)(codes + (q >> 2) * (16 * D) + db * 64 + (q & 3) * 4);
      w[j] = make_uint4(p[0], p[4], p[8], p[12]);
    }
  }
#pragma unroll
  for (int j = 0; j < IT; ++j) {
    const int it = tid + j * kKvThreads;
    if (it >= items) continue;
    uint32_t r[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
    if (!is_v) {
      const int t = it / (D / 16), c = it % (D / 16);
      if (t < t0 || t >= t1) continue;
      store_row16<T>(dst + (size_t)(row0 + t) * stride + c * 16, r, scale);
    } else {
      const int q = (it & 3) + 4 * (it / D), db = (it >> 2) % (D / 4);
      transpose4(r);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 4 * q + i;
        if (t >= t0 && t < t1) store_row4<T>(dst + (size_t)(row0 + t) * stride + db * 4, r[i], scale);
      }
    }
  }
}

// ---------------------------------------------------------------- launchers
// Items per thread that cover a page: the smallest built count.
template <template <typename, int, int> class K, typename T, int D, typename... A>
static void launch_by_items(const KvDev &kv, hipStream_t st, A... args) {
  const int items = (D << kv.page_shift) / 16;
  const dim3 grid(kv_max_touched(kv.n, kv.n_seqs, 1 << kv.page_shift), kv.H, 2);
  if (items <= kKvThreads) K<T, D, 1>::go(grid, st, kv, args...);
  else if (items <= 2 * kKvThreads) K<T, D, 2>::go(grid, st, kv, args...);
  else if (items <= 4 * kKvThreads) K<T, D, 4>::go(grid, st, kv, args...);
  else K<T, D, 8>::go(grid, st, kv, args...);
}
template <typename T, int D, int IT>
struct WriteK {
  static void go(dim3 grid, hipStream_t st, const KvDev &kv, const void *k, int ks, const void *v, int vs) {
    if constexpr (IT * kKvThreads * 16 <= D * 128)
      hipLaunchKernelGGL((kv_write_kernel<T, D, IT>), grid, dim3(kKvThreads), 0, st, kv, (const T *)k, ks, (const T *)v, vs);
  }
};
template <typename T, int D, int IT>
struct ReadK {
  static void go(dim3 grid, hipStream_t st, const KvDev &kv, void *k, int ks, void *v, int vs) {
    if constexpr (IT * kKvThreads * 16 <= D * 128)
      hipLaunchKernelGGL((kv_read_kernel<T, D, IT>), dim3(grid.y, grid.x, 2), dim3(kKvThreads), 0, st, kv, (T *)k, ks, (T *)v, vs);
  }
};
template <template <typename, int, int> class K, typename... A>
static hipError_t launch_by_type(const KvDev &kv, int dim, int dtype, hipStream_t st, A... args) {
  if (dtype == 0) {
    if (dim == 64) launch_by_items<K, float, 64>(kv, st, args...);
    else if (dim == 128) launch_by_items<K, float, 128>(kv, st, args...);
    else launch_by_items<K, float, 256>(kv, st, args...);
  } else {
    if (dim == 64) launch_by_items<K, u16, 64>(kv, st, args...);
    else if (dim == 128) launch_by_items<K, u16, 128>(kv, st, args...);
    else launch_by_items<K, u16, 256>(kv, st, args...);
  }
  return hipGetLastError();
}

hipError_t launch_kv_write(const KvDev &kv, int dim, int dtype, const void *k, int k_stride, const void *v, int v_stride,
                           hipStream_t st) {
  return launch_by_type<WriteK>(kv, dim, dtype, st, k, k_stride, v, v_stride);
}
hipError_t launch_kv_read(const KvDev &kv, int dim, int dtype, void *k, int k_stride, void *v, int v_stride,
                          hipStream_t st) {
  return launch_by_type<ReadK>(kv, dim, dtype, st, k, k_stride, v, v_stride);
}

}  // namespace lora
