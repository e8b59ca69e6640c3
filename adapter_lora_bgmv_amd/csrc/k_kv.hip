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
//
// With the rotation (lora_kv_write_rotary) keys turn between their load and the
// maximum, pairs within a thread's registers or a neighbour's, and queries in
// workgroups of their own behind those of the pages.  Angles are f64 products
// of position and frequency, brought to an eighth of the circle, cosine and
// sine series: in 64 bits for keys, whose f32 results decide codes, in f32 for
// queries, and once for all heads that a workgroup turns.  Latency bounds
// small calls as it does the plain write's (8.0 us for 64 rows) and, with HBM,
// large ones (8 x 512 rows of 32 + 2 x 8 heads x 128: 23 to 26 us, 3.5 to 4.1
// TB/s, each byte moved once): 165 registers leave 1.6 waves a SIMD on
// average, which wait 62 % of their time, and vector instructions take 29 %.
#include <algorithm>
#include <climits>

#include "common.hpp"
#include "e4m3.hpp"
#include "verify.hpp"

namespace lora {

constexpr int kKvThreads = 256;

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
// One (page, head) of K or of V.  IT items of 16 values per thread cover the
// page (P D = 16 IT 256 at most).
template <typename T, int D, int IT>
__device__ __forceinline__ void write_page(const KvDev &a, int u, int h, bool is_v, const T *krows, int k_stride, const T *vrows,
                                           int v_stride, uint32_t *wave_max) {
  const int tid = threadIdx.x, lane = tid & 63;
  SeqDev s;
  int seq, lp;
  if (!find_page(a, u, lane, &s, &seq, &lp)) return;
  const int page = page_of(a, seq, lp);
  if (page < 0) return;
  const int P = 1 << a.page_shift, t_page = lp << a.page_shift;
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
      for (int e = 0; e < 4; ++e) big = max(big, __float_as_uint(x[j][i].at(e)) & 0x7fffffffu);
  if (__any(big >= 0x7f800000u)) {  // infinities and NaN do not count
    big = 0;
#pragma unroll
    for (int j = 0; j < IT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) big = max(big, finite_bits(x[j][i].at(e)));
  }
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

// Grid: touched pages x heads x {K, V}.
template <typename T, int D, int IT>
__global__ __launch_bounds__(kKvThreads) void kv_write_kernel(KvDev a, const T *krows, int k_stride, const T *vrows,
                                                              int v_stride) {
  __shared__ uint32_t wave_max[kKvThreads / 64];
  write_page<T, D, IT>(a, blockIdx.x, blockIdx.y, blockIdx.z != 0, krows, k_stride, vrows, v_stride, wave_max);
}

// ---------------------------------------------------------------- write with rotation
// Pair i of a head's first `rot` dims turns by the angle p inv_freq[i] of its
// token's position p:
//     (x, y) -> (x cos - y sin, y cos + x sin).
// An item is eight pairs of one token, 16 dims: pairs (i, i + rot/2) take
// eight dims of either half, interleaved ones (2i, 2i + 1) and dims past
// `rot` sixteen side by side.
//
// The angle of a far position loses digits in 32 bits (p = 131071 at frequency
// 1: 0.008 of a turn's 2 pi in steps), so it is formed and reduced in 64.
// Keys are turned in 64 bits as well and rounded once to f32, so that the
// scale of a page and the codes next to a rounding border follow from the
// numbers and not from the order of operations.  64-bit arithmetic runs at
// the f32 rate here, but it and its registers are what large calls have beside
// memory: fewer cosines took 31.2 us to 23.3 (write_turned_page).
// Queries are turned in 32 bits from the same cosines.
template <typename T>
struct Raw8 {
  static constexpr int NV = sizeof(T) / 2;
  uint4 r[NV];
  __device__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < NV; ++i) r[i] = ldg16((const char *)p + 16 * i);
  }
  __device__ float at(int i) const {
    if constexpr (sizeof(T) == 4) {
      const uint4 v = r[i / 4];
      return __uint_as_float(i % 4 == 0 ? v.x : i % 4 == 1 ? v.y : i % 4 == 2 ? v.z : v.w);
    } else {
      const uint4 v = r[0];
      const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
      return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
    }
  }
};

// An angle's quarter turns k (their two low bits) and what is left, within
// pi/4: pi/2 in two parts loses nothing below 2^50, from where an angle in 64
// bits is no longer known to a quarter of a radian; such angles count as 0,
// and infinities and NaN as NaN.
__device__ __forceinline__ double off_quarters(double a, int *k) {
  a = fabs(a) < 1125899906842624.0 ? a : a * 0.0;
  const double z = fma(a, 0.63661977236758134308, 6755399441055744.0);  // + 1.5 2^52: a whole number in the low bits
  const double n = z - 6755399441055744.0;
  *k = (int)(uint32_t)__double_as_longlong(z);
  return fma(-n, 6.12323399573676603587e-17, fma(-n, 1.57079632679489655800, a));
}
// cos and sin by Taylor's series, to 1e-16.
__device__ __forceinline__ void cos_sin(double a, double *c, double *s) {
  int k;
  const double r = off_quarters(a, &k), q = r * r;
  double sp = -1.0 / 1307674368000.0, cp = 1.0 / 20922789888000.0;
  sp = fma(sp, q, 1.0 / 6227020800.0);
  cp = fma(cp, q, -1.0 / 87178291200.0);
  sp = fma(sp, q, -1.0 / 39916800.0);
  cp = fma(cp, q, 1.0 / 479001600.0);
  sp = fma(sp, q, 1.0 / 362880.0);
  cp = fma(cp, q, -1.0 / 3628800.0);
  sp = fma(sp, q, -1.0 / 5040.0);
  cp = fma(cp, q, 1.0 / 40320.0);
  sp = fma(sp, q, 1.0 / 120.0);
  cp = fma(cp, q, -1.0 / 720.0);
  sp = fma(sp, q, -1.0 / 6.0);
  cp = fma(cp, q, 1.0 / 24.0);
  cp = fma(cp, q, -0.5);
  sp = fma(sp * q, r, r);
  cp = fma(cp, q, 1.0);
  const double x = k & 1 ? sp : cp, y = k & 1 ? cp : sp;
  *c = (k + 1) & 2 ? -x : x;
  *s = k & 2 ? -y : y;
}
// The same to f32's last bits: the series run in 32.
__device__ __forceinline__ void cos_sin(double a, float *c, float *s) {
  int k;
  const float r = (float)off_quarters(a, &k), q = r * r;
  float sp = 1.f / 362880.f, cp = -1.f / 3628800.f;
  cp = fmaf(cp, q, 1.f / 40320.f);
  sp = fmaf(sp, q, -1.f / 5040.f);
  cp = fmaf(cp, q, -1.f / 720.f);
  sp = fmaf(sp, q, 1.f / 120.f);
  cp = fmaf(cp, q, 1.f / 24.f);
  sp = fmaf(sp, q, -1.f / 6.f);
  cp = fmaf(cp, q, -0.5f);
  sp = fmaf(sp * q, r, r);
  cp = fmaf(cp, q, 1.f);
  const float x = k & 1 ? sp : cp, y = k & 1 ? cp : sp;
  *c = (k + 1) & 2 ? -x : x;
  *s = k & 2 ? -y : y;
}

// The dims of item c of a head: eight at d0, eight at d1; whether they turn.
__device__ __forceinline__ bool item_dims(const RotaryDev &rot, int c, int *d0, int *d1) {
  const bool turns = c < rot.rot / 16;
  const bool split = turns && !rot.interleaved;
  *d0 = split ? 8 * c : 16 * c;
  *d1 = split ? rot.rot / 2 + 8 * c : 16 * c + 8;
  return turns;
}

// K of `heads` heads of a page from h on, whose cosines are formed once: they
// are most of the arithmetic (4096 rows of 8 heads, 32 query heads: 31.2 us
// with those of each head anew, 23.3 with two heads to a workgroup of K and eight to one of queries).
template <typename T, int D, int IT, int HB>
__device__ __forceinline__ void write_turned_page(const KvDev &a, const RotaryDev &rot, int u, int h0, const T *krows, int k_stride,
                                                  uint32_t *wave_max) {
  const int tid = threadIdx.x, lane = tid & 63;
  SeqDev s;
  int seq, lp;
  if (!find_page(a, u, lane, &s, &seq, &lp)) return;
  const int page = page_of(a, seq, lp);
  if (page < 0) return;
  const int P = 1 << a.page_shift, t_page = lp << a.page_shift;
  const int t0 = max(s.start - t_page, 0), t1 = min(s.len - t_page, P);
  const long long row0 = (long long)s.row0 + (t_page - s.start);  // row of the page's token 0, were it new
  const int items = P * D / 16;
  // 256 is a multiple of a token's D / 16 items: a thread has the same dims of every token
  static_assert(kKvThreads % (D / 16) == 0, "a thread's items share their dims");
  const int c = tid % (D / 16);
  int d0, d1;
  const bool turns = item_dims(rot, c, &d0, &d1);
  auto token = [&](int j) { return (tid + j * kKvThreads) / (D / 16); };
  auto live = [&](int j) { return tid + j * kKvThreads < items && token(j) >= t0 && token(j) < t1; };

  Raw8<T> raw[IT][2];
  auto fetch = [&](int h) {
#pragma unroll
    for (int j = 0; j < IT; ++j)
      if (live(j)) {
        const T *p = krows + (size_t)h * D + (size_t)(row0 + token(j)) * k_stride;
        raw[j][0].load(p + d0);
        raw[j][1].load(p + d1);
      }
  };
  fetch(h0);
  double cs[IT][8], sn[IT][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double f = turns ? (double)rot.inv_freq[8 * c + i] : 0.0;
#pragma unroll
    for (int j = 0; j < IT; ++j) cos_sin((double)(t_page + token(j)) * f, &cs[j][i], &sn[j][i]);
  }
#pragma unroll 1
  for (int h = h0; h < min(h0 + HB, a.H); ++h) {
    uint8_t *codes = a.k + ((size_t)page * a.H + h) * ((size_t)P * D);
    uint8_t *ep = a.ke + (size_t)page * a.H + h;
    const int before = t0 > 0 ? *ep : 0;
    float x[IT][16];
    uint32_t big = 0;
#pragma unroll
    for (int j = 0; j < IT; ++j) {
      const bool on = live(j);
#pragma unroll
      for (int e = 0; e < 16; ++e) x[j][e] = on ? raw[j][e / 8].at(e % 8) : 0.f;
      if (on && turns) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const double cc = cs[j][i], ss = sn[j][i];
          if (rot.interleaved) {
            const double v = x[j][2 * i], w = x[j][2 * i + 1];
            x[j][2 * i] = (float)(v * cc - w * ss);
            x[j][2 * i + 1] = (float)(w * cc + v * ss);
          } else {
            const double v = x[j][i], w = x[j][i + 8];
            x[j][i] = (float)(v * cc - w * ss);
            x[j][i + 8] = (float)(w * cc + v * ss);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) big = max(big, __float_as_uint(x[j][e]) & 0x7fffffffu);
    }
    if (__any(big >= 0x7f800000u)) {  // infinities and NaN do not count
      big = 0;
#pragma unroll
      for (int j = 0; j < IT; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) big = max(big, finite_bits(x[j][e]));
    }
    if (HB > 1 && h + 1 < min(h0 + HB, a.H)) fetch(h + 1);
    big = (uint32_t)wave_reduce((int)big, 0, [](int a, int b) { return max(a, b); });  // bits of finite numbers: no sign
    if (HB > 1 && h > h0) __syncthreads();  // the head before has been read
    if (lane == 0) wave_max[tid >> 6] = big;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kKvThreads / 64; ++w) big = max(big, wave_max[w]);
    const int e = min(max(before, exp_for(big)), kExpMax);
    const int by = before - e;  // old tokens move by 2^by
    const bool move = t0 > 0 && by != 0;
    const float inv = __uint_as_float((uint32_t)(254 - e) << 23);
    if (tid == 0) *ep = (uint8_t)e;
#pragma unroll
    for (int j = 0; j < IT; ++j) {
      const int it = tid + j * kKvThreads, t = token(j);
      if (it >= items) continue;
      uint8_t *row = codes + (t >> 4) * (16 * D) + ((t >> 2) & 3) * (4 * D) + (t & 3) * 16;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int d = i ? d1 : d0;
        uint2 *p = (uint2 *)(row + d / 16 * 64 + d % 16);
        const float *y = x[j] + 8 * i;
        if (t >= t0 && t < t1) *p = make_uint2(codes4(y[0], y[1], y[2], y[3], inv), codes4(y[4], y[5], y[6], y[7], inv));
        else if (move && t < t0) *p = make_uint2(moved4(p->x, by), moved4(p->y, by));
      }
    }
  }
}

// Queries: a workgroup takes 256 / (D/16) rows and `per` heads of them; a
// thread has one row's item, its cosines in registers, and walks the heads.
template <typename T, int D>
__device__ __forceinline__ void turn_queries(const KvDev &a, const RotaryDev &rot, const TurnArgs &q, int block, int *pos) {
  constexpr int kRows = kKvThreads / (D / 16);
  const int tid = threadIdx.x;
  const int rb = block / q.groups, r0 = rb * kRows, h0 = (block - rb * q.groups) * q.per;
  if (tid < kRows) pos[tid] = INT_MIN;
  __syncthreads();
  // every sequence with rows among the workgroup's leaves their positions; a row of none has none
  for (int i = tid; i < a.n_seqs; i += kKvThreads) {
    if (a.indptr[i + 1] <= r0 || a.indptr[i] >= r0 + kRows) continue;
    const SeqDev s = load_seq(a, i);
    for (int r = max(s.row0, r0); r < min(s.row0 + s.rows, r0 + kRows); ++r) pos[r - r0] = s.start + (r - s.row0);
  }
  __syncthreads();
  const int c = tid % (D / 16), r = r0 + tid / (D / 16), p = pos[tid / (D / 16)];
  if (p == INT_MIN) return;
  int d0, d1;
  const bool turns = item_dims(rot, c, &d0, &d1);
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
    if (turns) cos_sin((double)p * (double)rot.inv_freq[8 * c + i], &cs[i], &sn[i]);
  }
  const T *src = (const T *)q.q + (size_t)r * q.q_stride;
  T *dst = (T *)q.out + (size_t)r * q.out_stride;
#pragma unroll 4
  for (int h = h0; h < min(h0 + q.per, q.heads); ++h) {
    Raw8<T> in[2];
    in[0].load(src + (size_t)h * D + d0);
    in[1].load(src + (size_t)h * D + d1);
    float x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = in[e / 8].at(e % 8);
    if (turns) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (rot.interleaved) {
          const float v = x[2 * i], w = x[2 * i + 1];
          x[2 * i] = fmaf(v, cs[i], -w * sn[i]);
          x[2 * i + 1] = fmaf(w, cs[i], v * sn[i]);
        } else {
          const float v = x[i], w = x[i + 8];
          x[i] = fmaf(v, cs[i], -w * sn[i]);
          x[i + 8] = fmaf(w, cs[i], v * sn[i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      T *to = dst + (size_t)h * D + (i ? d1 : d0);
      const float *y = x + 8 * i;
      if constexpr (sizeof(T) == 4) {
        ((float4 *)to)[0] = make_float4(y[0], y[1], y[2], y[3]);
        ((float4 *)to)[1] = make_float4(y[4], y[5], y[6], y[7]);
      } else {
        *(uint4 *)to = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
      }
    }
  }
}

// Workgroups: touched pages x (groups of HB heads for K, heads for V), then
// the queries'.  A dimension of a grid holds less than 2^32 threads, so they
// are laid out in rows of kGridRow.
constexpr int kGridRow = 1 << 20;
template <typename T, int D, int IT, int HB>
__global__ __launch_bounds__(kKvThreads) void kv_write_rotary_kernel(KvDev a, RotaryDev rot, TurnArgs q, const T *krows,
                                                                     int k_stride, const T *vrows, int v_stride) {
  __shared__ uint32_t wave_max[kKvThreads / 64];
  __shared__ int pos[64];
  const int b = blockIdx.y * kGridRow + blockIdx.x;
  if (b >= q.first) {
    if (b < q.blocks) turn_queries<T, D>(a, rot, q, b - q.first, pos);
    return;
  }
  const int k_groups = (a.H + HB - 1) / HB, per = k_groups + a.H, u = b / per, h = b - u * per;
  if (h < k_groups) write_turned_page<T, D, IT, HB>(a, rot, u, h * HB, krows, k_stride, wave_max);
  else write_page<T, D, IT>(a, u, h - k_groups, true, krows, k_stride, vrows, v_stride, wave_max);
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
// Heads of a queries' workgroup: as many as leave the card two of them a CU.
// Heads of a workgroup of K: two where pages are small enough for their
// cosines to stay in registers and pages and heads still fill the card.
template <typename T, int D, int IT>
struct RotaryK {
  static void go(dim3 grid, hipStream_t st, const KvDev &kv, RotaryDev rot, TurnArgs q, const void *k, int ks, const void *v, int vs) {
    if constexpr (IT * kKvThreads * 16 <= D * 128) {
      const int rows = kKvThreads / (D / 16), row_blocks = (kv.n + rows - 1) / rows;
      q.per = std::max(1, std::min(q.heads, q.heads * row_blocks / 512));
      q.groups = (q.heads + q.per - 1) / q.per;
      constexpr int HB = IT <= 2 ? 2 : 1;
      const bool two = HB == 2 && (long long)grid.x * grid.y >= 512;
      q.first = (int)grid.x * (two ? (kv.H + 1) / 2 + kv.H : 2 * kv.H);
      q.blocks = q.first + row_blocks * q.groups;
      const dim3 all(std::min(q.blocks, kGridRow), (unsigned)(((long long)q.blocks + kGridRow - 1) / kGridRow)), block(kKvThreads);
      if (two) hipLaunchKernelGGL((kv_write_rotary_kernel<T, D, IT, HB>), all, block, 0, st, kv, rot, q, (const T *)k, ks, (const T *)v, vs);
      else hipLaunchKernelGGL((kv_write_rotary_kernel<T, D, IT, 1>), all, block, 0, st, kv, rot, q, (const T *)k, ks, (const T *)v, vs);
    }
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
hipError_t launch_kv_write_rotary(const KvDev &kv, const RotaryDev &rot, const TurnArgs &q, int dim, int dtype, const void *k,
                                  int k_stride, const void *v, int v_stride, hipStream_t st) {
  return launch_by_type<RotaryK>(kv, dim, dtype, st, rot, q, k, k_stride, v, v_stride);
}
hipError_t launch_kv_read(const KvDev &kv, int dim, int dtype, void *k, int k_stride, void *v, int v_stride,
                          hipStream_t st) {
  return launch_by_type<ReadK>(kv, dim, dtype, st, k, k_stride, v, v_stride);
}

}  // namespace lora
