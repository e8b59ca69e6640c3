// k_fp8.hip -- y = W x in 8-bit floating point with a scale for each block of 128, and the quantisation in front of it.
//
//     y[i][o] = sum over blocks b of  xs[i][b] ws[o/128][b]  sum over k in b of  x[i][k] W[o][k]
//
// with e4m3 codes x and W, a scale for each row of x and 128 columns and one
// for each 128 x 128 block of W.  A block's 128 columns are one step of the
// matrix instruction: bf16 calls run v_mfma_f32_16x16x128_f8f6f4 on the codes
// as they are, from zero, and a multiply-add by xs ws takes each block's sums
// into the f32 accumulators.  The instruction adds its 128 products with
// fewer bits than f32: among a few that it aligns to the largest, those below
// 2^-13 of it lose digits.  Of normally distributed values 1.4e-5 of the result
// is lost, of random codes up to 1.6e-4 of the sum of magnitudes, and at worst
// 2^-10.2 of it (one product 2^14 times the size of all others), against the
// 2^-9 to which a bf16 y is rounded and the 2^-4 of the codes themselves.  f32
// calls therefore bring the codes to bf16, exactly, and run
// v_mfma_f32_16x16x32_bf16, which keeps f32 sums.
//
// The quantisation reads a row once and keeps it in registers between its
// maximum and its codes; memory bounds it (22016 x 4096 bf16 in blocks of 128 x
// 128: 52 us, 5.2 TB/s).  The product has three forms, by its rows: few of
// them stream W into registers, more share x through LDS, and many are tiles.
// Times below are of two weights in turn; 64 rows by 32000 x 4096 take 39 us
// among weights of which no cache holds anything.
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "fp8.hpp"

namespace lora {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------- quantisation
constexpr int kQuantThreads = 256;

// Sixteen values of a row.
template <typename T>
struct Raw16 {
  static constexpr int NV = sizeof(T);
  uint4 r[NV];
  __device__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < NV; ++i) r[i] = ldg16((const char *)p + 16 * i);
  }
  __device__ void zero() {
#pragma unroll
    for (int i = 0; i < NV; ++i) r[i] = z4();
  }
  __device__ float at(int i) const {
    const uint4 v = r[i * sizeof(T) / 16];
    const int b = i * sizeof(T) % 16 / 4;
    const uint32_t w = b == 0 ? v.x : b == 1 ? v.y : b == 2 ? v.z : v.w;
    if constexpr (sizeof(T) == 4) return __uint_as_float(w);
    else return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
  __device__ uint32_t largest() const {
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) big = max(big, finite_bits(at(i)));
    return big;
  }
  __device__ uint4 codes(float inv) const {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = codes4(at(4 * i), at(4 * i + 1), at(4 * i + 2), at(4 * i + 3), inv);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

__device__ __forceinline__ float power_of(int e) { return __uint_as_float((uint32_t)e << 23); }

// A thread takes 16 columns of a row, eight neighbouring lanes a block of 128.
template <typename T>
__global__ __launch_bounds__(kQuantThreads) void quantize_rows_kernel(QuantArgs a) {
  const int unit = blockIdx.x * kQuantThreads + threadIdx.x;
  const int row = a.per_row.div(unit), c = unit - row * a.per_row.d;
  const bool live = row < a.n && 16 * c < a.k;
  Raw16<T> x;
  if (live) x.load((const T *)a.x + row * a.x_stride + 16 * c);
  else x.zero();
  uint32_t big = x.largest();
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) big = max(big, (uint32_t)__shfl_xor((int)big, off, 64));
  const int e = exp_for(big);
  if (!live) return;
  *(uint4 *)(a.codes + row * a.c_stride + 16 * c) = x.codes(power_of(254 - e));
  if ((c & 7) == 0) a.scale[row * a.s_stride + c / 8] = power_of(e);
}

// A workgroup takes a 128 x 128 block: four times 32 rows of eight threads.
template <typename T>
__global__ __launch_bounds__(kQuantThreads) void quantize_blocks_kernel(QuantArgs a) {
  __shared__ uint32_t wave_max[kQuantThreads / 64];
  const int tid = threadIdx.x, rb = a.per_row.div(blockIdx.x), cb = blockIdx.x - rb * a.per_row.d;
  const int col = cb * kFp8Block + (tid & 7) * 16;
  Raw16<T> x[4];
  uint32_t big = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = rb * kFp8Block + i * 32 + (tid >> 3);
    if (row < a.n && col < a.k) x[i].load((const T *)a.x + row * a.x_stride + col);
    else x[i].zero();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) big = max(big, x[i].largest());
  big = (uint32_t)wave_reduce((int)big, 0, [](int a, int b) { return max(a, b); });  // bits of finite numbers: no sign
  if ((tid & 63) == 0) wave_max[tid >> 6] = big;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQuantThreads / 64; ++w) big = max(big, wave_max[w]);
  const int e = exp_for(big);
  if (tid == 0) a.scale[rb * a.s_stride + cb] = power_of(e);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = rb * kFp8Block + i * 32 + (tid >> 3);
    if (row < a.n && col < a.k) *(uint4 *)(a.codes + row * a.c_stride + col) = x[i].codes(power_of(254 - e));
  }
}

hipError_t launch_quantize_fp8(const QuantArgs &q, int dtype, int block_rows, hipStream_t st) {
  QuantArgs a = q;
  const int blocks = (a.k + kFp8Block - 1) / kFp8Block;
  if (block_rows == 1) {
    a.per_row = fast_div(blocks * 8);
    const dim3 grid((unsigned)(((long long)a.n * blocks * 8 + kQuantThreads - 1) / kQuantThreads));
    if (dtype == 0) hipLaunchKernelGGL((quantize_rows_kernel<float>), grid, dim3(kQuantThreads), 0, st, a);
    else hipLaunchKernelGGL((quantize_rows_kernel<u16>), grid, dim3(kQuantThreads), 0, st, a);
  } else {
    a.per_row = fast_div(blocks);
    const dim3 grid((unsigned)((a.n + kFp8Block - 1) / kFp8Block * blocks));
    if (dtype == 0) hipLaunchKernelGGL((quantize_blocks_kernel<float>), grid, dim3(kQuantThreads), 0, st, a);
    else hipLaunchKernelGGL((quantize_blocks_kernel<u16>), grid, dim3(kQuantThreads), 0, st, a);
  }
  return hipGetLastError();
}

// ---------------------------------------------------------------- products of 128 columns
// 128 columns of a row as a lane holds them: its 16 codes of the first 64 and
// of the last.  Both operands take their columns in the same order, which is
// all that a sum needs.
struct Codes {
  uint4 h[2];
};
struct Bf16Codes {
  bf16x8 v[4];
};
__device__ __forceinline__ Bf16Codes to_bf16(const Codes &c) {
  Bf16Codes r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 u = c.h[i / 2];
    const uint32_t lo = i & 1 ? u.z : u.x, hi = i & 1 ? u.w : u.y;
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true);
    const bf16x2 c2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true);
    r.v[i] = bf16x8{a[0], a[1], b[0], b[1], c2[0], c2[1], d[0], d[1]};
  }
  return r;
}
// The operand of a call's type: codes for bf16 results, bf16 numbers for f32 ones.
template <typename Y>
struct Operand;
template <>
struct Operand<u16> {
  i32x8 v;
  __device__ explicit Operand(const Codes &c) : v(__builtin_bit_cast(i32x8, c)) {}
  __device__ static f32x4 product(const Operand &a, const Operand &b) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
  }
};
template <>
struct Operand<float> {
  Bf16Codes v;
  __device__ explicit Operand(const Codes &c) : v(to_bf16(c)) {}
  __device__ static f32x4 product(const Operand &a, const Operand &b) {
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v.v[i], b.v.v[i], s, 0, 0, 0);
    return s;
  }
};
// Four neighbouring outputs of a row.
__device__ __forceinline__ void store4(u16 *p, f32x4 v) {
  *(uint2 *)p = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}
__device__ __forceinline__ void store4(float *p, f32x4 v) { *(float4 *)p = make_float4(v[0], v[1], v[2], v[3]); }

// ---------------------------------------------------------------- few rows
// W is streamed once and bounds the call: one row by 22016 x 4096 19 us.  128 columns of a row of codes, by
// a lane's two 16-byte loads; columns past k are zeros.
__device__ __forceinline__ Codes fetch_block(const uint8_t *row, int block, int k) {
  const int c0 = ((int)threadIdx.x & 48) + block * kFp8Block;  // lane / 16 * 16
  Codes c;
#pragma unroll
  for (int h = 0; h < 2; ++h) c.h[h] = c0 + 64 * h < k ? ldg16(row + c0 + 64 * h) : z4();
  return c;
}

// A block's two scales apply as one f32 product.  Past f32's end that is an
// infinity, and the block's sum by it an infinity or NaN also where the result
// is 0 or a number.  There they have to apply one after the other.  A look at
// every product would cost up to a seventh of a call (36 rows by 6144 x 4096:
// 14.1 us for 12.3), but such a product leaves the sums infinite or NaN for
// good, so that a look at these does.  A wave that finds some looks at its
// scales, and only if one of their products is past the end forms its sums
// anew, the same bits for all other rows.
struct Doubt {
  float zero = 0.f;
  __device__ void look(const f32x4 &v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) zero = fmaf(v[i], 0.f, zero);  // NaN by an infinity or NaN
  }
  __device__ bool any() const { return __any(zero != 0.f); }
};
__device__ __forceinline__ bool held(float a, float b) {
  return __builtin_isfinite(a * b) || !__builtin_isfinite(a) || !__builtin_isfinite(b);
}
// Of 16 rows from r0 and 16 outputs from o0, the blocks first, first + step, ..
struct Sixteen {
  const uint8_t *wrow, *xrow;
  const float *xs, *ws;
  __device__ Sixteen(const Fp8Args &p, int o0, int r0) {
    const int lane = threadIdx.x & 63, r = min(r0 + (lane & 15), p.n - 1);
    wrow = p.W + min(o0 + (lane & 15), p.n_out - 1) * p.w_stride;
    xrow = p.x + r * p.x_stride;
    xs = p.x_scale + r * p.xs_stride;
    ws = p.w_scale + (min(o0, p.n_out - 1) / kFp8Block) * p.ws_stride;
  }
  // Every fourth block a lane, four of them side by side; at the end the last again.
  __device__ bool scales_held(int first, int step, int k) const {
    const int last = (k - 1) / kFp8Block;
    bool all = true;
#pragma unroll 1
    for (int at = first + ((threadIdx.x >> 4) & 3) * step; at <= last; at += 16 * step) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = xs[min(at + 4 * i * step, last)];
        b[i] = ws[min(at + 4 * i * step, last)];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) all &= held(a[i], b[i]);
    }
    return __all(all);
  }
  // Scales whose product is not held apply in turn: either is above 1, and a
  // sum of codes is 0 or 2^-18 or more, so that what passes f32's end on the
  // way is past it in the end, too.
  template <typename Y>
  __device__ f32x4 sums(int first, int step, int k) const {
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int at = first; at * kFp8Block < k; at += step) {
      const f32x4 v = Operand<Y>::product(Operand<Y>(fetch_block(wrow, at, k)), Operand<Y>(fetch_block(xrow, at, k)));
      const float a = xs[at], b = ws[at];
      const bool one = held(a, b);
      const float before = one ? 1.f : a, then = one ? a * b : b;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(v[i] * before, then, acc[i]);
    }
    return acc;
  }
};

// Up to 16 rows.  A workgroup owns 16 output features; its eight waves share
// the columns out by blocks, W and x straight into registers, and meet in LDS
// at the end, in the order of the waves.
constexpr int kFewWaves = 8;
template <typename Y>
__global__ __launch_bounds__(kFewWaves * 64) void matmul_few_kernel(Fp8Args p) {
  constexpr int U = 4;  // blocks of W in flight
  __shared__ f32x4 part[kFewWaves][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int o0 = blockIdx.x * 16, blocks = (p.k + kFp8Block - 1) / kFp8Block;
  const int r = min(lane & 15, p.n - 1);
  const uint8_t *wrow = p.W + min(o0 + (lane & 15), p.n_out - 1) * p.w_stride, *xrow = p.x + r * p.x_stride;
  const float *xs = p.x_scale + r * p.xs_stride, *ws = p.w_scale + (o0 / kFp8Block) * p.ws_stride;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  Codes w[U];
#pragma unroll
  for (int u = 0; u < U; ++u) w[u] = fetch_block(wrow, wave + u * kFewWaves, p.k);
  for (int kb = wave; kb < blocks; kb += U * kFewWaves) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = kb + u * kFewWaves;
      if (at >= blocks) break;
      const Codes x = fetch_block(xrow, at, p.k);
      const float s = xs[at] * ws[at];
      const Operand<Y> wo(w[u]);
      w[u] = fetch_block(wrow, at + U * kFewWaves, p.k);
      const f32x4 v = Operand<Y>::product(wo, Operand<Y>(x));
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(v[i], s, acc[i]);
    }
  }
  Doubt doubt;
  doubt.look(acc);
  if (__builtin_expect(doubt.any(), 0)) {
    const Sixteen own(p, o0, 0);
    if (!own.scales_held(wave, kFewWaves, p.k)) acc = own.template sums<Y>(wave, kFewWaves, p.k);
  }
  part[wave][lane] = acc;
  __syncthreads();
  if (tid >= 64) return;
  f32x4 v = part[0][lane];
#pragma unroll
  for (int s = 1; s < kFewWaves; ++s) v += part[s][lane];
  const int row = lane & 15, o = o0 + (lane >> 4) * 4;
  if (row < p.n && o < p.n_out) store4((Y *)p.y + row * p.y_stride + o, v);
}

// Up to 16 NB rows, W's stream again the bound (64 rows by 32000 x 4096: 30 us).  Every workgroup reads all of x, a part of 64 KB at a time
// (1024 columns of 64 rows), through registers into the half of LDS that the
// part before the last has left, while W streams into registers, eight blocks
// of a wave ahead and across the parts.  Of the eight waves RG take 16 output
// features each and KG = 8 / RG share the columns out by blocks, as many of
// the former as leave every CU a workgroup.  Rows of a block lie as in the
// tiles below.  Loads return in order, so that x straight into the operands'
// registers makes every wait for x one for W (64 rows by 32000 x 4096: 68 us;
// 40 with both operands through LDS).
template <typename Y, int NB, int RG>
__global__ __launch_bounds__(512) void matmul_rows_kernel(Fp8Args p) {
  constexpr int KG = 8 / RG, U = 8, kRows = 16 * NB;
  constexpr int kPart = 512 / kRows;  // blocks of a part
  constexpr int kEach = kPart / KG;   // of a wave
  constexpr int kIns = 512 * 8 / 512; // 16-byte chunks that a thread brings
  static_assert(kPart * kRows == 512 && kEach * KG == kPart && (U % kEach == 0 || kEach % U == 0), "parts of 512 rows of a block");
  __shared__ __attribute__((aligned(16))) uint4 xl[2][512 * 8];
  __shared__ float sl[2][512];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rg = wave % RG, kg = wave / RG;
  const int o0 = (blockIdx.x * RG + rg) * 16, blocks = (p.k + kFp8Block - 1) / kFp8Block;
  const uint8_t *wrow = p.W + min(o0 + (lane & 15), p.n_out - 1) * p.w_stride;
  const float *ws = p.w_scale + (min(o0, p.n_out - 1) / kFp8Block) * p.ws_stride;

  // This thread's chunks of a part: chunk tid % 8 of rows tid / 8 + 64 i, and the scale of row tid.
  uint4 xr[kIns];
  float sr;
  auto fetch_x = [&](int part) {
#pragma unroll
    for (int i = 0; i < kIns; ++i) {
      const int rr = (tid >> 3) + 64 * i, row = min(rr % kRows, p.n - 1);
      const int at = (part * kPart + rr / kRows) * kFp8Block + (tid & 7) * 16;
      xr[i] = ldg16(p.x + row * p.x_stride + (at < p.k ? at : 0));
    }
    sr = p.x_scale[min(tid % kRows, p.n - 1) * p.xs_stride + min(part * kPart + tid / kRows, blocks - 1)];
  };
  // Columns past k are zeros, by masks: loads inside a branch make the wave wait for all of them where it ends.
  auto keep_x = [&](int part) {
    uint4 *const to = xl[part & 1];
#pragma unroll
    for (int i = 0; i < kIns; ++i) {
      const int rr = (tid >> 3) + 64 * i, slot = (tid & 7) ^ ((rr >> 1) & 7);
      const uint32_t m = (part * kPart + rr / kRows) * kFp8Block + (tid & 7) * 16 < p.k ? ~0u : 0u;
      to[rr * 8 + slot] = make_uint4(xr[i].x & m, xr[i].y & m, xr[i].z & m, xr[i].w & m);
    }
    sl[part & 1][tid] = sr;
  };
  // W's columns past k are any others of the row: x is 0 there.
  auto fetch_w = [&](int block) {
    Codes c;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = block * kFp8Block + 64 * h + (lane >> 4) * 16;
      c.h[h] = ldg16(wrow + (at < p.k ? at : 0));
    }
    return c;
  };

  f32x4 acc[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int parts = (blocks + kPart - 1) / kPart, all = parts * kEach;  // blocks of a wave, the last part's empty ones too
  fetch_x(0);
  // W's scales, 64 blocks' in the lanes: a scalar load of each is a wait of its own
  auto fetch_ws = [&](int first) { return ws[min(first + lane, blocks - 1)]; };
  float wl = fetch_ws(0);
  Codes w[U];
#pragma unroll
  for (int u = 0; u < U; ++u) w[u] = fetch_w(kg + u * KG);
  keep_x(0);
  __syncthreads();
  for (int j0 = 0; j0 < all; j0 += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u, part = j / kEach;
      if (j >= all) break;
      if (j % kEach == 0) {
        if (part + 1 < parts) fetch_x(part + 1);
        if (part && part * kPart % 64 == 0) wl = fetch_ws(part * kPart);
      }
      const int kb = kg + j * KG;
      if (kb < blocks) {  // the branch keeps blocks apart: their reads of LDS side by side take registers that spill
        const float wsc = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wl), kb & 63));
        const Operand<Y> wo(w[u]);
        const uint4 *const xp = xl[part & 1] + kb % kPart * kRows * 8;
        const float *const sp = sl[part & 1] + kb % kPart * kRows;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const int row = 16 * b + (lane & 15), c = lane >> 4, x = (row >> 1) & 7;
          Codes v;
          v.h[0] = xp[row * 8 + (c ^ x)];
          v.h[1] = xp[row * 8 + ((4 + c) ^ x)];
          const float s = sp[row] * wsc;
          const f32x4 r = Operand<Y>::product(wo, Operand<Y>(v));
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[b][i] = fmaf(r[i], s, acc[b][i]);
        }
      }
      w[u] = fetch_w(kg + (j + U) * KG);
      if (j % kEach == kEach - 1 && part + 1 < parts) {
        keep_x(part + 1);
        __syncthreads();
      }
    }
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    Doubt doubt;
    doubt.look(acc[b]);
    if (__builtin_expect(doubt.any(), 0)) {
      const Sixteen own(p, o0, 16 * b);
      if (!own.scales_held(kg, KG, p.k)) acc[b] = own.template sums<Y>(kg, KG, p.k);
    }
  }
  const int o = o0 + (lane >> 4) * 4;
  if constexpr (KG > 1) {
    f32x4 *const sums = (f32x4 *)xl;  // [KG][RG][NB][64]
    __syncthreads();  // every wave is done with x
#pragma unroll
    for (int b = 0; b < NB; ++b) sums[(wave * NB + b) * 64 + lane] = acc[b];
    __syncthreads();
    if (kg) return;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int g = 1; g < KG; ++g) acc[b] += sums[((g * RG + rg) * NB + b) * 64 + lane];
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int row = 16 * b + (lane & 15);
    if (row < p.n && o < p.n_out) store4((Y *)p.y + row * p.y_stride + o, acc[b]);
  }
}

// ---------------------------------------------------------------- many rows
// The rows from `first` on of an n-row matrix of `stride` bytes a row and `width` of them in use.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_rsrc(const void *base, int first, int n, long long stride, int width) {
  const long long bytes = (n - first - 1) * stride + width;
  return __builtin_amdgcn_make_buffer_rsrc((void *)((uintptr_t)base + first * stride), 0, (int)min(bytes, 0xffffffffll), 0x00020000);
}
// dma16 and dma4 (common.hpp) through a buffer resource.
__device__ __forceinline__ void dma16_buffer(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" : : "v"(voff), "s"(r), "s"(soff), "s"(lds) : "memory");
}
__device__ __forceinline__ void dma4_buffer(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dword %0, %1, %2 offen lds" : : "v"(voff), "s"(r), "s"(soff), "s"(lds) : "memory");
}

// A workgroup owns BO output features x BR rows.  A stage is one block of 128
// columns of every row of the tile, brought to LDS by LDS-DMA: 128 bytes a
// row, its eight 16-byte chunks at slot c ^ ((r >> 1) & 7), so that the
// operands' reads hit distinct banks.  The rows' scales come by eight blocks
// at a time, a part of the next eight with every stage: a scale a row and
// stage is as many cache lines as the codes are (4096 x 22016 x 4096: 529 us
// that way).  NS stages form a ring with NS - 1 in flight; the waits are
// explicit, and a stage is read only after every wave's share of it landed.
// Rows past the ends read as nothing and are not stored; chunks past k are
// zeroed once they have landed.  No one unit bounds the largest tiles: 4096 x
// 22016 x 4096 take 392 to 402 us, 1.9 PFLOP/s, in which the matrix units are
// busy for 43 % and vector instructions, a multiply-add for each result of the
// matrix ones above all, for 34 %; the two waves of a SIMD wait 35 % of their
// time, and 1376 tiles are 5.4 rounds that take 6.  (Single passes range
// from 376 to 487 us as the clock follows the load.)
template <typename Y, int BO, int BR, int WGO, int WGR, int NS>
__global__ __launch_bounds__(WGO *WGR * 64) void matmul_tile_kernel(Fp8Args p, int n_otiles, int n_rtiles) {
  constexpr int NW = WGO * WGR;
  constexpr int WO = BO / WGO, WR = BR / WGR, NBO = WO / 16, NBR = WR / 16;
  constexpr int RS = BO + BR, LPW = RS / 8 / NW, JW = BO / 8 / NW;
  static_assert(LPW * 8 * NW == RS && JW * 8 * NW == BO, "a stage's rows split evenly over the waves");
  static_assert(BR % 64 == 0 && BR / 64 <= NW, "a wave's lanes bring 64 rows' scales");
  static_assert(NS >= 2 && (NS - 2) * (LPW + 1) < 64, "ring depth / vmcnt range");
  static_assert(WO <= kFp8Block && kFp8Block % WO == 0, "a wave's outputs share their scales");
  constexpr bool kSpread = NBO >= 8;  // small tiles have little to spread them over (512 x 4096 x 4096: 22 us, 27 spread)
  __shared__ __attribute__((aligned(16))) uint4 ring[NS][RS * 8];
  __shared__ float xs[3][BR * 8];  // [row][block] of the eight blocks in use, the next and, for waves behind, the last
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wo = wave % WGO, wr = wave / WGO;
  // An XCD's workgroups take neighbouring tiles, which its L2 then serves:
  // groups of up to 8 row tiles, rows fastest.
  const int G = n_otiles * n_rtiles, b = blockIdx.x, xq = G / 8, xr = G % 8, xcd = b % 8;
  const int t = xcd * xq + min(xcd, xr) + b / 8;
  const int g0 = t / (8 * n_otiles) * 8, gsz = min(8, n_rtiles - g0), tg = t - g0 * n_otiles;
  const int r0 = (g0 + tg % gsz) * BR, o0 = tg / gsz * BO;
  const int nst = (p.k + kFp8Block - 1) / kFp8Block;

  // Operands through buffer resources that begin at the tile and end with the
  // last row's k columns.  A lane's offset, which is checked against that end,
  // carries the row, which may lie past it and is then not read; the scalar
  // offset, which need not be checked, carries the stage's first column, and
  // in the last stage lanes past k step back to it (stage_column).
  const __amdgpu_buffer_rsrc_t wsrc = tile_rsrc(p.W, o0, p.n_out, p.w_stride, p.k), xsrc = tile_rsrc(p.x, r0, p.n, p.x_stride, p.k);
  const __amdgpu_buffer_rsrc_t ssrc = tile_rsrc(p.x_scale, r0, p.n, 4 * p.xs_stride, 4 * nst);
  const int chunk = stage_chunk(wave * 8 + (lane >> 3), lane & 7);  // this lane's place in the stage's rows
  uint32_t woff = (wave * 8 + (lane >> 3)) * (uint32_t)p.w_stride + chunk, xoff = (wave * 8 + (lane >> 3)) * (uint32_t)p.x_stride + chunk;
  // part i of 8 of the scales of blocks 8 g .. 8 g + 7: BR / 8 rows, a wave 8 of them
  const uint32_t soff = (wave % (BR / 64) * 8 + (lane >> 3)) * 4 * (uint32_t)p.xs_stride + 4 * (lane & 7);
  auto bring_scales = [&](int g, int i) {
    dma4_buffer(ssrc, soff + 4 * (i * (BR / 8) * (uint32_t)p.xs_stride + 8 * g), 0, lds_addr(&xs[g % 3][(i * (BR / 8) + wave % (BR / 64) * 8) * 8]));
  };
  // Before the last stage's first transfer.
  auto step_back = [&] {
    const uint32_t by = chunk - stage_column(chunk, (nst - 1) * kFp8Block, p.k);
    woff -= by;
    xoff -= by;
  };
  // Stages past the last bring the last again, into places that nothing reads
  // any more, so that the waits count the same in every stage.
  auto issue = [&](int st, int from, int to) {
    const uint32_t k0 = min(st, nst - 1) * kFp8Block;
#pragma unroll
    for (int j = from; j < to; ++j) {
      const uint32_t lds = lds_addr(&ring[st % NS][(wave + NW * j) * 64]);
      if (j < JW) dma16_buffer(wsrc, woff + 8 * NW * j * (uint32_t)p.w_stride, k0, lds);
      else dma16_buffer(xsrc, xoff + 8 * NW * (j - JW) * (uint32_t)p.x_stride, k0, lds);
    }
  };
  for (int i = 0; i < 8; ++i) bring_scales(0, i);
  for (int st = 0; st < NS - 1; ++st) {
    if (st == nst - 1) step_back();
    issue(st, 0, LPW);
    bring_scales(st / 8 + 1, st % 8);
  }

  f32x4 acc[NBO][NBR];
#pragma unroll
  for (int a = 0; a < NBO; ++a)
#pragma unroll
    for (int c = 0; c < NBR; ++c) acc[a][c] = f32x4{0.f, 0.f, 0.f, 0.f};
  const float *ws = p.w_scale + (long long)min((o0 + wo * WO) / kFp8Block, (p.n_out - 1) / kFp8Block) * p.ws_stride;
  auto read = [&](int st, int r) {
    const uint4 *sl = ring[st % NS];
    const int c = lane >> 4, x = (r >> 1) & 7;
    Codes v;
    v.h[0] = sl[r * 8 + (c ^ x)];
    v.h[1] = sl[r * 8 + ((4 + c) ^ x)];
    return v;
  };
  float wl = 0.f;  // the scales of 64 blocks in the lanes
  for (int st = 0; st < nst; ++st) {
    if (st % 64 == 0) wl = ws[min(st + lane, nst - 1)];
    const float wsc = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wl), st & 63));
    wait_vmcnt<(NS - 2) * (LPW + 1)>();
    if ((st + 1) * kFp8Block > p.k) {
      if (st * kFp8Block + chunk >= p.k)
#pragma unroll
        for (int j = 0; j < LPW; ++j) ring[st % NS][(wave + NW * j) * 64 + lane] = z4();
    }
    // zeros are there, and the last stage's reads have returned before its place is written again
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    block_barrier();
    // Every wave is done with stage st - 1: its place takes stage st + NS - 1,
    // whose transfers go out among the products, as all of them together hold
    // the waves up.
    if (st + NS - 1 == nst - 1) step_back();
    if constexpr (!kSpread) {
      issue(st + NS - 1, 0, LPW);
      bring_scales((st + NS - 1) / 8 + 1, (st + NS - 1) % 8);
    }
    float s[NBR];
#pragma unroll
    for (int c = 0; c < NBR; ++c) s[c] = xs[st / 8 % 3][(wr * WR + c * 16 + (lane & 15)) * 8 + st % 8] * wsc;
    Codes xf[NBR], wf = read(st, wo * WO + (lane & 15)), next;
#pragma unroll
    for (int c = 0; c < NBR; ++c) xf[c] = read(st, BO + wr * WR + c * 16 + (lane & 15));
#pragma unroll
    for (int a = 0; a < NBO; ++a) {
      if (a + 1 < NBO) next = read(st, wo * WO + (a + 1) * 16 + (lane & 15));
      if constexpr (kSpread) {
        if (a < 4) issue(st + NS - 1, a * LPW / 4, (a + 1) * LPW / 4);
        if (a == 3) bring_scales((st + NS - 1) / 8 + 1, (st + NS - 1) % 8);
      }
      const Operand<Y> w(wf);
#pragma unroll
      for (int c = 0; c < NBR; ++c) {
        const f32x4 r = Operand<Y>::product(w, Operand<Y>(xf[c]));
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[a][c][i] = fmaf(r[i], s[c], acc[a][c][i]);
      }
      wf = next;
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  wait_vmcnt<0>();  // nothing is on its way into LDS when the workgroup ends
  Doubt doubt;
#pragma unroll
  for (int c = 0; c < NBR; ++c) {
    const int row = r0 + wr * WR + c * 16 + (lane & 15);
    if (row >= p.n) continue;
    Y *to = (Y *)p.y + row * p.y_stride;
#pragma unroll
    for (int a = 0; a < NBO; ++a) {
      const int o = o0 + wo * WO + a * 16 + (lane >> 4) * 4;
      if (o >= p.n_out) continue;
      store4(to + o, acc[a][c]);
      doubt.look(acc[a][c]);
    }
  }
  // behind the stores, so that no sum has to be kept beside this
  if (__builtin_expect(!doubt.any(), 1)) return;
#pragma unroll 1
  for (int c = 0; c < NBR; ++c) {
    const int r16 = r0 + wr * WR + c * 16;
    if (Sixteen(p, o0 + wo * WO, r16).scales_held(0, 1, p.k)) continue;
#pragma unroll 1
    for (int a = 0; a < NBO; ++a) {
      const int o16 = o0 + wo * WO + a * 16, row = r16 + (lane & 15), o = o16 + (lane >> 4) * 4;
      const f32x4 v = Sixteen(p, o16, r16).template sums<Y>(0, 1, p.k);
      if (row < p.n && o < p.n_out) store4((Y *)p.y + row * p.y_stride + o, v);
    }
  }
}

// Of matmul_rows_kernel: a CU takes in W at about 25 bytes a ns and x, from
// L2, at about 45, and has room for one workgroup: the rounds of workgroups
// times what one brings and a little to begin with.  64 rows by k of 4096 in
// bf16, us with RG of 8, 4, 2, 1: n_out 32000 31.7 39.6 55.7 94; 22016 26.1
// 34.2 40.3 68; 11008 24.8 17.5 26.9 36; 6144 24.3 17.0 14.1 24.  The rule is
// fitted to these and sees neither k nor the type; of n_out 4096, 11008 and
// 32000 it takes the best also at k of 1024 and 11008 and in f32, or one within
// 6 % of it (k of 11008, 4096 outputs: 28.1, 26.5 with RG of 2).
static float rows_cost(int groups, int nb, int *best) {
  float least = 0.f;
  *best = 0;
  for (int rg = 8; rg >= 1; rg /= 2) {
    const int rounds = ((groups + rg - 1) / rg + 255) / 256;
    const float cost = rounds * (rg / 25.f + nb / 45.f + 0.02f);
    if (*best && cost >= least) continue;
    *best = rg;
    least = cost;
  }
  return least;
}
template <typename Y, int NB>
static void launch_rows(const Fp8Args &a, int rg, hipStream_t st) {
#define LORA_ROWS(RG) \
  hipLaunchKernelGGL((matmul_rows_kernel<Y, NB, RG>), dim3((a.n_out + 16 * RG - 1) / (16 * RG)), dim3(512), 0, st, a)
  if (rg == 8) LORA_ROWS(8);
  else if (rg == 4) LORA_ROWS(4);
  else if (rg == 2) LORA_ROWS(2);
  else LORA_ROWS(1);
#undef LORA_ROWS
}
// Up to 64 rows.  Up to 16 of them by matmul_few_kernel where it takes less:
// several of its workgroups fit a CU, so that there are no rounds, but each
// reads its rows of x again, and no wave has W of its own in flight behind
// them.  Us with it and with matmul_rows_kernel, k of 4096: 1 row n_out 4096
// 5.3 8.4, 32000 26.1 23.4; 16 rows 4096 7.0 8.6, 11008 16.1 14.1, 32000 38 24,
// and in f32 the same choice is the better one.  Fitted at that k, it changes
// over too early at others: k of 1024, 1 row n_out 32000 9.0 20.8, 16 rows
// 11008 7.2 13.2, 32000 12.8 21.1; k of 11008, 1 row 32000 71 95.
template <typename Y>
static void launch_few(const Fp8Args &a, hipStream_t st) {
  const int groups = (a.n_out + 15) / 16;
  int rg;
  if (a.n <= 16) {
    const float few = 1.25f * (groups / 256.f) * (1.f / 25.f + a.n / 16.f / 45.f);
    if (few <= rows_cost(groups, 1, &rg))
      hipLaunchKernelGGL((matmul_few_kernel<Y>), dim3((a.n_out + 15) / 16), dim3(kFewWaves * 64), 0, st, a);
    else launch_rows<Y, 1>(a, rg, st);
  } else if (a.n <= 32) {
    rows_cost(groups, 2, &rg);
    launch_rows<Y, 2>(a, rg, st);
  } else {
    rows_cost(groups, 4, &rg);
    launch_rows<Y, 4>(a, rg, st);
  }
}
template <typename Y>
static void launch_tiles(const Fp8Args &a, hipStream_t st) {
#define LORA_TILE(BO, BR, WGO, WGR, NS)                                                                                  \
  hipLaunchKernelGGL((matmul_tile_kernel<Y, BO, BR, WGO, WGR, NS>),                                                      \
                     dim3(((a.n_out + BO - 1) / BO) * ((a.n + BR - 1) / BR)), dim3(WGO * WGR * 64), 0, st, a,             \
                     (a.n_out + BO - 1) / BO, (a.n + BR - 1) / BR)
  // Time in units of what a CU takes for a round of the largest tiles (k of
  // 4096: 62 us).  A CU holds one workgroup of 256 x 256, two of 128 x 128 and
  // two of 64 x 64, of which the first alone takes as long as both.  Us with
  // tiles of 64, 128, 256, k of 4096: 129 x 4096 17.7 25.0 51.6, 1024 x 4096
  // 40 28 57, 512 x 22016 105 63 60, 4096 x 4096 144 82 72, 4096 x 22016 757
  // 460 400.  Fitted in bf16 at that k; of 31 sizes of 128 to 2048 rows by 4096
  // and 11008 in f32 and at k of 1024 and 11008 three take over 5 % longer than
  // they might: at k of 1024, with 128 and the 256 taken, 2048 x 11008 42.1
  // 45.5, in f32 59.9 67.8, and 1024 x 11008 in f32 33.0 35.8.
  auto tiles = [&](int e) { return (long long)((a.n_out + e - 1) / e) * ((a.n + e - 1) / e); };
  auto rounds = [](long long n, int of) { return (n + of - 1) / of; };
  const float big = 1.f * rounds(tiles(256), 256), small = 0.33f * rounds(tiles(64), 512);
  const float mid = 0.67f * (tiles(128) / 512) + (tiles(128) % 512 == 0 ? 0.f : tiles(128) % 512 <= 256 ? 0.43f : 0.67f);
  if (small <= mid && small <= big) LORA_TILE(64, 64, 2, 2, 4);
  else if (mid < big) LORA_TILE(128, 128, 2, 4, 2);
  else LORA_TILE(256, 256, 2, 4, 2);
#undef LORA_TILE
}

hipError_t launch_matmul_fp8(const Fp8Args &a, int dtype, hipStream_t st) {
  // Tiles from 65 rows on: 100 rows by k of 4096 at n_out 4096, 11008, 22016,
  // 32000 take 17 21 27 28 us with them, 19 27 39 41 with eight blocks of 16 in
  // matmul_rows_kernel; 64 rows 17 21 26 27 and 13 17 26 29.
  if (a.n <= 64) {
    if (dtype == 0) launch_few<float>(a, st);
    else launch_few<u16>(a, st);
  } else {
    if (dtype == 0) launch_tiles<float>(a, st);
    else launch_tiles<u16>(a, st);
  }
  return hipGetLastError();
}

}  // namespace lora
