// k_attend.hip -- attention of ragged query rows over the 8-bit paged cache.
//
// For a sequence with rows j = 0 .. m-1 at positions start + j, query head h
// and key/value head h / G:
//     o_j = sum_t w_jt v_t / sum_t w_jt,  w_jt = exp(scale q_j . k_t),
// over the tokens t <= start + j (and t > start + j - window), k_t = 2^a c_t
// and v_t = 2^b d_t with the page's exponents a, b and e4m3 codes c, d.
//
// The codes go into the matrix instructions as they are: e4m3 numbers are
// exact in bf16 and in f16, so a code costs half a conversion instruction
// and the scales never touch an element.  With S = q . c the weight times
// the page's value scale is
//     2^(S 2^a scale log2(e) + b - M),
// one fma and one exp2 a score, and M, the running maximum of that exponent,
// keeps it in (0, 1]; the accumulators sum it against the codes d and the
// denominator sums it times 2^-b.  No choice of page scales overflows or
// loses bits this way.
//
// A column is a (row, query head of the group) pair; a wave holds 16 NB
// columns and walks tiles of 64 tokens.  K's tile is the A operand (64
// tokens x D), the columns the B operand, and the order of tokens within the
// tile is chosen so that lane (column, g) ends up with the scores of the 16
// tokens of 16-token group g: those are the B operand of the second product
// as they stand, V's 16 bytes of a dim the A operand, and a lane's 16 tokens
// share one page, one a and one b.  No score crosses a lane but in the
// column's maximum, and every load is 16 bytes a lane in runs of 256.
//
// Rounding: bf16 calls take q as it is and round the weights to f16 (2^-12,
// an eighth of the output's own half step); f32 calls split q and the
// weights into three bf16 terms (24 bits) and take three products of each.
// Scores, sums and outputs accumulate in f32.
//
// Two forms share the code.  Decode and verify (few columns a sequence): the
// workgroup's four waves take every fourth tile of the unit and are joined
// through LDS.  Wide (many rows): the waves take 16 NB columns each.  In
// both, the call's tiles are shared out in chunks of equal length over about
// kAttendTarget workgroups, from the lengths in device memory, so long and
// short sequences balance; a unit (sequence, head, columns) of several
// chunks is joined inside the launch by the last to arrive, in groups of
// about the square root of their number so that no join is long.
#include "common.hpp"
#include "verify.hpp"

namespace lora {

constexpr int kTile = 64;      // tokens
constexpr int kMaxGroup = 32;  // chunks of a group, groups of a unit
static_assert(kMaxGroup * kMaxGroup >= kAttendTarget, "two levels of groups cover a unit's chunks");

typedef int i32x2 __attribute__((ext_vector_type(2)));

// max / sum over the four lane groups l / 16 that hold a column's tokens.
__device__ __forceinline__ float groups_max(float x) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float groups_sum(float x) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// Eight codes (two dwords) as a matrix operand.
__device__ __forceinline__ uint4 codes_bf16(uint32_t lo, uint32_t hi) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return make_uint4(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, c),
                    __builtin_bit_cast(uint32_t, d));
}
__device__ __forceinline__ uint4 codes_f16(uint32_t lo, uint32_t hi) {
  const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
  const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
  const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
  const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
  return make_uint4(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, c),
                    __builtin_bit_cast(uint32_t, d));
}
__device__ __forceinline__ f32x4 mfma16_f16(uint4 a, uint4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const f32x2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const f32x2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}

// Eight f32 as three bf16 operands whose sum holds all 24 bits.
__device__ __forceinline__ void split3(const float x[8], uint4 t[3]) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
  for (int n = 0; n < 3; ++n) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = pack_bf16(r[2 * i], r[2 * i + 1]);
      r[2 * i] -= __uint_as_float(w[i] << 16);
      r[2 * i + 1] -= __uint_as_float(w[i] & 0xffff0000u);
    }
    t[n] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Bytes that hold a NaN code, 0xff each.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  const uint32_t f = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
  return (f >> 7) * 0xffu;
}

// Bytes of four tokens from t0 that lie in [lo, hi).
__device__ __forceinline__ uint32_t live_bytes(int t0, int lo, int hi) {
  const int a = min(max(lo - t0, 0), 4), b = min(max(hi - t0, 0), 4);
  return b > a ? (uint32_t)((1ull << (8 * b)) - (1ull << (8 * a))) : 0u;
}

// ---------------------------------------------------------------- the call's work
struct Work {
  SeqDev s;
  int seq, block, chunk, nc, slot;  // slot: of the unit's chunk 0, in steps of H
};

template <int CB>
__device__ __forceinline__ int seq_blocks(const AttendArgs &a, const SeqDev &s) {
  const int cols = s.rows * a.G;
  return cols > a.cols_lo && cols <= a.cols_hi ? (cols + CB - 1) / CB : 0;
}
// Tiles that some row of the sequence sees; 1 where none does (its rows are written as zeros).
__device__ __forceinline__ int seq_tiles(const AttendArgs &a, const SeqDev &s, int cap) {
  const int lo = a.window ? max(0, s.start + 1 - a.window) : 0, hi = min(s.len, cap);
  return hi > lo ? ((hi + kTile - 1) / kTile) - lo / kTile : 1;
}

// Item u of a head's list: units in order, each with its chunks.  Every wave
// finds it by itself (lane l counts `per` sequences).
template <int CB>
__device__ __forceinline__ bool find_work(const AttendArgs &a, int u, int lane, Work *w) {
  const int per = (a.kv.n_seqs + 63) >> 6, cap = kv_cap(a.kv);
  const int i0 = lane * per, i1 = min(i0 + per, a.kv.n_seqs);
  SeqDev first = {0, 0, 0, 0};  // the lane's only sequence where per is 1
  if (i0 < i1) first = load_seq(a.kv, i0);
  long long total = 0;
  for (int i = i0; i < i1; ++i) {
    const SeqDev s = i == i0 ? first : load_seq(a.kv, i);
    total += (long long)seq_blocks<CB>(a, s) * seq_tiles(a, s, cap);
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) total += __shfl_xor(total, off, 64);
  const long long len = (total + a.per_head - 1) / a.per_head;
  const int c = (int)min(max(len, 1ll), 1ll << 30);  // tiles of a chunk at most
  int items = 0, slots = 0;
  for (int i = i0; i < i1; ++i) {
    const SeqDev s = i == i0 ? first : load_seq(a.kv, i);
    const int b = seq_blocks<CB>(a, s), nc = (seq_tiles(a, s, cap) + c - 1) / c;
    items += b * nc;
    slots += nc > 1 ? b * nc : 0;
  }
  const int incl = wave_incl_scan(items, lane), sincl = wave_incl_scan(slots, lane);
  int found = -1, block = 0, chunk = 0, nc_of = 1, slot = 0;
  if (u < incl && u >= incl - items) {
    int at = incl - items, sat = sincl - slots;
    for (int i = i0; i < i1; ++i) {
      const SeqDev s = i == i0 ? first : load_seq(a.kv, i);
      const int b = seq_blocks<CB>(a, s), nc = (seq_tiles(a, s, cap) + c - 1) / c;
      if (u < at + b * nc) {
        found = i;
        nc_of = nc;
        const int unit = (u - at) / nc;
        chunk = (u - at) - unit * nc;
        block = b - 1 - unit;  // the later rows of a prompt see the most tokens: first
        slot = sat + unit * nc;
        break;
      }
      at += b * nc;
      sat += nc > 1 ? b * nc : 0;
    }
  }
  const unsigned long long who = __ballot(found >= 0);
  if (!who) return false;
  const int src = __ffsll(who) - 1;
  w->seq = __builtin_amdgcn_readlane(found, src);
  w->block = __builtin_amdgcn_readlane(block, src);
  w->chunk = __builtin_amdgcn_readlane(chunk, src);
  w->nc = __builtin_amdgcn_readlane(nc_of, src);
  w->slot = __builtin_amdgcn_readlane(slot, src);
  w->s = load_seq(a.kv, w->seq);
  w->s.row0 = __builtin_amdgcn_readfirstlane(w->s.row0);
  w->s.rows = __builtin_amdgcn_readfirstlane(w->s.rows);
  w->s.len = __builtin_amdgcn_readfirstlane(w->s.len);
  w->s.start = __builtin_amdgcn_readfirstlane(w->s.start);
  return true;
}

// ---------------------------------------------------------------- results
// Four dims of a finished column: row0 + j, head; v already divided.
template <bool F32>
__device__ __forceinline__ void store_out(const AttendArgs &a, int row, int head, int D, int d, f32x4 v) {
  if constexpr (F32)
    *(float4 *)((float *)a.out + (size_t)row * a.out_stride + head * D + d) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *(uint2 *)((u16 *)a.out + (size_t)row * a.out_stride + head * D + d) =
        make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}
__device__ __forceinline__ void store_lse(const AttendArgs &a, int row, int head, float M, float l) {
  // a column that saw nothing has M = -inf and l = 0
  if (a.lse) a.lse[(size_t)row * a.heads + head] = M == -INFINITY ? -INFINITY : 0.6931471805599453f * (M + __builtin_amdgcn_logf(l));
}
// A row that sees nothing is zero; a NaN denominator stays one.
__device__ __forceinline__ float denominator(float l) { return l == 0.f ? 0.f : 1.f / l; }

// A partial result's place: [CB][D] sums, then M and l per column.
template <int D, int CB>
struct Slot {
  static constexpr int kFloats = CB * (D + 2);
  float *p;
  __device__ Slot(const AttendArgs &a, int i) : p(a.part + (size_t)i * kFloats) {}
  __device__ __amdgpu_buffer_rsrc_t sums() const { return coherent_rsrc(p, CB * D * 4); }
  __device__ void put_ml(int col, float M, float l) const {
    __hip_atomic_store(p + CB * D + col, M, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(p + CB * D + CB + col, l, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
};

// Joins the partials of slots slot0, slot0 + step, ... (count of them, at
// most kMaxGroup), all columns below ncols: into slot0 again, or, `last`,
// into the output.  Called by the whole workgroup; every partial is complete.
template <int D, int CB, bool F32>
__device__ __forceinline__ void join(const AttendArgs &a, const Work &w, int h, int slot0, int step, int count, int ncols,
                                     bool last, float *lds) {
  float *lm = lds, *ll = lds + kMaxGroup * CB;
  __syncthreads();
  for (int i = threadIdx.x; i < count * ncols; i += 256) {
    const int k = i / ncols, col = i - k * ncols;
    const Slot<D, CB> s(a, slot0 + k * step);
    lm[k * CB + col] = __hip_atomic_load(s.p + CB * D + col, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    ll[k * CB + col] = __hip_atomic_load(s.p + CB * D + CB + col, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < ncols * (D / 4); i += 256) {
    const int col = i / (D / 4), d = (i % (D / 4)) * 4;
    float M = -INFINITY, l = 0.f;
    for (int k = 0; k < count; ++k) M = fmaxf(M, lm[k * CB + col]);
    const float base = M == -INFINITY ? 0.f : M;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    for (int k0 = 0; k0 < count; k0 += 8) {
      f32x4 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)  // past the end: the last again, with no weight
        v[k] = ld16_coherent(Slot<D, CB>(a, slot0 + min(k0 + k, count - 1) * step).sums(), (uint32_t)(col * D + d) * 4, 0);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k0 + k >= count) break;
        const float f = __builtin_amdgcn_exp2f(lm[(k0 + k) * CB + col] - base);
        l += f * ll[(k0 + k) * CB + col];
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += f * v[k][e];
      }
    }
    if (last) {
      const int c = w.block * CB + col, row = w.s.row0 + c / a.G, head = h * a.G + c % a.G;
      const float r = denominator(l);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] *= r;
      store_out<F32>(a, row, head, D, d, sum);
      if (d == 0) store_lse(a, row, head, M, l);
    } else {
      // every thread reads and writes its own elements of slot0; M and l are in LDS
      const Slot<D, CB> s(a, slot0);
      st16_coherent(s.sums(), (uint32_t)(col * D + d) * 4, 0, sum);
      if (d == 0) s.put_ml(col, M, l);
    }
  }
}

// One arrival at counter `c` of `of`: whether it is the last, which leaves
// the counter at zero.  The workgroup's stores are complete before it counts.
__device__ __forceinline__ bool arrive(unsigned *c, unsigned of, unsigned *lds) {
  wait_vmcnt<0>();
  asm volatile("" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0) {
    const unsigned got = __hip_atomic_fetch_add(c, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (got == of - 1) __hip_atomic_store(c, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *lds = got;
  }
  __syncthreads();
  const bool last = *lds == of - 1;
  __syncthreads();
  return last;
}

// ---------------------------------------------------------------- kernel
template <int D, int NB, bool F32, bool WIDE>
__global__ __launch_bounds__(256) void attend_kernel(AttendArgs a) {
  constexpr int CW = 16 * NB;             // columns of a wave
  constexpr int CB = WIDE ? 4 * CW : CW;  // columns of a unit
  constexpr int NI = D / 64, NS = D / 32, ND = D / 16, NT = F32 ? 3 : 1;
  constexpr int kMergeBytes = WIDE ? 0 : 4 * ND * 64 * 16, kJoinBytes = kMaxGroup * CB * 8;
  __shared__ __attribute__((aligned(16))) char smem[kMergeBytes > kJoinBytes ? kMergeBytes : kJoinBytes];
  __shared__ float wave_ml[4][2][CW];
  __shared__ unsigned arrived;

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = blockIdx.x % a.kv.H;
  Work w;
  if (!find_work<CB>(a, blockIdx.x / a.kv.H, lane, &w)) return;
  const int cap = kv_cap(a.kv), n_cols = min(CB, w.s.rows * a.G - w.block * CB);
  const int r = lane & 15, g = lane >> 4;

  // the tokens that the unit's columns see, [lo_u, hi_u), and this chunk's tiles of them
  const int j_first = (w.block * CB) / a.G, j_last = (w.block * CB + n_cols - 1) / a.G;
  const int hi_u = max(min(w.s.start + j_last + 1, cap), 0);
  const int lo_u = a.window ? max(w.s.start + j_first + 1 - a.window, 0) : 0;
  const int tile0 = lo_u / kTile, tiles = hi_u > lo_u ? (hi_u + kTile - 1) / kTile - tile0 : 0;
  int ta = tile0 + (int)((long long)tiles * w.chunk / w.nc);
  int tb = tile0 + (int)((long long)tiles * (w.chunk + 1) / w.nc);

  // this wave's columns, and the tokens that all of them see
  const int c0 = w.block * CB + (WIDE ? wave * CW : 0);
  const int c1 = min(c0 + CW, w.s.rows * a.G);
  int j0 = j_first, j1 = j_last;
  if constexpr (WIDE) {
    j0 = c0 / a.G;
    j1 = (c1 - 1) / a.G;
    if (c0 < c1) {
      tb = min(tb, (max(min(w.s.start + j1 + 1, cap), 0) + kTile - 1) / kTile);
      if (a.window) ta = max(ta, max(w.s.start + j0 + 1 - a.window, 0) / kTile);
    } else {
      tb = ta;
    }
  } else {
    ta += wave;
  }
  constexpr int step = WIDE ? 1 : 4;
  const int hi_all = w.s.start + j0 + 1, lo_all = a.window ? w.s.start + j1 + 1 - a.window : 0;

  int hi_c[NB], lo_c[NB];
  uint4 q[NB][NS][NT];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int c = c0 + nb * 16 + r;
    const bool ok = c < c1;
    const int j = ok ? c / a.G : 0;
    hi_c[nb] = ok ? w.s.start + j + 1 : 0;
    lo_c[nb] = ok && a.window ? w.s.start + j + 1 - a.window : 0;
    const size_t at = (size_t)(w.s.row0 + j) * a.q_stride + (h * a.G + (ok ? c - j * a.G : 0)) * D;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int d = 16 * (4 * (s >> 1) + g) + 8 * (s & 1);
      if constexpr (F32) {
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (ok) {
          const uint4 u = ldg16((const float *)a.q + at + d), v = ldg16((const float *)a.q + at + d + 4);
          x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y); x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
          x[4] = __uint_as_float(v.x); x[5] = __uint_as_float(v.y); x[6] = __uint_as_float(v.z); x[7] = __uint_as_float(v.w);
        }
        split3(x, q[nb][s]);
      } else {
        q[nb][s][0] = ok ? ldg16((const u16 *)a.q + at + d) : z4();
      }
    }
  }

  f32x4 acc[NB][ND];
  float M[NB], l[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    M[nb] = -INFINITY;
    l[nb] = 0.f;
#pragma unroll
    for (int dt = 0; dt < ND; ++dt) acc[nb][dt] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // Pages of the wave's next 16 tiles, lane 4 i + k for 16-token group k of
  // tile i: the group's index among all groups of the pool, and the page's
  // exponent bytes, with bit 16 where there is a page.
  int gidx = 0, ex = 0;
  auto load_info = [&](int tile) {
    const int t = tile + (lane >> 2) * step, tok = t * kTile + 16 * (lane & 3);
    gidx = 0;
    ex = 127 | 127 << 8;
    if (t < tb && tok < cap) {
      const int page = page_of(a.kv, w.seq, tok >> a.kv.page_shift);
      if (page >= 0) {
        const size_t ph = (size_t)page * a.kv.H + h;
        ex = max((int)a.kv.ke[ph], 1) | (a.kv.ve[ph] << 8) | 0x10000;
        gidx = (int)((ph << (a.kv.page_shift - 4)) + ((tok & ((1 << a.kv.page_shift) - 1)) >> 4));
      }
    }
  };
  uint4 kr[4][NI], vr[ND];
  auto load_k = [&](int i) {
    const uint8_t *p = a.kv.k + (size_t)(unsigned)__shfl(gidx, 4 * i + (r >> 2), 64) * (16 * D) + g * 64 + (r & 3) * 16;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int n = 0; n < NI; ++n) kr[j][n] = ldg16(p + j * (4 * D) + n * 256);
  };
  auto load_v = [&](int i) {
    const uint8_t *p = a.kv.v + (size_t)(unsigned)__shfl(gidx, 4 * i + g, 64) * (16 * D) + r * 16;
#pragma unroll
    for (int dt = 0; dt < ND; ++dt) vr[dt] = ldg16(p + dt * 256);
  };

  int bi = 0;  // the tile's place among the 16 whose pages are known
  if (ta < tb) {
    load_info(ta);
    load_k(0);
    load_v(0);
  }
  for (int t = ta; t < tb; t += step) {
    const int my_ex = __shfl(ex, 4 * bi + g, 64);
    // scores: lane (column r, g) gets tokens 16 g + 4 j + i of the tile
    f32x4 S[NB][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) S[nb][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const uint4 &x = kr[j][s >> 1];
        const uint4 kf = s & 1 ? codes_bf16(x.z, x.w) : codes_bf16(x.x, x.y);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int n = 0; n < NT; ++n) S[nb][j] = mfma16(kf, q[nb][s][NT - 1 - n], S[nb][j]);
      }
    }
    const bool more = t + step < tb;
    if (more) {
      if (++bi == 16) {
        load_info(t + step);
        bi = 0;
      }
      load_k(bi);
    }

    const int tok0 = t * kTile + 16 * g;
    const bool masked = t * kTile < lo_all || (t + 1) * kTile > min(hi_all, cap) || __any(!(my_ex >> 16));
    bool poison = false;  // a NaN value that some of the columns do not see
    if (masked) {
      const bool page = my_ex >> 16;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tok = tok0 + 4 * j + i;
            if (!page || tok >= hi_c[nb] || tok < lo_c[nb]) S[nb][j][i] = -INFINITY;
          }
    }
    const float ve = (float)(((my_ex >> 8) & 255) - 127);
    const float cs = a.scale * __uint_as_float((uint32_t)(my_ex & 255) << 23);
    const float inv = __uint_as_float((uint32_t)(254 - min((my_ex >> 8) & 255, 253)) << 23);
    uint4 pf[NB][2][NT];
    float alpha[NB];
    bool grew = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float mx = S[nb][0][0];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = fmaxf(mx, S[nb][j][i]);
      const float top = groups_max(fmaf(mx, cs, ve));
      const float Mn = fmaxf(M[nb], top);
      const float base = Mn == -INFINITY ? 0.f : Mn;
      alpha[nb] = __builtin_amdgcn_exp2f(M[nb] - base);
      grew |= Mn > M[nb];
      M[nb] = Mn;
      const float b = ve - base;
      float sum = 0.f;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          p[e] = __builtin_amdgcn_exp2f(fmaf(S[nb][2 * s + (e >> 2)][e & 3], cs, b));
          sum += p[e];
        }
        if constexpr (F32) split3(p, pf[nb][s]);
        else pf[nb][s][0] = make_uint4(pack_f16(p[0], p[1]), pack_f16(p[2], p[3]), pack_f16(p[4], p[5]), pack_f16(p[6], p[7]));
      }
      l[nb] = l[nb] * alpha[nb] + sum * inv;
    }
    if (__any(grew)) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int dt = 0; dt < ND; ++dt)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[nb][dt][e] *= alpha[nb];
    }
    if (masked) {
      // tokens that no column sees may hold anything: their bytes become
      // zeros, and so do NaN codes, which would reach the columns that do
      // not see them too
      const bool page = my_ex >> 16;
      uint32_t keep[4], any_nan = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) keep[i] = page ? live_bytes(tok0 + 4 * i, lo_u, hi_u) : 0u;
#pragma unroll
      for (int dt = 0; dt < ND; ++dt) {
        vr[dt].x &= keep[0];
        vr[dt].y &= keep[1];
        vr[dt].z &= keep[2];
        vr[dt].w &= keep[3];
        any_nan |= nan_bytes(vr[dt].x) | nan_bytes(vr[dt].y) | nan_bytes(vr[dt].z) | nan_bytes(vr[dt].w);
      }
      poison = __any(any_nan != 0);
    }
    if (poison) {
      // columns that see a NaN value: count them by a product of ones
      uint4 see[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int t0 = tok0 + 8 * s + 2 * e;
            o[e] = (t0 < hi_c[nb] && t0 >= lo_c[nb] ? 0x3c00u : 0u) |
                   (t0 + 1 < hi_c[nb] && t0 + 1 >= lo_c[nb] ? 0x3c000000u : 0u);
          }
          see[nb][s] = make_uint4(o[0], o[1], o[2], o[3]);
        }
#pragma unroll
      for (int dt = 0; dt < ND; ++dt) {
        const uint4 x = vr[dt];
        const uint4 nan = make_uint4(nan_bytes(x.x), nan_bytes(x.y), nan_bytes(x.z), nan_bytes(x.w));
        vr[dt] = make_uint4(x.x & ~nan.x, x.y & ~nan.y, x.z & ~nan.z, x.w & ~nan.w);
        // 0x38 is 1.0 in e4m3
        const uint4 lo = codes_f16(nan.x & 0x38383838u, nan.y & 0x38383838u);
        const uint4 hi = codes_f16(nan.z & 0x38383838u, nan.w & 0x38383838u);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          f32x4 n = mfma16_f16(lo, see[nb][0], f32x4{0.f, 0.f, 0.f, 0.f});
          n = mfma16_f16(hi, see[nb][1], n);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n[e] > 0.f) acc[nb][dt][e] = __uint_as_float(0x7fc00000u);
        }
      }
    }
#pragma unroll
    for (int dt = 0; dt < ND; ++dt) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t lo = s ? vr[dt].z : vr[dt].x, hi = s ? vr[dt].w : vr[dt].y;
        if constexpr (F32) {
          const uint4 vf = codes_bf16(lo, hi);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int n = 0; n < 3; ++n) acc[nb][dt] = mfma16(vf, pf[nb][s][2 - n], acc[nb][dt]);
        } else {
          const uint4 vf = codes_f16(lo, hi);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) acc[nb][dt] = mfma16_f16(vf, pf[nb][s][0], acc[nb][dt]);
        }
      }
    }
    if (more) load_v(bi);
  }
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) l[nb] = groups_sum(l[nb]);

  const bool split = w.nc > 1;
  const Slot<D, CB> slot(a, split ? (w.slot + w.chunk) * a.kv.H + h : 0);
  if constexpr (WIDE) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int c = c0 + nb * 16 + r, col = c - w.block * CB;
      if (c >= c1) continue;
      const int row = w.s.row0 + c / a.G, head = h * a.G + c % a.G;
      const float rl = denominator(l[nb]);
#pragma unroll
      for (int dt = 0; dt < ND; ++dt) {
        f32x4 v = acc[nb][dt];
        if (split) {
          st16_coherent(slot.sums(), (uint32_t)(col * D + 16 * dt + 4 * g) * 4, 0, v);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] *= rl;
          store_out<F32>(a, row, head, D, 16 * dt + 4 * g, v);
        }
      }
      if (g == 0) {
        if (split) slot.put_ml(col, M[nb], l[nb]);
        else store_lse(a, row, head, M[nb], l[nb]);
      }
    }
  } else {
    // the four waves' sums, each scaled to the common maximum, through LDS
    if (g == 0) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        wave_ml[wave][0][nb * 16 + r] = M[nb];
        wave_ml[wave][1][nb * 16 + r] = l[nb];
      }
    }
    __syncthreads();
    f32x4 *box = (f32x4 *)smem;  // [wave][dt][lane]
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float Mx = -INFINITY;
#pragma unroll
      for (int k = 0; k < 4; ++k) Mx = fmaxf(Mx, wave_ml[k][0][nb * 16 + r]);
      const float base = Mx == -INFINITY ? 0.f : Mx;
      float lx = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) lx += wave_ml[k][1][nb * 16 + r] * __builtin_amdgcn_exp2f(wave_ml[k][0][nb * 16 + r] - base);
      const float f = __builtin_amdgcn_exp2f(M[nb] - base);
#pragma unroll
      for (int dt = 0; dt < ND; ++dt) {
        f32x4 v = acc[nb][dt];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] *= f;
        box[(wave * ND + dt) * 64 + lane] = v;
      }
      __syncthreads();
      const int c = c0 + nb * 16 + r, col = c - w.block * CB;
      if (c < c1) {
        const int row = w.s.row0 + c / a.G, head = h * a.G + c % a.G;
        const float rl = denominator(lx);
#pragma unroll
        for (int k = 0; k < ND / 4; ++k) {
          const int dt = wave * (ND / 4) + k;
          f32x4 v = box[dt * 64 + lane];
#pragma unroll
          for (int o = 1; o < 4; ++o) {
            const f32x4 u = box[(o * ND + dt) * 64 + lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += u[e];
          }
          if (split) {
            st16_coherent(slot.sums(), (uint32_t)(col * D + 16 * dt + 4 * g) * 4, 0, v);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] *= rl;
            store_out<F32>(a, row, head, D, 16 * dt + 4 * g, v);
          }
        }
        if (wave == 0 && g == 0) {
          if (split) slot.put_ml(col, Mx, lx);
          else store_lse(a, row, head, Mx, lx);
        }
      }
      if (nb + 1 < NB) __syncthreads();
    }
  }
  if (!split) return;

  // groups of gs chunks, then the unit's groups
  int gs = 1;
  while (gs * gs < w.nc) ++gs;
  const int H = a.kv.H, groups = (w.nc + gs - 1) / gs, gi = w.chunk / gs;
  const int in_group = min(gs, w.nc - gi * gs), slot_g = (w.slot + gi * gs) * H + h;
  if (!arrive(a.cnt + slot_g, in_group, &arrived)) return;
  join<D, CB, F32>(a, w, h, slot_g, H, in_group, n_cols, groups == 1, (float *)smem);
  if (groups == 1) return;
  if (!arrive(a.cnt + kAttendSlots + w.slot * H + h, groups, &arrived)) return;
  join<D, CB, F32>(a, w, h, w.slot * H + h, gs * H, groups, n_cols, true, (float *)smem);
}

// ---------------------------------------------------------------- launcher
template <int D, int NB, bool F32, bool WIDE>
static void go(const AttendArgs &a, hipStream_t st) {
  constexpr int CB = (WIDE ? 64 : 16) * NB;
  const int s = a.kv.n < a.kv.n_seqs ? a.kv.n : a.kv.n_seqs;
  const long long blocks = s + ((long long)a.kv.n * a.G - s) / CB;  // sum of ceil(cols / CB) over s sequences at most
  hipLaunchKernelGGL((attend_kernel<D, NB, F32, WIDE>), dim3((unsigned)((a.per_head + blocks) * a.kv.H)), dim3(256), 0, st, a);
}
// Column blocks of a wave that its registers hold (accumulators 4 D / 16 and
// the tile's codes D / 2 of them), at most.
template <int D>
static hipError_t go_dim(const AttendArgs &a, int dtype, int nb, bool wide, hipStream_t st) {
  if (dtype == 0) go<D, 1, true, false>(a, st);
  else if (wide) go<D, attend_wide_nb(D), false, true>(a, st);
  else if (nb == 1 || D > 128) go<D, 1, false, false>(a, st);
  else if constexpr (D <= 128) {
    if (nb == 2) go<D, 2, false, false>(a, st);
    else go<D, 3, false, false>(a, st);
  }
  return hipGetLastError();
}

hipError_t launch_attend(const AttendArgs &a, int dim, int dtype, int nb, bool wide, hipStream_t st) {
  return dim == 64 ? go_dim<64>(a, dtype, nb, wide, st)
         : dim == 128 ? go_dim<128>(a, dtype, nb, wide, st) : go_dim<256>(a, dtype, nb, wide, st);
}

}  // namespace lora
