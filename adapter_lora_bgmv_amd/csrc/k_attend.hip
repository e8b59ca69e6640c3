// k_attend.hip -- attention of ragged query rows over the 8-bit paged cache.
//
// For a sequence with rows j = 0 .. m-1 at positions start + j, query head h
// and key/value head h / G:
//     o_j = sum_t w_jt v_t / sum_t w_jt,  w_jt = exp(scale q_j . k_t),
// over the tokens t <= start + j (and t > start + j - window), k_t = 2^a c_t
// and v_t = 2^b d_t with the page's exponents a, b and e4m3 codes c, d.
//
// The codes go into the matrix instructions as they are: e4m3 numbers are
// exact in bf16 and in f16, and the instruction that converts two of them
// multiplies by a power of two as well, so the pages' scales cost nothing.
// Keys become bf16, 2^a c, whose range holds every exponent.  Values of bf16
// calls become f16, 2^b d: exact for b within [-21, 0] (pages whose largest
// value lies between 1e-4 and 448), which is what models hold.  The weights
// of other pages take the rest of the exponent, 2^rest p, and then two
// maxima run, of the exponents with and without the rest, so that neither
// the sums against v nor the denominators lose anything (`mixed`).
//
// A column is a (row, query head of the group) pair; a wave holds 16 NB
// columns and walks tiles of 64 tokens.  K's tile is the A operand (64
// tokens x D), the columns the B operand, and the order of tokens within the
// tile is chosen so that lane (column, g) ends up with the scores of the 16
// tokens of 16-token group g: those are the B operand of the second product
// as they stand, V's 16 bytes of a dim the A operand, and a lane's 16 tokens
// share one page, one a and one b.  The running maximum M is allowed to lag
// the true one by 2^kLag: only a tile that exceeds it looks across lanes and
// rescales the sums, which after a few tiles is rare.
//
// Rounding: bf16 calls take q as it is and round the weights, 2^8 at the
// running maximum, to f16 (2^-11, an eighth of the output's own half step, for
// weights down to 2^-22 of the largest; steps of 2^-32 of it below, which show
// only where every larger weight meets a zero); f32 calls split q and the
// weights into three bf16 terms (24 bits) and take three products of each.
// Scores, sums and outputs accumulate in f32.
//
// Two forms share the code.  Narrow (up to 16 columns a sequence: decode):
// each wave of a workgroup takes every fourth tile straight into registers,
// and the four are joined through LDS; a decode batch is bound by HBM (64 rows
// over 1 to 8192 tokens: 111 us, 4.8 TB/s), one row by latency (701 tokens:
// 7.8 us, 1.5 more where a wider page table adds the join).  Wide (more columns): the waves take 16 NB columns each and share
// the tiles, which LDS-DMA brings in two or three ahead.  With two blocks a
// wave it is bound by issue: 62 products and 313 other vector instructions a
// tile (1024 rows over 16 000 tokens: 914 TFLOP/s, matrix unit busy 36 %).
// Two blocks instead of one halve the conversions a product; three do not fit
// the registers of two waves a SIMD.
//
// The call's tiles are shared out in chunks of equal length over about one
// round of workgroups, from the lengths in device memory, so long and short
// sequences balance; a unit (sequence, head, columns) of several chunks leaves
// its sums in the workspace, and a second kernel joins them (5 us; the last
// workgroup to arrive took 20 us for 16 chunks of 36 columns, alone).
//
// What is rare (masks, missing pages, maxima that moved, NaN codes, rests) is
// kept out of the main loop, and in the wide form takes one block after the
// other: inside, it costs copies of all sums and spills, 15 % and more.
#include <algorithm>

#include "attend.hpp"
#include "common.hpp"
#include "verify.hpp"

namespace lora {

// ---------------------------------------------------------------- pages
// Pages of 16 tiles, lane 4 i + k for 16-token group k of tile i (`step`
// tiles after the one before): the group's index among all groups of the
// pool, and the page's exponent bytes (those of group 0 where there is no
// page, which nothing is made of).
struct PageInfo {
  int group, ke, ve;
  unsigned long long there;  // a bit a lane: it has a page
  // The lane's page of the tiles from `tile` to `end`, or -1; then what is known of it.
  static __device__ __forceinline__ int page(const KvDev &kv, int seq, int tile, int step, int end, int lane) {
    const int t = tile + (lane >> 2) * step, tok = (int)((unsigned)t * kTile) + 16 * (lane & 3);
    return t < end && tok < kv_cap(kv) ? page_of(kv, seq, tok >> kv.page_shift) : -1;
  }
  __device__ __forceinline__ void set(const KvDev &kv, int h, int page, int tile, int step, int lane) {
    const int tok = (int)((unsigned)(tile + (lane >> 2) * step) * kTile) + 16 * (lane & 3);
    const size_t ph = page >= 0 ? (size_t)page * kv.H + h : 0;
    ke = kv.ke[ph];
    ve = kv.ve[ph];
    group = page >= 0 ? (int)((ph << (kv.page_shift - 4)) + ((tok & ((1 << kv.page_shift) - 1)) >> 4)) : 0;
    there = __ballot(page >= 0);
  }
  __device__ __forceinline__ void load(const KvDev &kv, int seq, int h, int tile, int step, int end, int lane) {
    set(kv, h, page(kv, seq, tile, step, end, lane), tile, step, lane);
  }
  // Whether tile i has all its pages and lies within the tokens that every column sees.
  __device__ __forceinline__ bool whole(int i, int tile, int lo_all, int hi_all) const {
    return (there >> (4 * i) & 15) == 15 && tile * kTile >= lo_all && (tile + 1) * kTile <= hi_all;
  }
  // Tile i's exponent bytes: of the keys' group that the lane loads (r / 4),
  // of the values of group g, and whether group g has a page.
  struct Tile {
    int ke, ve;
    bool page;
  };
  __device__ __forceinline__ Tile tile(int i, int r, int g) const {
    return {__shfl(ke, 4 * i + (r >> 2), 64), __shfl(ve, 4 * i + g, 64), (bool)(there >> (4 * i + g) & 1)};
  }
};

// ---------------------------------------------------------------- a wave's columns
template <int D, int NB, bool F32>
struct Columns {
  static_assert(NB <= 2, "the masked form takes one or two blocks");
  static constexpr int NS = D / 32, ND = D / 16, NT = F32 ? 3 : 1;
  uint4 q[NB][NS][NT];
  f32x4 acc[NB][ND];
  // sums run against 2^(M - kTop), the denominators l against 2^(Ml - kTop); Ml is M unless `mixed`
  float M[NB], Ml[NB], l[NB];
  int hi[NB];  // a column sees the tokens [hi - window, hi), or [0, hi)
  bool mixed;

  // Columns [c0, c1) of the sequence.
  __device__ __forceinline__ void load(const AttendArgs &a, const Work &w, int h, int c0, int c1, int r, int g) {
    mixed = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int c = c0 + nb * 16 + r;
      const bool ok = c < c1;
      const int j = ok ? a.G.div(c) : 0;
      hi[nb] = ok ? w.s.start + j + 1 : 0;
      const size_t at = (size_t)(w.s.row0 + j) * a.q_stride + (h * a.G.d + (ok ? c - j * a.G.d : 0)) * D;
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
      M[nb] = Ml[nb] = kNone;
      l[nb] = 0.f;
#pragma unroll
      for (int dt = 0; dt < ND; ++dt) acc[nb][dt] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }

  static __device__ __forceinline__ uint32_t &word(uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

  // The largest of the lane's scores of a column.
  __device__ __forceinline__ static float largest(const f32x4 (&S)[4]) {
    float mx = S[0][0];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) mx = fmaxf(mx, S[j][e]);
    return mx;
  }

  // The weights p = 2^(S cs + b) of a column's scores as operands, and their sum.
  __device__ __forceinline__ static float weigh(const f32x4 (&S)[4], float cs, float b, uint4 (&pf)[2][NT]) {
    float sum = 0.f;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        p[e] = __builtin_amdgcn_exp2f(fmaf(S[2 * s + (e >> 2)][e & 3], cs, b));
        sum += p[e];
      }
      if constexpr (F32) split3(p, pf[s]);
      else pf[s][0] = make_uint4(pack_f16(p[0], p[1]), pack_f16(p[2], p[3]), pack_f16(p[4], p[5]), pack_f16(p[6], p[7]));
    }
    return sum;
  }

  // sums of those blocks += weights x sixteen dims' codes of the tile
  template <int B0, int BN>
  __device__ __forceinline__ void add(int dt, const uint4 &x, float scale, const uint4 (&pf)[BN][2][NT]) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t lo = s ? x.z : x.x, hi = s ? x.w : x.y;
      if constexpr (F32) {
        const uint4 vf = codes_bf16(lo, hi, scale);
#pragma unroll
        for (int i = 0; i < BN; ++i)
#pragma unroll
          for (int n = 0; n < 3; ++n) acc[B0 + i][dt] = mfma16(vf, pf[i][s][2 - n], acc[B0 + i][dt]);
      } else {
        const uint4 vf = codes_f16(lo, hi, scale);
#pragma unroll
        for (int i = 0; i < BN; ++i) acc[B0 + i][dt] = mfma16_f16(vf, pf[i][s][0], acc[B0 + i][dt]);
      }
    }
  }

  // Scores of the column blocks [B0, B0 + BN): lane (column r, g) gets tokens
  // 16 g + 4 j + i of the tile; kf(j, n) gives 16 bytes of keys.
  template <int B0, int BN, typename K>
  __device__ __forceinline__ void score(f32x4 (&S)[BN][4], float scale, K kf) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int i = 0; i < BN; ++i) S[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int n = 0; n < D / 64; ++n) {
        const uint4 x = kf(j, n);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const uint4 kk = s ? codes_bf16(x.z, x.w, scale) : codes_bf16(x.x, x.y, scale);
#pragma unroll
          for (int i = 0; i < BN; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t) S[i][j] = mfma16(kk, q[B0 + i][2 * n + s][NT - 1 - t], S[i][j]);
        }
      }
    }
  }

  // The rest of a tile that every column sees all of, from its scores and
  // values vf(dt); false, and nothing changed, where something unusual sends
  // it through `careful`.  AHEAD: the next tile's scores, from its keys
  // kf(j, n) under `scale`, take the place of S.  In one wave the matrix
  // products hide the conversions and exponentials between them, so those
  // scores are computed among this tile's weights and the order is asked for:
  // one product, then its share of the rest.
  template <bool AHEAD, typename V, typename K>
  __device__ __forceinline__ bool plain(f32x4 (&S)[NB][4], PageInfo::Tile info, float cs, V vf, float scale, K kf) {
    using X = ValueExp<F32>;
    if (__builtin_expect(mixed || __any(info.ve < X::kLo || info.ve > X::kHi), 0)) return false;
    float top[NB];
    bool far = false, old = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      top[nb] = largest(S[nb]) * cs;
      far |= top[nb] > M[nb] + kLag;
      old |= top[nb] > M[nb] + kLag && M[nb] != kNone;
    }
    if (__builtin_expect(__any(far), 0)) {
      if (__any(old)) return false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) M[nb] = M[nb] == kNone ? fmaxf(kNone, groups_max(top[nb])) : M[nb];  // the first: nothing to rescale
    }
    const float vs = scale_of(info.ve + X::kAdd);
    uint4 pf[NB][2][NT];
    if constexpr (!AHEAD) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) l[nb] += weigh(S[nb], cs, kTop - M[nb], pf[nb]);
      uint4 next = vf(0);
#pragma unroll
      for (int dt = 0; dt < ND; ++dt) {
        const uint4 now = next;
        if (dt + 1 < ND) next = vf(dt + 1);
        add<0, NB>(dt, now, vs, pf);
      }
    } else {
      // step k: a 32-dim half of a key fragment against every column block,
      // with kEach weights of each block and the conversion of the next half
      constexpr int kFrags = 4 * (D / 64), kSteps = 2 * kFrags, kEach = 16 / kSteps;
      uint4 x[3] = {kf(0, 0), kf(1 / (D / 64), 1 % (D / 64)), z4()};
      f32x4 T[NB][4];
      float f[NB], p[NB][16], b[NB];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        b[nb] = kTop - M[nb];
        f[nb] = fmaf(S[nb][0][0], cs, b[nb]);
#pragma unroll
        for (int j = 0; j < 4; ++j) T[nb][j] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      uint4 cur = codes_bf16(x[0].x, x[0].y, scale);
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const int m = k / 2, j = m / (D / 64), n = m % (D / 64);
        if (k % 2 == 0) {  // two fragments ahead; the values follow the keys
          if (m + 2 < kFrags) x[(m + 2) % 3] = kf((m + 2) / (D / 64), (m + 2) % (D / 64));
          else x[(m + 2) % 3] = vf(m + 2 - kFrags);
        }
        const uint4 &y = x[((k + 1) / 2) % 3];
        uint4 after = z4();
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          __builtin_amdgcn_sched_barrier(0);
          T[nb][j] = mfma16(cur, q[nb][2 * n + k % 2][0], T[nb][j]);
          if (nb == 0) {
            const uint32_t w = k % 2 ? y.x : y.z;
            const uint2 c = k + 1 < kSteps ? pair_bf16(w, scale) : pair_f16(w, vs);
            after.x = c.x;
            after.y = c.y;
          }
          if (nb == NB - 1) {
            const uint32_t w = k % 2 ? y.y : y.w;
            const uint2 c = k + 1 < kSteps ? pair_bf16(w, scale) : pair_f16(w, vs);
            after.z = c.x;
            after.w = c.y;
          }
#pragma unroll
          for (int i = 0; i < kEach; ++i) {
            const int e = k * kEach + i;
            p[nb][e] = __builtin_amdgcn_exp2f(f[nb]);
            if (e + 1 < 16) f[nb] = fmaf(S[nb][(e + 1) >> 2][(e + 1) & 3], cs, b[nb]);
            if (e > 0) l[nb] += p[nb][e - 1];
            if (e >= 2 && e % 2 == 0) word(pf[nb][(e - 2) / 8][0], (e - 2) / 2 % 4) = pack_f16(p[nb][e - 2], p[nb][e - 1]);
          }
        }
        cur = after;
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        l[nb] += p[nb][15];
        pf[nb][1][0].w = pack_f16(p[nb][14], p[nb][15]);
#pragma unroll
        for (int j = 0; j < 4; ++j) S[nb][j] = T[nb][j];
      }
      // step k: half of sixteen dims' values against every block's weights
#pragma unroll
      for (int k = 0; k < 2 * ND; ++k) {
        const int dt = k / 2, m = kFrags + dt;
        if (k % 2 == 0 && dt + 2 < ND) x[(m + 2) % 3] = vf(dt + 2);
        const uint4 &y = x[(kFrags + (k + 1) / 2) % 3];
        uint4 after = z4();
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          __builtin_amdgcn_sched_barrier(0);
          acc[nb][dt] = mfma16_f16(cur, pf[nb][k % 2][0], acc[nb][dt]);
          if (k + 1 == 2 * ND) continue;
          if (nb == 0) {
            const uint2 c = pair_f16(k % 2 ? y.x : y.z, vs);
            after.x = c.x;
            after.y = c.y;
          }
          if (nb == NB - 1) {
            const uint2 c = pair_f16(k % 2 ? y.y : y.w, vs);
            after.z = c.x;
            after.w = c.y;
          }
        }
        cur = after;
      }
    }
    return true;
  }

  // The rest of any tile, from token tok0 of the lane, for column block B0:
  // masks, missing pages, value exponents out of the operand's range, maxima
  // that moved, NaN codes.  [lo_any, hi_any) are the tokens that any column
  // of the workgroup sees.
  template <int B0, typename V>
  __device__ __forceinline__ void careful(f32x4 (&S)[1][4], int tok0, PageInfo::Tile info, int window, float cs, int lo_any,
                                          int hi_any, V vf) {
    using X = ValueExp<F32>;
    const int vc = min(max(info.ve, X::kLo), X::kHi);
    const float rest = (float)(info.ve - vc), vs = scale_of(vc + X::kAdd);
    const uint32_t see = info.page ? sees(hi[B0], window, tok0) : 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t m = (uint32_t)((int32_t)(see << (31 - 4 * j - i)) >> 31);
        S[0][j][i] = __uint_as_float((__float_as_uint(S[0][j][i]) & m) | (0xff800000u & ~m));
      }
    const float topl = largest(S[0]) * cs, top = topl + rest;
    if (__any(top > M[B0] + kLag || topl > Ml[B0] + kLag)) {
      const float Mn = fmaxf(M[B0], groups_max(top)), Mln = fmaxf(Ml[B0], groups_max(topl));
      const float f = __builtin_amdgcn_exp2f(M[B0] - Mn);
      l[B0] *= __builtin_amdgcn_exp2f(Ml[B0] - Mln);
      M[B0] = Mn;
      Ml[B0] = Mln;
#pragma unroll
      for (int dt = 0; dt < ND; ++dt) acc[B0][dt] *= f;
    }
    uint4 pf[1][2][NT];
    const float sum = weigh(S[0], cs, kTop - M[B0] + rest, pf[0]);
    if (mixed) {
      const float bl = kTop - Ml[B0];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) l[B0] += __builtin_amdgcn_exp2f(fmaf(S[0][j][e], cs, bl));
    } else {
      l[B0] += sum;
    }
    // a NaN code, even where nothing is seen, would reach every column
    uint32_t any = 0;
#pragma unroll
    for (int dt = 0; dt < ND; ++dt) {
      const uint4 x = vf(dt);
      any |= has_nan(x.x) | has_nan(x.y) | has_nan(x.z) | has_nan(x.w);
    }
    asm volatile("" ::: "memory");  // read anew: held, the values would take the registers of the sums
    if (__builtin_expect(!__any((any & 0x80808080u) != 0), 1)) {
#pragma unroll
      for (int dt = 0; dt < ND; ++dt) add<B0, 1>(dt, vf(dt), vs, pf);
      return;
    }
    uint32_t keep[4];  // bytes of tokens that some column sees
#pragma unroll
    for (int i = 0; i < 4; ++i) keep[i] = info.page ? live_bytes(tok0 + 4 * i, lo_any, hi_any) : 0u;
#pragma unroll
    for (int dt = 0; dt < ND; ++dt) {
      uint4 x = vf(dt);
      x = make_uint4(x.x & keep[0], x.y & keep[1], x.z & keep[2], x.w & keep[3]);
      const uint4 nan = make_uint4(nan_bytes(x.x), nan_bytes(x.y), nan_bytes(x.z), nan_bytes(x.w));
      x = make_uint4(x.x & ~nan.x, x.y & ~nan.y, x.z & ~nan.z, x.w & ~nan.w);
      // columns that see a NaN value: count them by a product of ones (0x38 is 1.0 in e4m3, 0x3c00 in f16)
      f32x4 n = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t m = see >> (8 * s + 2 * e);
          o[e] = (m & 1 ? 0x3c00u : 0u) | (m & 2 ? 0x3c000000u : 0u);
        }
        n = mfma16_f16(codes_f16((s ? nan.z : nan.x) & 0x38383838u, (s ? nan.w : nan.y) & 0x38383838u, 1.f),
                       make_uint4(o[0], o[1], o[2], o[3]), n);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n[e] > 0.f) acc[B0][dt][e] = __uint_as_float(0x7fc00000u);
      add<B0, 1>(dt, x, vs, pf);
    }
  }
  // Before a careful tile: with no rest so far M and Ml move together.
  __device__ __forceinline__ void meet(PageInfo::Tile info) {
    if (mixed) return;
    mixed = __any(info.ve < ValueExp<F32>::kLo || info.ve > ValueExp<F32>::kHi);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) Ml[nb] = M[nb];
  }

  // q as operands in LDS, the lane's [NS][NT] in steps of 64, and the scores
  // from there: the 12 D / 32 registers of three terms are wanted for tiles on
  // their way (f32, 256 dims: without this the loop spills, and every reload
  // waits for those tiles).
  __device__ __forceinline__ void keep(uint4 *mine) const {
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int t = 0; t < NT; ++t) mine[(s * NT + t) * 64] = q[0][s][t];
  }
  template <typename K>
  static __device__ __forceinline__ void score_kept(f32x4 (&S)[1][4], float scale, const uint4 *mine, K kf) {
#pragma unroll
    for (int j = 0; j < 4; ++j) S[0][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      uint4 kk[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 x = kf(j, s / 2);
        kk[j] = s & 1 ? codes_bf16(x.z, x.w, scale) : codes_bf16(x.x, x.y, scale);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint4 y = mine[(s * NT + NT - 1 - t) * 64];
#pragma unroll
        for (int j = 0; j < 4; ++j) S[0][j] = mfma16(kk[j], y, S[0][j]);
      }
    }
  }

  // Waits for q here rather than at its first use, which is in the loop.
  __device__ __forceinline__ void arrive() {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          asm volatile("" : "+v"(q[nb][s][t].x), "+v"(q[nb][s][t].y), "+v"(q[nb][s][t].z), "+v"(q[nb][s][t].w));
  }

  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      l[nb] = groups_sum(l[nb]);
      if (!mixed) Ml[nb] = M[nb];
    }
  }
};

// ---------------------------------------------------------------- kernels
// LDS of the wide form: stages of a tile, each its 4 groups of K and 4 of V.
// A 16-byte read serves 16 lanes at a time, in sets that take two of the four
// token quads r / 4 from lanes g = 0 and the other two from g = 1 (and so for
// 2 and 3): free of conflicts where a lane's 64-byte place modulo 256 is its
// quad's alone.  V lies so by itself.  K's 64-byte units (quad j, chunk c) of
// group q are put at unit 4 c + (j + q) % 4: the DMA's lanes fetch them from
// where they are (conflicts 3.3 -> 0 cycles a read).
template <int D>
struct Stage {
  static constexpr int kPitch = 16 * D, kBytes = 8 * kPitch, kCount = D > 128 ? 2 : 4;
  static constexpr int kDma = 2 * (D / 64);  // instructions of a wave (its group's K and V) a stage
};

template <int D, int NB, bool F32, bool WIDE>
__global__ __launch_bounds__(256, attend_per_cu(D, F32, WIDE ? kWide : kNarrow)) void attend_kernel(AttendArgs a) {
  constexpr int CW = 16 * NB;             // columns of a wave
  constexpr int CB = WIDE ? 4 * CW : CW;  // columns of a unit
  constexpr int ND = D / 16;
  static_assert(WIDE || NB == 1, "the narrow form holds 16 columns");
  __shared__ __attribute__((aligned(16))) char smem[WIDE ? Stage<D>::kBytes * Stage<D>::kCount : 4 * ND * 64 * 16];
  __shared__ float wave_ml[WIDE ? 1 : 4][3][16];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int H = a.kv.H, item = a.H.div(blockIdx.x), h = blockIdx.x - item * H;
  Work w;
  int all_slots;
  const bool found = find_work<CB>(a, item, lane, &w, &all_slots);
  if (blockIdx.x == 0 && tid == 0) *a.used = all_slots * H;
  if (!found) return;
  const int cap = kv_cap(a.kv), n_cols = min(CB, w.s.rows * a.G.d - w.block * CB);
  const int r = lane & 15, g = lane >> 4;

  // the tokens that the unit's columns see, [lo_u, hi_u), and this chunk's tiles of them
  const int j_first = a.G.div(w.block * CB), j_last = a.G.div(w.block * CB + n_cols - 1);
  const int hi_u = max(min(w.s.start + j_last + 1, cap), 0);
  const int lo_u = first_seen(w.s.start + j_first + 1, a.window);
  const int tile0 = lo_u / kTile, tiles = hi_u > lo_u ? (hi_u + kTile - 1) / kTile - tile0 : 0;
  int ta = tile0, tb = tile0 + tiles;
  if (w.nc > 1) {  // the first tiles % nc chunks take one more
    const int each = tiles / w.nc, more = tiles - each * w.nc;
    ta += w.chunk * each + min(w.chunk, more);
    tb = ta + each + (w.chunk < more);
  }

  // this wave's columns, the tokens that all of them see and those that any does
  const int c0 = w.block * CB + (WIDE ? wave * CW : 0);
  const int c1 = min(c0 + CW, w.s.rows * a.G.d);
  const int j0 = WIDE ? a.G.div(c0) : j_first, j1 = WIDE ? a.G.div(max(c1 - 1, 0)) : j_last;
  const int hi_all = min(w.s.start + j0 + 1, cap), lo_all = first_seen(w.s.start + j1 + 1, a.window);
  Columns<D, NB, F32> cols;
  PageInfo info;

  if constexpr (!WIDE) {
    constexpr bool kKeep = F32 && D > 64;
    __shared__ uint4 kept[kKeep ? D / 32 * 3 * 64 : 1];  // the waves' columns are the same
    cols.load(a, w, h, c0, c1, r, g);
    if constexpr (kKeep) cols.keep(kept + lane);
    info.load(a.kv, w.seq, h, ta + wave, 4, tb, lane);
    uint4 kr[4][D / 64], vr[ND];
    auto load_k = [&](int i) {
      const uint8_t *p = a.kv.k + (size_t)(unsigned)__shfl(info.group, 4 * i + (r >> 2), 64) * (16 * D) + g * 64 + (r & 3) * 16;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int n = 0; n < D / 64; ++n) kr[j][n] = ldg16(p + j * (4 * D) + n * 256);
    };
    auto load_v = [&](int i) {
      const uint8_t *p = a.kv.v + (size_t)(unsigned)__shfl(info.group, 4 * i + g, 64) * (16 * D) + r * 16;
#pragma unroll
      for (int dt = 0; dt < ND; ++dt) vr[dt] = ldg16(p + dt * 256);
    };
    int i = 0;  // the tile's place among the 16 whose pages are known
    if (ta + wave < tb) {
      load_k(0);
      load_v(0);
    }
    for (int t = ta + wave; t < tb; t += 4) {
      auto kf = [&](int j, int n) { return kr[j][n]; };
      auto vf = [&](int dt) { return vr[dt]; };
      const PageInfo::Tile pages = info.tile(i, r, g);
      const bool whole = info.whole(i, t, lo_all, hi_all);
      f32x4 S[1][4];
      if constexpr (kKeep) cols.score_kept(S, scale_of(pages.ke), kept + lane, kf);
      else cols.template score<0, 1>(S, scale_of(pages.ke), kf);
      if (t + 4 < tb) {
        if (++i == 16) {
          info.load(a.kv, w.seq, h, t + 4, 4, tb, lane);
          i = 0;
        }
        load_k(i);
      }
      if (!whole || !cols.template plain<false>(S, pages, a.scale, vf, 0.f, kf)) {
        cols.meet(pages);
        cols.template careful<0>(S, t * kTile + 16 * g, pages, a.window, a.scale, lo_u, hi_u, vf);
      }
      if (t + 4 < tb) load_v(i);
    }
  } else {
    using St = Stage<D>;
    constexpr int N = St::kCount;
    constexpr bool kAhead = NB == 2;  // a tile's scores are computed during the one before
    const uint32_t base = lds_addr(smem);
    // wave k brings group k of the tile; lane l's unit is 4 c + l / 4 % 4 of 4 c .. 4 c + 3, c = 4 n + l / 16
    const int from_k = ((((lane >> 2) - wave) & 3) * (D / 16) + (lane >> 4)) * 64 + (lane & 3) * 16;
    auto bring = [&](int groups, int i, int stage) {
      const size_t at = (size_t)(unsigned)__builtin_amdgcn_readlane(groups, 4 * i + wave) * (16 * D);
      const uint32_t to = base + stage * St::kBytes + wave * St::kPitch;
#pragma unroll
      for (int n = 0; n < D / 64; ++n) dma16(a.kv.k + at + from_k + n * 256, to + n * 1024);
#pragma unroll
      for (int n = 0; n < D / 64; ++n) dma16(a.kv.v + at + lane * 16 + n * 1024, to + 4 * St::kPitch + n * 1024);
    };
    // the page table's round trip beside q's
    const int page = PageInfo::page(a.kv, w.seq, ta, 1, tb, lane);
    cols.load(a, w, h, c0, c1, r, g);
    cols.arrive();
    info.set(a.kv, h, page, ta, 1, lane);
#pragma unroll
    for (int k = 0; k < N - 1; ++k)
      if (ta + k < tb) bring(info.group, k, k);
    const int wave_lo = first_seen(w.s.start + j0 + 1, a.window);
    const int wave_hi = c0 < c1 ? min(w.s.start + j1 + 1, cap) : 0;
    PageInfo later = info;  // of the next 16 tiles
    int later_page = -1, i = 0, stage = 0;
    f32x4 S[NB][4];
    bool ahead = false;  // S holds the tile's scores

    for (int t = ta; t < tb; ++t) {
      // this wave's part of the tile (of the next one too, where its keys are
      // read) is here, then everybody's; nobody reads the tile before any more
      wait_stages<St::kDma, N - 2>(min(tb - 1 - t, N - 2) - kAhead);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      block_barrier();
      if (i == 16) {
        info = later;
        i = 0;
      }
      // what waits for the page table does so here, where only the next tile is in flight
      if (i == 4) later_page = PageInfo::page(a.kv, w.seq, t + 12, 1, tb, lane);
      if (i == 8) later.set(a.kv, h, later_page, t + 8, 1, lane);
      if (t + N - 1 < tb)
        bring(i + N - 1 < 16 ? info.group : later.group, (i + N - 1) & 15, stage == 0 ? N - 1 : stage - 1);
      if (t * kTile < wave_hi && (t + 1) * kTile > wave_lo) {
        // the lane's places anew: the registers that would hold them are wanted
        const int again = lane_again(), r = again & 15, g = again >> 4;
        const char *kp = smem + stage * St::kBytes + (r >> 2) * St::kPitch + g * 256 + (r & 3) * 16;
        const char *vp = smem + stage * St::kBytes + (4 + g) * St::kPitch + r * 16;
        auto kf = [&](int j, int n) { return *(const uint4 *)(kp + (((r >> 2) + j) & 3) * 64 + n * 1024); };
        auto vf = [&](int dt) { return *(const uint4 *)(vp + dt * 256); };
        const PageInfo::Tile pages = info.tile(i, r, g);
        bool done = info.whole(i, t, lo_all, hi_all);
        if (__builtin_expect(done, 1)) {
          if (!ahead) cols.template score<0, NB>(S, scale_of(pages.ke), kf);
          if (kAhead && t + 1 < tb) {
            const char *np = smem + (stage == N - 1 ? 0 : stage + 1) * St::kBytes + (kp - smem - stage * St::kBytes);
            auto nf = [&](int j, int n) { return *(const uint4 *)(np + (((r >> 2) + j) & 3) * 64 + n * 1024); };
            const int nk = __shfl(i == 15 ? later.ke : info.ke, 4 * ((i + 1) & 15) + (r >> 2), 64);
            done = cols.template plain<kAhead>(S, pages, a.scale, vf, scale_of(nk), nf);
            ahead = done;
          } else {
            done = cols.template plain<false>(S, pages, a.scale, vf, 0.f, kf);
          }
        }
        if (__builtin_expect(!done, 0)) {  // one block after the other, for the registers
          ahead = false;
          cols.meet(pages);
          f32x4 S[1][4];
          cols.template score<0, 1>(S, scale_of(pages.ke), kf);
          cols.template careful<0>(S, t * kTile + 16 * g, pages, a.window, a.scale, lo_u, hi_u, vf);
          if constexpr (NB == 2) {
            asm volatile("" ::: "memory");
            cols.template score<1, 1>(S, scale_of(pages.ke), kf);
            cols.template careful<1>(S, t * kTile + 16 * g, pages, a.window, a.scale, lo_u, hi_u, vf);
          }
        }
      }
      ++i;
      stage = stage == N - 1 ? 0 : stage + 1;
    }
  }
  cols.finish();

  const bool split = w.nc > 1;
  const int slot = split ? (w.slot + w.chunk) * H + h : 0;
  float *part = a.part + (size_t)slot * CB * (D + 3), *ml = part + CB * D;
  if (split && tid == 0) {
    const AttendRecord rec = {w.slot * H + h, H, w.nc, w.chunk, n_cols, w.s.row0, w.block * CB, h};
    a.records[slot] = rec;
  }
  // four dims of a column of the unit, from its sums or divided by them
  auto put = [&](int col, int d, f32x4 v, float M, float Ml, float l) {
    if (split) {
      *(float4 *)(part + col * D + d) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      const int c = w.block * CB + col, j = a.G.div(c), row = w.s.row0 + j, head = h * a.G.d + c - j * a.G.d;
      const float f = final_scale<F32>(M, Ml, l);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= f;
      store_out<F32>(a.out, (size_t)row * a.out_stride + head * D + d, v);
    }
  };
  auto put_ml = [&](int col, float M, float Ml, float l) {
    if (split) {
      ml[col] = M;
      ml[CB + col] = Ml;
      ml[2 * CB + col] = l;
    } else if (a.lse) {
      const int c = w.block * CB + col, j = a.G.div(c), row = w.s.row0 + j, head = h * a.G.d + c - j * a.G.d;
      a.lse[(size_t)row * a.heads + head] = lse_of(Ml, l);
    }
  };
  if constexpr (WIDE) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int c = c0 + nb * 16 + r, col = c - w.block * CB;
      if (c >= c1) continue;
#pragma unroll
      for (int dt = 0; dt < ND; ++dt) put(col, 16 * dt + 4 * g, cols.acc[nb][dt], cols.M[nb], cols.Ml[nb], cols.l[nb]);
      if (g == 0) put_ml(col, cols.M[nb], cols.Ml[nb], cols.l[nb]);
    }
  } else {
    // the four waves' sums, each scaled to the common maximum, through LDS
    if (g == 0) {
      wave_ml[wave][0][r] = cols.M[0];
      wave_ml[wave][1][r] = cols.Ml[0];
      wave_ml[wave][2][r] = cols.l[0];
    }
    __syncthreads();
    float M = kNone, Ml = kNone, l = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      M = fmaxf(M, wave_ml[k][0][r]);
      Ml = fmaxf(Ml, wave_ml[k][1][r]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) l += wave_ml[k][2][r] * __builtin_amdgcn_exp2f(wave_ml[k][1][r] - Ml);
    const float f = __builtin_amdgcn_exp2f(cols.M[0] - M);
    f32x4 *box = (f32x4 *)smem;  // [wave][dt][lane]
#pragma unroll
    for (int dt = 0; dt < ND; ++dt) {
      f32x4 v = cols.acc[0][dt];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= f;
      box[(wave * ND + dt) * 64 + lane] = v;
    }
    __syncthreads();
    const int col = r;
    if (col >= n_cols) return;
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
      put(col, 16 * dt + 4 * g, v, M, Ml, l);
    }
    if (wave == 0 && g == 0) put_ml(col, M, Ml, l);
  }
}

// Joins the chunks of split units.  A unit of nc chunks has nc slots, and
// the k-th slot's workgroup takes the items k, k + nc, .. of the unit, an
// item being 64 dims of a column: the items are spread like the chunks were.
// The workgroup's 16 groups of 16 threads share an item's chunks where those
// are many, and take an item each where they are few.
template <int D, bool F32>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendJoin a) {
  constexpr int kGroups = 16, kParts = D / 64;
  __shared__ f32x4 sums[256];
  __shared__ float ml[kGroups][3];
  const AttendJoin::Form f = a.form[blockIdx.z];
  if ((int)blockIdx.x >= f.slots) return;
  const int used = *f.used;
  const AttendRecord rec = f.records[blockIdx.x];  // in one round trip with `used`
  if ((int)blockIdx.x >= used) return;
  const int tid = threadIdx.x, group = tid >> 4, lane = tid & 15;
  const size_t floats = (size_t)f.cb * (D + 3);
  int share = 1;  // groups to an item: eight chunks at a time each
  while (share < kGroups && 8 * share < rec.nc) share *= 2;
  const int abreast = kGroups / share, sub = group & (share - 1);
  const int items = rec.n_cols * kParts;
  for (int i0 = rec.k; i0 < items; i0 += rec.nc * abreast) {
    const int item = i0 + group / share * rec.nc, col = item / kParts, d = item % kParts * 64 + lane * 4;
    const bool live = item < items;
    float M = kNone, Ml = kNone, l = 0.f;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    for (int i1 = sub; live && i1 < rec.nc; i1 += 8 * share) {
      f32x4 v[8];
      float m[8], n[8], o[8];
      float Mx = M, Mlx = Ml;
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // past the end: the first again, with no weight
        const int at = i1 + i * share;
        const float *p = f.part + (size_t)(rec.slot0 + (at < rec.nc ? at : i1) * rec.step) * floats;
        v[i] = *(const f32x4 *)(p + col * D + d);
        p += f.cb * D + col;
        m[i] = p[0];
        n[i] = p[f.cb];
        o[i] = p[2 * f.cb];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        Mx = fmaxf(Mx, m[i]);
        Mlx = fmaxf(Mlx, n[i]);
      }
      const float s = __builtin_amdgcn_exp2f(M - Mx);
      l *= __builtin_amdgcn_exp2f(Ml - Mlx);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] *= s;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i1 + i * share >= rec.nc) continue;
        const float t = __builtin_amdgcn_exp2f(m[i] - Mx);
        l += o[i] * __builtin_amdgcn_exp2f(n[i] - Mlx);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += t * v[i][e];
      }
      M = Mx;
      Ml = Mlx;
    }
    if (share > 1) {
      __syncthreads();
      sums[tid] = sum;
      if (lane == 0) {
        ml[group][0] = M;
        ml[group][1] = Ml;
        ml[group][2] = l;
      }
      __syncthreads();
      if (sub != 0 || !live) continue;
      for (int i = 1; i < share; ++i) {
        M = fmaxf(M, ml[group + i][0]);
        Ml = fmaxf(Ml, ml[group + i][1]);
      }
      l = 0.f;
      sum = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int i = 0; i < share; ++i) {
        const float t = __builtin_amdgcn_exp2f(ml[group + i][0] - M);
        l += ml[group + i][2] * __builtin_amdgcn_exp2f(ml[group + i][1] - Ml);
        const f32x4 v = sums[tid + i * 16];
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += t * v[e];
      }
    } else if (!live) {
      continue;
    }
    const int c = rec.col0 + col, j = a.G.div(c), row = rec.row0 + j, head = rec.h * a.G.d + c - j * a.G.d;
    const float t = final_scale<F32>(M, Ml, l);
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] *= t;
    store_out<F32>(a.out, (size_t)row * a.out_stride + head * D + d, sum);
    if (d == 0 && a.lse) a.lse[(size_t)row * a.heads + head] = lse_of(Ml, l);
  }
}

// ---------------------------------------------------------------- launchers
template <int D, int NB, bool F32, bool WIDE>
static void go(const AttendArgs &a, hipStream_t st) {
  constexpr int CB = (WIDE ? 64 : 16) * NB;
  const int s = a.kv.n < a.kv.n_seqs ? a.kv.n : a.kv.n_seqs;
  const long long blocks = s + ((long long)a.kv.n * a.G.d - s) / CB;  // sum of ceil(cols / CB) over s sequences at most
  // without splits there is a chunk a unit; a narrow launch of few units is
  // faster with idle workgroups beside them (7.7 us for 8.2 with 384 beside 8)
  hipLaunchKernelGGL((attend_kernel<D, NB, F32, WIDE>), dim3((unsigned)(((a.split || !WIDE ? a.per_head : 0) + blocks) * a.kv.H)), dim3(256), 0, st, a);
}
template <int D>
static void go_dim(const AttendArgs &a, int dtype, AttendForm f, hipStream_t st) {
  if (f == kNarrow) dtype == 0 ? go<D, 1, true, false>(a, st) : go<D, 1, false, false>(a, st);
  else if (dtype == 0) go<D, 1, true, true>(a, st);
  else if (f == kWide || D > 128) go<D, 1, false, true>(a, st);
  else if constexpr (D <= 128) go<D, 2, false, true>(a, st);
}
hipError_t launch_attend(const AttendArgs &a, int dim, int dtype, AttendForm f, hipStream_t st) {
  dim == 64 ? go_dim<64>(a, dtype, f, st) : dim == 128 ? go_dim<128>(a, dtype, f, st) : go_dim<256>(a, dtype, f, st);
  return hipGetLastError();
}

template <int D>
static void join_dim(const AttendJoin &a, int dtype, int forms, hipStream_t st) {
  const dim3 grid(forms > 1 ? std::max(a.form[0].slots, a.form[1].slots) : a.form[0].slots, 1, forms);
  if (dtype == 0) hipLaunchKernelGGL((attend_join_kernel<D, true>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((attend_join_kernel<D, false>), grid, dim3(256), 0, st, a);
}
hipError_t launch_attend_join(const AttendJoin &a, int dim, int dtype, int forms, hipStream_t st) {
  dim == 64 ? join_dim<64>(a, dtype, forms, st) : dim == 128 ? join_dim<128>(a, dtype, forms, st) : join_dim<256>(a, dtype, forms, st);
  return hipGetLastError();
}

}  // namespace lora
