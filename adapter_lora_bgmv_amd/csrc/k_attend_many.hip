// k_attend_many.hip -- attention over the 8-bit paged cache where sequences bring many rows (prompts), bf16.
//
// The mathematics, the lagging maximum and the values' exponents are those
// of k_attend.hip.  What differs is who converts: there every wave converts
// the codes of the tile for its own columns, 128 conversions for 64 matrix
// products, which cost as much as a third of the products.  Here a workgroup
// is eight waves of 32 columns, each converts an eighth of the tile (halves of
// a 16-token group of K and of V, loaded straight into registers) and puts it
// into LDS as bf16 or f16 times the page's scale, once, and all of them read
// finished operands.  A tile costs a wave 16 conversions for its 64 products, 32
// exponentials, and 32 LDS reads of 16 bytes a lane, about half of what the
// LDS can give.
//
// The matrix products take longer than all else together, and hide it where
// one wave alternates them: a step is one operand against both column blocks,
// with a share of the other work between: the next tile's scores run among
// this tile's weights, and the sums among the conversions of K two tiles ahead
// and of V one ahead.
//
// In LDS a fragment's 16 rows of 16 bytes lie side by side, so that reads and
// writes are free of bank conflicts.  K: [4 quads j][D/16 chunks c][half s]
// [16]; row 4 q + token of group q's quad, with q exchanged by the chunk
// (q ^ {0, 3, 1, 2}[c % 4]) because the four chunks that a read takes at once
// would otherwise share banks in writing.  V: [4 groups][half s][D].
#include "attend.hpp"
#include "common.hpp"
#include "verify.hpp"

namespace lora {

constexpr int kManyThreads = 512;

template <int D>
struct ManyLds {
  static constexpr int kKeys = 8 * D, kValues = 8 * D;  // 16-byte units of a tile
  uint4 k[3][kKeys], v[2][kValues];
  int info[2][4][2];  // of the groups of a tile, by the halves of V: bit 0 it has a page, bit 1 NaN codes, from bit 8 on 256 + rest
};

template <int D>
struct ManyColumns {
  static constexpr int NB = 2, NS = D / 32, ND = D / 16;
  using X = ValueExp<false>;
  uint4 q[NB][NS];
  f32x4 acc[NB][ND];
  f32x4 S[NB][4];              // a tile's scores, where `ahead` already
  float M[NB], Ml[NB], l[NB];  // as in k_attend.hip
  int hi[NB];
  bool mixed, ahead;

  __device__ __forceinline__ void load(const AttendArgs &a, const Work &w, int h, int c0, int c1, int r, int g) {
    mixed = ahead = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int c = c0 + nb * 16 + r;
      const bool ok = c < c1;
      const int j = ok ? a.G.div(c) : 0;
      hi[nb] = ok ? w.s.start + j + 1 : 0;
      const u16 *p = (const u16 *)a.q + (size_t)(w.s.row0 + j) * a.q_stride + (h * a.G.d + (ok ? c - j * a.G.d : 0)) * D;
#pragma unroll
      for (int s = 0; s < NS; ++s) q[nb][s] = ok ? ldg16(p + 16 * (4 * (s >> 1) + g) + 8 * (s & 1)) : z4();
      M[nb] = Ml[nb] = kNone;
      l[nb] = 0.f;
#pragma unroll
      for (int dt = 0; dt < ND; ++dt) acc[nb][dt] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }

  // Waits for q here rather than at its first use, which is in the loop and
  // would wait for what is on its way there.
  __device__ __forceinline__ void arrive() {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int s = 0; s < NS; ++s) asm volatile("" : "+v"(q[nb][s].x), "+v"(q[nb][s].y), "+v"(q[nb][s].z), "+v"(q[nb][s].w));
  }

  static __device__ __forceinline__ float largest(const f32x4 (&s)[4]) {
    float mx = s[0][0];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) mx = fmaxf(mx, s[j][e]);
    return mx;
  }
  static __device__ __forceinline__ uint32_t &word(uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

  // Fragment f of a tile's keys: two quads in turn over all parts (chunks 4 n +
  // g and half s, 2 n + s), then the other two, so that no sum is added to
  // twice in a row and the scores before make room for those after; of its
  // values, 16 dims dt and half s.
  static constexpr int kKeyFrags = 8 * (D / 64), kValueFrags = 2 * ND;
  static __device__ __forceinline__ int quad_of(int f) { return f / (kKeyFrags / 2) * 2 + f % 2; }
  static __device__ __forceinline__ int part_of(int f) { return f % (kKeyFrags / 2) / 2; }
  static __device__ __forceinline__ int dims_of(int f) { return f / 4 * 2 + f % 2; }
  static __device__ __forceinline__ int half_of(int f) { return f / 2 % 2; }
  static __device__ __forceinline__ uint4 key(const uint4 *k, int f) {
    return k[((quad_of(f) * (D / 16) + part_of(f) / 2 * 4) * 2 + part_of(f) % 2) * 16];
  }
  static __device__ __forceinline__ uint4 value(const uint4 *v, int f) { return v[half_of(f) * D + dims_of(f) * 16]; }

  __device__ __forceinline__ void score(const uint4 *k) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < 4; ++j) S[nb][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int f = 0; f < kKeyFrags; ++f) {
      const uint4 x = key(k, f);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) S[nb][quad_of(f)] = mfma16(x, q[nb][part_of(f)], S[nb][quad_of(f)]);
    }
  }

  // The rest of a tile that every column sees all of and that has nothing
  // unusual in it, from S and values v; false, and nothing changed, where the
  // maximum has to move.  Afterwards S holds the scores of the next tile's
  // keys (after the last tile: of whatever lies there).
  // side(k), k < kValueFrags, is other work for the vector unit.
  template <typename Side>
  __device__ __forceinline__ bool plain(float cs, const uint4 *v, const uint4 *next, Side side) {
    constexpr int kAhead = 6;  // fragments on their way from LDS: a step is 33 cycles, a read 130 and more
    constexpr int kSteps = kKeyFrags, kEach = 16 / kSteps;
    uint4 x[kAhead];
#pragma unroll
    for (int f = 0; f < kAhead; ++f) x[f] = key(next, f);
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
    uint4 pf[NB][2];
    f32x4 T[NB][4];
    float f[NB], p[NB][16], b[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      b[nb] = kTop - M[nb];
      f[nb] = fmaf(S[nb][0][0], cs, b[nb]);
#pragma unroll
      for (int j = 0; j < 4; ++j) T[nb][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        __builtin_amdgcn_sched_barrier(0);
        T[nb][quad_of(k)] = mfma16(x[k % kAhead], q[nb][part_of(k)], T[nb][quad_of(k)]);
        if (nb == NB - 1) x[k % kAhead] = k + kAhead < kSteps ? key(next, k + kAhead) : value(v, k + kAhead - kSteps);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const int e = k * kEach + i;
          p[nb][e] = __builtin_amdgcn_exp2f(f[nb]);
          if (e + 1 < 16) f[nb] = fmaf(S[nb][(e + 1) >> 2][(e + 1) & 3], cs, b[nb]);
          if (e > 0) l[nb] += p[nb][e - 1];
          if (e >= 2 && e % 2 == 0) word(pf[nb][(e - 2) / 8], (e - 2) / 2 % 4) = pack_f16(p[nb][e - 2], p[nb][e - 1]);
        }
      }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      l[nb] += p[nb][15];
      pf[nb][1].w = pack_f16(p[nb][14], p[nb][15]);
#pragma unroll
      for (int j = 0; j < 4; ++j) S[nb][j] = T[nb][j];
    }
#pragma unroll
    for (int k = 0; k < kValueFrags; ++k) {
      __builtin_amdgcn_sched_barrier(0);
      uint4 &y = x[(kSteps + k) % kAhead];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) acc[nb][dims_of(k)] = mfma16_f16(y, pf[nb][half_of(k)], acc[nb][dims_of(k)]);
      if (k + kAhead < kValueFrags) y = value(v, k + kAhead);
      side(k);
    }
    return true;
  }

  // The rest of any tile for column block B0, from token tok0 of the lane and
  // keys k: masks, rests, maxima that moved, NaN codes.
  template <int B0>
  __device__ __forceinline__ void careful(float cs, int tok0, int info, bool nans, int window, const uint4 *k, const uint4 *v) {
    f32x4 s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int f = 0; f < kKeyFrags; ++f) s[quad_of(f)] = mfma16(key(k, f), q[B0][part_of(f)], s[quad_of(f)]);
    const float rest = (float)((info >> 8) - 256);
    const uint32_t see = info & 1 ? sees(hi[B0], window, tok0) : 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t m = (uint32_t)((int32_t)(see << (31 - 4 * j - i)) >> 31);
        s[j][i] = __uint_as_float((__float_as_uint(s[j][i]) & m) | (0xff800000u & ~m));
      }
    const float topl = largest(s) * cs, top = topl + rest;
    if (__any(top > M[B0] + kLag || topl > Ml[B0] + kLag)) {
      const float Mn = fmaxf(M[B0], groups_max(top)), Mln = fmaxf(Ml[B0], groups_max(topl));
      const float f = __builtin_amdgcn_exp2f(M[B0] - Mn);
      l[B0] *= __builtin_amdgcn_exp2f(Ml[B0] - Mln);
      M[B0] = Mn;
      Ml[B0] = Mln;
#pragma unroll
      for (int dt = 0; dt < ND; ++dt) acc[B0][dt] *= f;
    }
    uint4 pf[2];
    const float b = kTop - M[B0] + rest, bl = kTop - Ml[B0];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float y = s[2 * h + (e >> 2)][e & 3];
        p[e] = __builtin_amdgcn_exp2f(fmaf(y, cs, b));
        l[B0] += mixed ? __builtin_amdgcn_exp2f(fmaf(y, cs, bl)) : p[e];
      }
      pf[h] = make_uint4(pack_f16(p[0], p[1]), pack_f16(p[2], p[3]), pack_f16(p[4], p[5]), pack_f16(p[6], p[7]));
    }
    if (__builtin_expect(!nans, 1)) {
#pragma unroll
      for (int f = 0; f < kValueFrags; ++f) acc[B0][dims_of(f)] = mfma16_f16(value(v, f), pf[half_of(f)], acc[B0][dims_of(f)]);
      return;
    }
    // NaN values would reach every column: they become zeros, and the columns
    // that see one are counted by a product of ones (0x3c00 is 1.0 in f16)
#pragma unroll
    for (int f = 0; f < kValueFrags; ++f) {
      uint4 x = value(v, f), one = z4();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t &y = word(x, i);
        const uint32_t lo = (y & 0x7fffu) > 0x7c00u ? 0xffffu : 0u, hi4 = (y & 0x7fff0000u) > 0x7c000000u ? 0xffff0000u : 0u;
        word(one, i) = (lo | hi4) & 0x3c003c00u;
        y &= ~(lo | hi4);
      }
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t m = see >> (8 * half_of(f) + 2 * e);
        o[e] = (m & 1 ? 0x3c00u : 0u) | (m & 2 ? 0x3c000000u : 0u);
      }
      const f32x4 n = mfma16_f16(one, make_uint4(o[0], o[1], o[2], o[3]), f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n[e] > 0.f) acc[B0][dims_of(f)][e] = __uint_as_float(0x7fc00000u);
      acc[B0][dims_of(f)] = mfma16_f16(x, pf[half_of(f)], acc[B0][dims_of(f)]);
    }
  }
};

template <int D>
__global__ __launch_bounds__(kManyThreads, 2) void attend_many_kernel(AttendArgs a) {
  constexpr int CB = kAttendManyCols, ND = D / 16, U = D / 64;
  __shared__ ManyLds<D> lds;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int H = a.kv.H, item = a.H.div(blockIdx.x), h = blockIdx.x - item * H;
  Work w;
  int all_slots;
  const bool found = find_work<CB>(a, item, lane, &w, &all_slots);
  if (blockIdx.x == 0 && tid == 0) *a.used = all_slots * H;
  if (!found) return;
  const int cap = kv_cap(a.kv), n_cols = min(CB, w.s.rows * a.G.d - w.block * CB);
  const int r = lane & 15, g = lane >> 4;

  const int j_first = a.G.div(w.block * CB), j_last = a.G.div(w.block * CB + n_cols - 1);
  const int hi_u = max(min(w.s.start + j_last + 1, cap), 0);
  const int lo_u = a.window ? max(w.s.start + j_first + 1 - a.window, 0) : 0;
  const int tile0 = lo_u / kTile, tiles = hi_u > lo_u ? (hi_u + kTile - 1) / kTile - tile0 : 0;
  int ta = tile0, tb = tile0 + tiles;
  if (w.nc > 1) {  // the first tiles % nc chunks take one more
    const int each = tiles / w.nc, more = tiles - each * w.nc;
    ta += w.chunk * each + min(w.chunk, more);
    tb = ta + each + (w.chunk < more);
  }
  const int c0 = w.block * CB + wave * 32, c1 = min(c0 + 32, w.s.rows * a.G.d);
  const int j0 = a.G.div(c0), j1 = a.G.div(max(c1 - 1, 0));
  const int hi_all = min(w.s.start + j0 + 1, cap), lo_all = a.window ? w.s.start + j1 + 1 - a.window : 0;
  const int wave_lo = a.window ? max(w.s.start + j0 + 1 - a.window, 0) : 0;
  const int wave_hi = c0 < c1 ? min(w.s.start + j1 + 1, cap) : 0;

  ManyColumns<D> cols;
  cols.load(a, w, h, c0, c1, r, g);

  // This wave's share of the tiles: half of group `mine`, of K two tiles ahead and of V one.
  constexpr int kLanes = D / 2;  // a 16-byte unit each: 16 dims of a token of K, 16 tokens of a dim of V
  const int mine = wave >> 1, unit = (wave & 1) * kLanes + (lane & (kLanes - 1));
  const bool works = kLanes == 64 || lane < kLanes;
  const int c = (unit >> 2) % (D / 16), x = ((c >> 1) & 1) ^ ((c & 1) * 3);
  const int to_k = ((unit >> 2) / (D / 16) * (D / 16) + c) * 32 + 4 * (mine ^ x) + (unit & 3), to_v = mine * 2 * D + unit;
  int first = ta - 64, group = 0, ke = 0, ve = 0;  // lane l's page of tile first + l
  unsigned long long there = 0;
  auto pages = [&](int t) {  // the pages of 64 tiles from t on
    first = t;
    const int tok = (t + lane) * kTile + 16 * mine;
    const int page = t + lane < tb && tok < cap ? page_of(a.kv, w.seq, tok >> a.kv.page_shift) : -1;
    const size_t ph = page >= 0 ? (size_t)page * H + h : 0;
    ke = a.kv.ke[ph];
    ve = a.kv.ve[ph];
    group = page >= 0 ? (int)((ph << (a.kv.page_shift - 4)) + ((tok & ((1 << a.kv.page_shift) - 1)) >> 4)) : 0;
    there = __ballot(page >= 0);
  };
  // What is on its way: a unit of K of tile tk, of V of tile tv, and their exponents.  Past the last tile: it again.
  uint4 raw_k, raw_v;
  int exp_k, exp_v, rest_v;
  uint32_t there_k, there_v;  // all ones, or 0 without a page
  auto fetch_k = [&](int t) {
    const int at = min(t, tb - 1) - first;
    raw_k = ldg16(a.kv.k + (size_t)(unsigned)__builtin_amdgcn_readlane(group, at) * (16 * D) + unit * 16);
    exp_k = __builtin_amdgcn_readlane(ke, at);
    there_k = there >> at & 1 ? ~0u : 0u;
  };
  auto fetch_v = [&](int t) {
    const int at = min(t, tb - 1) - first;
    raw_v = ldg16(a.kv.v + (size_t)(unsigned)__builtin_amdgcn_readlane(group, at) * (16 * D) + unit * 16);
    const int e = __builtin_amdgcn_readlane(ve, at);
    there_v = there >> at & 1 ? ~0u : 0u;
    exp_v = there_v ? min(max(e, ValueExp<false>::kLo), ValueExp<false>::kHi) : 127;
    rest_v = there_v ? e - exp_v : 0;
  };
  // The conversions in parts: half p of the unit of K into a place of three, of V into one of two.
  auto put_k = [&](int place, int p) {
    const uint32_t lo = (p ? raw_k.z : raw_k.x) & there_k, hi = (p ? raw_k.w : raw_k.y) & there_k;
    const uint4 y = codes_bf16(lo, hi, scale_of(exp_k));
    if (works) lds.k[place][to_k + 16 * p] = y;
  };
  auto put_v = [&](int place, int p) {
    const uint32_t lo = (p ? raw_v.z : raw_v.x) & there_v, hi = (p ? raw_v.w : raw_v.y) & there_v;
    const uint4 y = codes_f16(lo, hi, scale_of(exp_v + ValueExp<false>::kAdd));
    if (works) lds.v[place][to_v + D * p] = y;
  };
  auto put_info = [&](int place) {
    const uint32_t any = has_nan(raw_v.x) | has_nan(raw_v.y) | has_nan(raw_v.z) | has_nan(raw_v.w);
    const int nan = __any((any & there_v & 0x80808080u) != 0) ? 2 : 0;
    lds.info[place][mine][wave & 1] = (int)(there_v & 1) | nan | (rest_v + 256) << 8;  // the same from every lane
  };

  int kb = 0;
  if (ta < tb) {
    pages(ta);
    fetch_k(ta);
    fetch_v(ta);
    put_k(0, 0);
    put_k(0, 1);
    fetch_k(ta + 1);
    put_v(0, 0);
    put_v(0, 1);
    put_info(0);
    fetch_v(ta + 1);
    put_k(1, 0);
    put_k(1, 1);
    fetch_k(ta + 2);
    cols.arrive();
  }
  for (int t = ta; t < tb; ++t) {
    if (t + 3 >= first + 64) pages(t);
    __syncthreads();  // tile t's V and tile t + 1's K are there; nobody reads what is written next
    const int vb = (t - ta) & 1, kn = kb == 2 ? 0 : kb + 1, kw = kn == 2 ? 0 : kn + 1;
    auto side = [&](int k) {  // tile t + 2's K, tile t + 1's V, and the fetches after them
      if (k == 1) put_k(kw, 0);
      if (k == 2) put_k(kw, 1);
      if (k == 3) fetch_k(t + 3);
      if (k == 4) put_v(vb ^ 1, 0);
      if (k == 5) put_v(vb ^ 1, 1);
      if (k == 6) put_info(vb ^ 1);
      if (k == 7) fetch_v(t + 2);
    };
    bool done = false;
    if (t * kTile < wave_hi && (t + 1) * kTile > wave_lo) {
      const int again = lane_again(), r = again & 15, g = again >> 4, x = ((g >> 1) & 1) ^ ((g & 1) * 3);
      const int at_k = g * 32 + 4 * ((r >> 2) ^ x) + (r & 3);
      const uint4 *v = &lds.v[vb][g * 2 * D + r];
      const int info = lds.info[vb][g][0] | (lds.info[vb][g][1] & 2);
      const bool usual = __all((info & ~2) == (1 | 256 << 8));
      if (__builtin_expect(usual && !cols.mixed && t * kTile >= lo_all && (t + 1) * kTile <= hi_all, 1)) {
        if (!cols.ahead) cols.score(&lds.k[kb][at_k]);
        done = cols.plain(a.scale, v, &lds.k[kn][at_k], side);
      }
      cols.ahead = done;
      if (__builtin_expect(!done, 0)) {
        const bool nans = __any(info & 2);
        if (!cols.mixed) {  // with no rest so far M and Ml move together
          cols.mixed = __any(info >> 8 != 256);
          cols.Ml[0] = cols.M[0];
          cols.Ml[1] = cols.M[1];
        }
        cols.template careful<0>(a.scale, t * kTile + 16 * g, info, nans, a.window, &lds.k[kb][at_k], v);
        asm volatile("" ::: "memory");  // read anew: held, the fragments would take the registers of the sums
        cols.template careful<1>(a.scale, t * kTile + 16 * g, info, nans, a.window, &lds.k[kb][at_k], v);
      }
    }
    if (!done) {
#pragma unroll
      for (int k = 0; k < 8; ++k) side(k);
    }
    kb = kn;
  }

  const bool split = w.nc > 1;
  const int slot = split ? (w.slot + w.chunk) * H + h : 0;
  float *part = a.part + (size_t)slot * CB * (D + 3), *ml = part + CB * D;
  if (split && tid == 0) {
    const AttendRecord rec = {w.slot * H + h, H, w.nc, w.chunk, n_cols, w.s.row0, w.block * CB, h};
    a.records[slot] = rec;
  }
#pragma unroll
  for (int nb = 0; nb < 2; ++nb) {
    const float l = groups_sum(cols.l[nb]), M = cols.M[nb], Ml = cols.mixed ? cols.Ml[nb] : M;
    const int c = c0 + nb * 16 + r, col = c - w.block * CB;
    if (c >= c1) continue;
    const int j = a.G.div(c), row = w.s.row0 + j, head = h * a.G.d + c - j * a.G.d;
    const float f = split ? 1.f : final_scale<false>(M, Ml, l);
#pragma unroll
    for (int dt = 0; dt < ND; ++dt) {
      f32x4 v = cols.acc[nb][dt];
      const int d = 16 * dt + 4 * g;
      if (split) {
        *(float4 *)(part + col * D + d) = make_float4(v[0], v[1], v[2], v[3]);
      } else {
        v *= f;
        store_out<false>(a.out, (size_t)row * a.out_stride + head * D + d, v);
      }
    }
    if (g != 0) continue;
    if (split) {
      ml[col] = M;
      ml[CB + col] = Ml;
      ml[2 * CB + col] = l;
    } else if (a.lse) {
      a.lse[(size_t)row * a.heads + head] = lse_of(Ml, l);
    }
  }
}

template <int D>
static void go_many(const AttendArgs &a, hipStream_t st) {
  constexpr int CB = kAttendManyCols;
  const int s = a.kv.n < a.kv.n_seqs ? a.kv.n : a.kv.n_seqs;
  const long long blocks = s + ((long long)a.kv.n * a.G.d - s) / CB;  // sum of ceil(cols / CB) over s sequences at most
  hipLaunchKernelGGL((attend_many_kernel<D>), dim3((unsigned)((a.per_head + blocks) * a.kv.H)), dim3(kManyThreads), 0, st, a);
}
hipError_t launch_attend_many(const AttendArgs &a, int dim, hipStream_t st) {
  dim == 64 ? go_many<64>(a, st) : go_many<128>(a, st);
  return hipGetLastError();
}

}  // namespace lora
