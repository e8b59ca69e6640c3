// k_attend_many.hip -- attention over the 8-bit paged cache where sequences bring many rows (prompts), bf16.
//
// The mathematics, the lagging maximum and the values' exponents are those
// of k_attend.hip.  What differs is who converts: there every wave converts
// the codes of the tile for its own columns, 128 conversions for 64 matrix
// products, which cost as much as a third of the products.  Here a workgroup
// is eight waves of 32 columns, each converts an eighth of the tile (a 16-token
// group of K or of V, loaded straight into registers) and puts it into LDS as
// bf16 or f16 times the page's scale, once, and all of them read finished
// operands.  A tile costs a wave 16 conversions for its 64 products, 32
// exponentials, and 32 LDS reads of 16 bytes a lane, about half of what the
// LDS can give.
//
// The matrix products take longer than all else together, and hide it where
// one wave alternates them: a step is one operand against both column blocks,
// with a share of the other work between.  The next tile's scores run among
// this tile's weights, so K is kept a tile ahead of V: while a tile is worked
// on, waves 0-3 convert K two tiles ahead and waves 4-7 V one ahead.
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
  int info[2][4];  // of the groups of a tile of V: bit 0 it has a page, bit 1 NaN codes, from bit 8 on 256 + rest
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

  static __device__ __forceinline__ float largest(const f32x4 (&s)[4]) {
    float mx = s[0][0];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) mx = fmaxf(mx, s[j][e]);
    return mx;
  }
  static __device__ __forceinline__ uint32_t &word(uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

  // Fragment f of a tile's keys, f = (j D/64 + n) 2 + s: quad j, chunks 4 n + g, half s; of its values, f = 2 dt + s.
  static __device__ __forceinline__ uint4 key(const uint4 *k, int f) {
    const int s = f & 1, n = (f >> 1) % (D / 64), j = (f >> 1) / (D / 64);
    return k[((j * (D / 16) + 4 * n) * 2 + s) * 16];
  }
  static __device__ __forceinline__ uint4 value(const uint4 *v, int f) { return v[(f & 1) * D + (f >> 1) * 16]; }
  static constexpr int kKeyFrags = 8 * (D / 64), kValueFrags = 2 * ND;
  static __device__ __forceinline__ int quad_of(int f) { return (f >> 1) / (D / 64); }
  static __device__ __forceinline__ int part_of(int f) { return 2 * ((f >> 1) % (D / 64)) + (f & 1); }

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
  __device__ __forceinline__ bool plain(float cs, const uint4 *v, const uint4 *next) {
    constexpr int kAhead = 3;  // fragments on their way from LDS
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
      for (int nb = 0; nb < NB; ++nb) acc[nb][k >> 1] = mfma16_f16(y, pf[nb][k & 1], acc[nb][k >> 1]);
      if (k + kAhead < kValueFrags) y = value(v, k + kAhead);
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
      for (int f = 0; f < kValueFrags; ++f) acc[B0][f >> 1] = mfma16_f16(value(v, f), pf[f & 1], acc[B0][f >> 1]);
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
        const uint32_t m = see >> (8 * (f & 1) + 2 * e);
        o[e] = (m & 1 ? 0x3c00u : 0u) | (m & 2 ? 0x3c000000u : 0u);
      }
      const f32x4 n = mfma16_f16(one, make_uint4(o[0], o[1], o[2], o[3]), f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n[e] > 0.f) acc[B0][f >> 1][e] = __uint_as_float(0x7fc00000u);
      acc[B0][f >> 1] = mfma16_f16(x, pf[f & 1], acc[B0][f >> 1]);
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

  // This wave's share of the tiles: group q of K, `lead` = 2 tiles ahead, or of V, 1 ahead.
  const bool keys = wave < 4;
  const int mine = wave & 3, lead = keys ? 2 : 1;
  const uint8_t *pool = keys ? a.kv.k : a.kv.v, *exps = keys ? a.kv.ke : a.kv.ve;
  int first = ta - 64, group = 0, exp = 0;  // lane l's page of tile first + l
  unsigned long long there = 0;
  uint4 raw[U];
  int raw_exp = 0;
  bool raw_there = false;
  auto fetch = [&](int t) {  // tile t's share, on its way
    if (t >= tb) return;
    if (t >= first + 64) {
      first = t;
      const int tok = (t + lane) * kTile + 16 * mine;
      const int page = t + lane < tb && tok < cap ? page_of(a.kv, w.seq, tok >> a.kv.page_shift) : -1;
      const size_t ph = page >= 0 ? (size_t)page * H + h : 0;
      exp = exps[ph];
      group = page >= 0 ? (int)((ph << (a.kv.page_shift - 4)) + ((tok & ((1 << a.kv.page_shift) - 1)) >> 4)) : 0;
      there = __ballot(page >= 0);
    }
    const uint8_t *p = pool + (size_t)(unsigned)__builtin_amdgcn_readlane(group, t - first) * (16 * D) + lane * 16;
#pragma unroll
    for (int i = 0; i < U; ++i) raw[i] = ldg16(p + i * 1024);
    raw_exp = __builtin_amdgcn_readlane(exp, t - first);
    raw_there = there >> (t - first) & 1;
  };
  auto convert = [&](int t) {  // what was fetched, into tile t's place
    if (t >= tb) return;
    const int i = t - ta;
    if (keys) {
      const float scale = scale_of(raw_exp);
#pragma unroll
      for (int n = 0; n < U; ++n) {
        const int u = lane + 64 * n, c = (u >> 2) % (D / 16), j = (u >> 2) / (D / 16);
        const int x = ((c >> 1) & 1) ^ ((c & 1) * 3);
        uint4 *to = &lds.k[i % 3][(j * (D / 16) + c) * 32 + 4 * (mine ^ x) + (u & 3)];
        to[0] = raw_there ? codes_bf16(raw[n].x, raw[n].y, scale) : z4();
        to[16] = raw_there ? codes_bf16(raw[n].z, raw[n].w, scale) : z4();
      }
    } else {
      using X = ValueExp<false>;
      const int vc = min(max(raw_exp, X::kLo), X::kHi);
      const float scale = scale_of(vc + X::kAdd);
      uint32_t any = 0;
#pragma unroll
      for (int n = 0; n < U; ++n) {
        uint4 *to = &lds.v[i & 1][mine * 2 * D + lane + 64 * n];
        to[0] = raw_there ? codes_f16(raw[n].x, raw[n].y, scale) : z4();
        to[D] = raw_there ? codes_f16(raw[n].z, raw[n].w, scale) : z4();
        any |= has_nan(raw[n].x) | has_nan(raw[n].y) | has_nan(raw[n].z) | has_nan(raw[n].w);
      }
      const int nan = raw_there && __any((any & 0x80808080u) != 0) ? 2 : 0;
      if (lane == 0) lds.info[i & 1][mine] = (int)raw_there | nan | (raw_there ? raw_exp - vc + 256 : 256) << 8;
    }
  };
  fetch(ta);
  convert(ta);
  fetch(ta + 1);
  if (keys) {
    convert(ta + 1);
    fetch(ta + 2);
  }

  int kb = 0;
  for (int t = ta; t < tb; ++t) {
    __syncthreads();  // tile t's V and tile t + 1's K are there; nobody reads what is written next
    const int i = t - ta, kn = kb == 2 ? 0 : kb + 1;
    if (t * kTile < wave_hi && (t + 1) * kTile > wave_lo) {
      const int again = lane_again(), r = again & 15, g = again >> 4, x = ((g >> 1) & 1) ^ ((g & 1) * 3);
      const int at_k = g * 32 + 4 * ((r >> 2) ^ x) + (r & 3);
      const uint4 *v = &lds.v[i & 1][g * 2 * D + r];
      const int info = lds.info[i & 1][g];
      const bool usual = __all((info & ~2) == (1 | 256 << 8)), nans = __any(info & 2);
      bool done = usual && !cols.mixed && t * kTile >= lo_all && (t + 1) * kTile <= hi_all;
      if (__builtin_expect(done, 1)) {
        if (!cols.ahead) cols.score(&lds.k[kb][at_k]);
        done = cols.plain(a.scale, v, &lds.k[kn][at_k]);
        cols.ahead = done;
      }
      if (__builtin_expect(!done, 0)) {
        cols.ahead = false;
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
    convert(t + lead);
    fetch(t + lead + 1);
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
