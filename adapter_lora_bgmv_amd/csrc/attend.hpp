// attend.hpp -- what the attention kernels share: operands from codes, masks, the call's work, results.  Not part of the ABI.
#pragma once

#include "common.hpp"
#include "verify.hpp"

namespace lora {

constexpr int kTile = 64;    // tokens
constexpr float kLag = 7.f;  // log2 of how far the running maximum may lag
constexpr float kTop = 8.f;  // log2 of the weight at the running maximum: with the lag 2^15, in f16's range
constexpr float kNone = -3e38f;  // the maximum of a column that saw nothing yet

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

// 2^(e - 127).
__device__ __forceinline__ float scale_of(int e) { return __uint_as_float((uint32_t)e << 23); }

// Four codes, and eight, times a power of two as parts of a matrix operand.
__device__ __forceinline__ uint2 pair_bf16(uint32_t w, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true);
  return make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
}
__device__ __forceinline__ uint2 pair_f16(uint32_t w, float scale) {
  const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, false);
  const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, true);
  return make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
}
__device__ __forceinline__ uint4 codes_bf16(uint32_t lo, uint32_t hi, float scale) {
  const uint2 a = pair_bf16(lo, scale), b = pair_bf16(hi, scale);
  return make_uint4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ uint4 codes_f16(uint32_t lo, uint32_t hi, float scale) {
  const uint2 a = pair_f16(lo, scale), b = pair_f16(hi, scale);
  return make_uint4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ f32x4 mfma16_f16(uint4 a, uint4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
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

// Bit 7 of the bytes that hold a NaN code (and other bits that mean nothing);
// those bytes, 0xff each.
__device__ __forceinline__ uint32_t has_nan(uint32_t w) { return (w & 0x7f7f7f7fu) + 0x01010101u; }
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((has_nan(w) & 0x80808080u) >> 7) * 0xffu; }

// The lane's number, computed where it is asked for.
__device__ __forceinline__ int lane_again() {
  int l;
  asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
  return l;
}

// The lowest n of 16 bits, 0 <= n <= 16 once clamped.
__device__ __forceinline__ uint32_t live_bits(int n) { return (1u << min(max(n, 0), 16)) - 1u; }

// The first token that a column sees whose last token is hi - 1.  hi may be
// negative and a window as large as an int: no difference is taken below 0.
__device__ __forceinline__ int first_seen(int hi, int window) { return window && hi > window ? hi - window : 0; }

// Of the 16 tokens from tok0, those that such a column sees.
__device__ __forceinline__ uint32_t sees(int hi, int window, int tok0) {
  return live_bits(hi - tok0) & ~live_bits(first_seen(hi, window) - tok0);
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
  const int cols = s.rows * a.G.d;
  return cols > a.cols_lo && cols <= a.cols_hi ? (cols + CB - 1) / CB : 0;
}
// Tiles that a unit of the sequence sees at most; 1 where it sees none (its rows are written as zeros).
template <int CB>
__device__ __forceinline__ int unit_tiles(const AttendArgs &a, const SeqDev &s, int cap) {
  const int lo = first_seen(s.start + 1, a.window), hi = min(s.len, cap);
  if (hi <= lo) return 1;
  const int all = (hi + kTile - 1) / kTile - lo / kTile;
  // tokens under a window: its own and one more for every further row of the unit
  return a.window ? min(all, (int)(((long long)a.window + CB + kTile) / kTile) + 1) : all;
}

// Item u of a head's list: units in order, each with its chunks.  Every wave
// finds it by itself (lane l counts `per` sequences).  *all_slots: of a head's
// split units together.  The launch and the workspace have room for the items
// and slots of ranges that do not overlap.  A range begins where the one
// before ends, so they do as soon as one falls: such a call has no work.
template <int CB>
__device__ __forceinline__ bool find_work(const AttendArgs &a, int u, int lane, Work *w, int *all_slots) {
  const int per = (a.kv.n_seqs + 63) >> 6, cap = kv_cap(a.kv);
  const int i0 = lane * per, i1 = min(i0 + per, a.kv.n_seqs);
  SeqDev first = {0, 0, 0, 0};  // the lane's only sequence where per is 1
  bool falls = false;
  if (i0 < i1) first = load_seq(a.kv, i0, &falls);
  long long total = 0;
  for (int i = i0; i < i1; ++i) {
    const SeqDev s = i == i0 ? first : load_seq(a.kv, i, &falls);
    total += (long long)seq_blocks<CB>(a, s) * unit_tiles<CB>(a, s, cap);
  }
  *all_slots = 0;
  if (__any(falls)) return false;
  // over the lanes in two parts of 24 and up to 32 bits
  total = min(total, 1ll << 50);
  const unsigned low = (unsigned)__builtin_amdgcn_readlane(wave_incl_scan((int)(total & 0xffffff)), 63);
  const unsigned high = (unsigned)__builtin_amdgcn_readlane(wave_incl_scan((int)(total >> 24)), 63);
  total = ((long long)high << 24) + low;
  // tiles of a chunk at most (few tiles, the common case, need no 64-bit division)
  int c = a.min_tiles;
  if (total > (long long)c * a.per_head)
    c = total < 1ll << 31 ? (int)(((unsigned)total + a.per_head - 1) / (unsigned)a.per_head)
                          : (int)min((total + a.per_head - 1) / a.per_head, 1ll << 30);
  int items = 0, slots = 0;
  for (int i = i0; i < i1; ++i) {
    const SeqDev s = i == i0 ? first : load_seq(a.kv, i);
    const int b = seq_blocks<CB>(a, s), nc = (unit_tiles<CB>(a, s, cap) + c - 1) / c;
    items += b * nc;
    slots += nc > 1 ? b * nc : 0;
  }
  const int incl = wave_incl_scan(items), sincl = wave_incl_scan(slots);
  *all_slots = __builtin_amdgcn_readlane(sincl, 63);
  int found = -1, block = 0, chunk = 0, nc_of = 1, slot = 0;
  SeqDev its = first;
  if (u < incl && u >= incl - items) {
    int at = incl - items, sat = sincl - slots;
    for (int i = i0; i < i1; ++i) {
      const SeqDev s = i == i0 ? first : load_seq(a.kv, i);
      const int b = seq_blocks<CB>(a, s), nc = (unit_tiles<CB>(a, s, cap) + c - 1) / c;
      if (u < at + b * nc) {
        found = i;
        its = s;
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
  w->s = seq_of_lane(its, src);
  return true;
}

// ---------------------------------------------------------------- results
// The exponents b of values that the matrix operand takes, as bytes, and
// what it adds to them.  For f32 calls bf16's range would reach further than
// the f32 sums': up to 2^60, 2^31 tokens of codes up to 2^9 under weights up
// to 2^15 stay below 2^115.
template <bool F32>
struct ValueExp {
  static constexpr int kLo = F32 ? 10 : 106, kHi = F32 ? 187 : 127, kAdd = F32 ? 0 : 6;
};
// What a column's sums are multiplied by at the end.  A row that saw nothing
// has l = 0 and is zero; a NaN denominator stays one.
template <bool F32>
__device__ __forceinline__ float final_scale(float M, float Ml, float l) {
  return l == 0.f ? 0.f : 1.f / l * __builtin_amdgcn_exp2f(M - Ml - (float)ValueExp<F32>::kAdd);
}
// Four dims of a finished column.
template <bool F32>
__device__ __forceinline__ void store_out(void *out, size_t at, f32x4 v) {
  if constexpr (F32) *(float4 *)((float *)out + at) = make_float4(v[0], v[1], v[2], v[3]);
  else *(uint2 *)((u16 *)out + at) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}
__device__ __forceinline__ float lse_of(float Ml, float l) {
  return l == 0.f ? -INFINITY : 0.6931471805599453f * (Ml - kTop + __builtin_amdgcn_logf(l));
}

}  // namespace lora
