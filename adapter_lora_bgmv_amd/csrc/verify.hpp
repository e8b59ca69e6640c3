// verify.hpp -- arguments and launchers of the KV cache, attention and scoring kernels.  Not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"

namespace lora {

// The cache and the sequences of one call (lora_kv_cache, lora_kv_seqs), as the kernels take them.
struct KvDev {
  uint8_t *k, *v;    // [n_pages][H][P D] codes
  uint8_t *ke, *ve;  // [n_pages][H] exponent bytes
  int n_pages, H;
  int page_shift;    // log2 of the page's tokens P
  const int32_t *table;  // [n_seqs][table_stride]
  int table_stride, max_pages;
  const int32_t *indptr;  // [n_seqs + 1]
  const int32_t *kv_len;  // [n_seqs]
  int n_seqs, n;
};

// One sequence's rows and tokens, made safe: rows [row0, row0 + rows) lie in
// [0, n); row j holds position start + j, start = len - rows, which may be
// negative; tokens at or past `cap` have no page.
struct SeqDev {
  int row0, rows, len, start;
};

// *falls is set where the range ends before it begins.
__device__ __forceinline__ SeqDev load_seq(const KvDev &a, int i, bool *falls = nullptr) {
  const int lo = a.indptr[i], hi = a.indptr[i + 1], len = a.kv_len[i];
  SeqDev s;
  s.row0 = min(max(lo, 0), a.n);
  const int rows = min(max(hi, 0), a.n) - s.row0;
  if (falls) *falls |= rows < 0;
  s.rows = max(rows, 0);
  s.len = max(len, 0);
  s.start = s.len - s.rows;
  return s;
}

// Tokens the page table has room for (the host keeps max_pages << page_shift below 2^31).
__device__ __forceinline__ int kv_cap(const KvDev &a) { return a.max_pages << a.page_shift; }

// The page of logical page `p` of sequence i, or -1: an entry outside
// [0, n_pages) names none.
__device__ __forceinline__ int page_of(const KvDev &a, int i, int p) {
  const int id = a.table[(size_t)i * a.table_stride + p];
  return (unsigned)id < (unsigned)a.n_pages ? id : -1;
}

// Sums over the lanes up to and including this one, in registers: within rows
// of 16 lanes, then the last lanes of rows 0 and 2 over rows 1 and 3, then
// lane 31 over rows 2 and 3.
__device__ __forceinline__ int wave_incl_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast:15
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast:31
  return v;
}
// Over the whole wave, the same way: f(v, what the other lane has, or `none`), lane 63's at the end.
template <typename F>
__device__ __forceinline__ int wave_reduce(int v, int none, F f) {
  v = f(v, __builtin_amdgcn_update_dpp(none, v, 0x111, 0xf, 0xf, false));
  v = f(v, __builtin_amdgcn_update_dpp(none, v, 0x112, 0xf, 0xf, false));
  v = f(v, __builtin_amdgcn_update_dpp(none, v, 0x114, 0xf, 0xf, false));
  v = f(v, __builtin_amdgcn_update_dpp(none, v, 0x118, 0xf, 0xf, false));
  v = f(v, __builtin_amdgcn_update_dpp(none, v, 0x142, 0xa, 0xf, false));
  v = f(v, __builtin_amdgcn_update_dpp(none, v, 0x143, 0xc, 0xf, false));
  return __builtin_amdgcn_readlane(v, 63);
}
__device__ __forceinline__ SeqDev seq_of_lane(const SeqDev &s, int lane) {
  return {__builtin_amdgcn_readlane(s.row0, lane), __builtin_amdgcn_readlane(s.rows, lane),
          __builtin_amdgcn_readlane(s.len, lane), __builtin_amdgcn_readlane(s.start, lane)};
}

// The e4m3 byte pair conversions (gfx950).
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

hipError_t launch_kv_write(const KvDev &kv, int dim, int dtype, const void *k, int k_stride, const void *v, int v_stride,
                           hipStream_t st);
hipError_t launch_kv_read(const KvDev &kv, int dim, int dtype, void *k, int k_stride, void *v, int v_stride,
                          hipStream_t st);

// n / d for 0 <= n < 2^31 and a d of the host's: with 2^(s-1) < d <= 2^s, m =
// floor(2^(31+s) / d) + 1 exceeds 2^(31+s) / d by a part that stays below 1 / d
// of a quotient, so that floor(n m / 2^(31+s)) is exact.
struct FastDiv {
  int d;
  uint32_t m;
  int s;
  __device__ __forceinline__ int div(int n) const { return s ? (int)(__umulhi((uint32_t)n, m) >> (s - 1)) : n; }
};
inline FastDiv fast_div(int d) {
  FastDiv f{d, 0, 0};
  while ((1ll << f.s) < d) ++f.s;
  f.m = (uint32_t)((1ull << (31 + f.s)) / (uint64_t)d + 1);
  return f;
}

// The attention over the cache (k_attend.hip).
// A chunk of a split unit leaves [CB][D] sums, then M, Ml and l per column,
// and this record, by which the join knows the unit.
struct AttendRecord {
  int slot0, step, nc, k;     // the unit's slots are slot0 + i step, this is the k-th of nc
  int n_cols, row0, col0, h;  // its columns, the sequence's first row, the unit's first column, the head
};
struct AttendArgs {
  KvDev kv;
  const void *q;  // [n][q_stride], head h at h D
  int q_stride;
  void *out;      // [n][out_stride]
  int out_stride;
  float *lse;     // [n][heads] or null
  int heads;      // query heads
  FastDiv G, H;   // query heads per key/value head, and those
  float scale;    // softmax scale times log2(e)
  int window;     // 0: none
  int cols_lo, cols_hi;  // takes the sequences whose rows x G lie in (cols_lo, cols_hi]
  int per_head;   // workgroups per key/value head that the tiles are spread over
  int min_tiles;  // of a chunk: fewer are not split
  bool split;     // a unit may have more than that
  AttendRecord *records;  // of split units' chunks
  int *used;              // slots in use, written by the call
  float *part;            // their partial results
};
// The forms of the attention, by the columns (row, query head of the group)
// that a sequence brings: narrow up to 16, wide above (units of 64), and wider
// (128) where bf16 calls of up to 128 dims may bring more than 64.
enum AttendForm { kNarrow, kWide, kWider };
constexpr int kAttendNarrowCols = 16, kAttendWideCols = 64;
constexpr int attend_cols(AttendForm f) { return f == kNarrow ? kAttendNarrowCols : f == kWide ? kAttendWideCols : 128; }
// Workgroups of a CU that a form's registers allow, those that a launch's
// tiles are spread over, and the partial slots that takes: a unit is split
// into nc > 1 chunks only where its tiles exceed a chunk's, so the split
// units' chunks are fewer than twice as many. The tiles are spread over one
// round of the card, and over three quarters of one in the narrow form with
// two workgroups a CU: its units round up to whole chunks, which at a full
// round leaves a few of them to a second (8 sequences of up to 30000: 63.5 us
// over 512, 58.2 over 384, 61.3 over 320, 67.8 over 256; 16 of up to 8000:
// 32.2, 29.0, 29.8, 32.0; 64 of up to 8191 and calls of many short ones: the
// same within 3 % either way). The wide form loses by it (4 of 9 rows: 25.1
// us over a full round, 26.8 over three quarters), the others do not change.
constexpr int attend_per_cu(int dim, bool f32, AttendForm f) { return dim > 128 && (f32 || f == kNarrow) ? 1 : 2; }
constexpr int attend_target(int dim, int dtype, AttendForm f) {
  const int per_cu = attend_per_cu(dim, dtype == 0, f);
  return f == kNarrow && per_cu == 2 ? 384 : 256 * per_cu;
}
constexpr int attend_slots(int dim, int dtype, AttendForm f) { return 2 * attend_target(dim, dtype, f); }
// Tiles that are worth a chunk of their own: four a wave of the narrow form;
// four of the wide form, whose workgroups wait for memory; eight of the wider,
// whose units are many and write more than they read in the prompts that this
// leaves whole.  Each helps some calls and costs others (us, 8 heads of 128
// unless said, tables of 8192 tokens; at half as many tiles, at this, at twice):
//   narrow  1 row over 701 tokens 10.6 / 9.9 / 9.9, over 4001 11.0 / 12.6 / 15.7;
//           32 rows over 1001 19.5 / 17.5 / 17.5; 4 in f32 over 1501 14.4 / 15.9 / 19.0
//   wide    4 x 9 rows over 709 12.9 / 15.5 / 18.0; 16 x 9 over 509 18.2 / 18.9 / 17.3;
//           a prompt of 512 rows 256 wide 37.5 / 37.4 / 26.1
//   wider   prompts of 512 rows: one 32.1 / 23.2 / 23.2, two 40.3 / 26.3 / 26.5; 512
//           rows over 2512 49 / 48 / 55; 100 over 800 24.4 / 31.0 / 30.6; 40 over
//           3040 26.1 / 29.2 / 43.2; 1024 rows 44.6 / 44.6 / 37.9
constexpr int attend_min_tiles(AttendForm f) { return f == kNarrow ? 16 : f == kWide ? 4 : 8; }
hipError_t launch_attend(const AttendArgs &a, int dim, int dtype, AttendForm f, hipStream_t st);

// The join of split units, of one or both forms.
struct AttendJoin {
  struct Form {
    const AttendRecord *records;
    const int *used;
    const float *part;
    int slots, cb;  // slots at most, and the columns of each
  } form[2];
  void *out;
  int out_stride;
  float *lse;
  int heads;
  FastDiv G;
};
hipError_t launch_attend_join(const AttendJoin &a, int dim, int dtype, int forms, hipStream_t st);

// Scores of given tokens over rows of logits (k_score.hip).
constexpr int kScoreThreads = 256;
constexpr int kScoreMaxTop = 32;
constexpr int kScoreMaxChunks = 128;  // of a row: score_split stays within it
constexpr int kScoreBatch = 32;       // logits of a thread at a time
struct ScoreArgs {
  const void *logits;  // [n][stride]
  long long stride;
  int n, n_vocab, top;
  const int32_t *ids;  // [n]
  float *logp, *entropy;  // [n], or null
  int32_t *rank;          // [n] or null
  int32_t *top_ids;       // [n][top]
  float *top_logp;        // [n][top]
  int chunks;      // workgroups of a row
  int batches;     // of a chunk
  float *part;     // [n][chunks] records, see k_score.hip
  unsigned *cnt;   // [n] arrivals, zero between calls
};
struct ScoreSplit {
  int chunks, batches;
};
ScoreSplit score_split(int n, int n_vocab, int dtype);
// Bytes of one chunk's record: maximum, sum, weighted sum, count, then the top keys.
__host__ __device__ inline size_t score_record_bytes(int top) { return 16 + 8 * (size_t)((top + 1) / 2 * 2); }
hipError_t launch_score(const ScoreArgs &a, int dtype, hipStream_t st);

// Upper bound of the pages that n rows of n_seqs sequences touch: a sequence
// of m rows touches at most m pages and at most (m + P - 2) / P + 1.
inline int kv_max_touched(int n, int n_seqs, int page) {
  const int s = n < n_seqs ? n : n_seqs;
  const int by_page = n / page + 2 * s;
  return n < by_page ? n : by_page;
}

}  // namespace lora
