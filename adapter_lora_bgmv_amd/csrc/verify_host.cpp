// verify_host.cpp -- the C ABI of the KV cache, the attention over it and the token scores.
//
// Host side only, like lora_host.cpp: argument checks before any launch,
// workspace layouts, launch geometry.  Nothing here allocates, frees,
// synchronises or reads device memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>

#include "../../include/lora_mi355x.h"
#include "host.hpp"
#include "verify.hpp"

using namespace lora;

namespace lora {

int check_type(const char *what, int32_t dtype) {
  if (dtype != LORA_F32 && dtype != LORA_BF16)
    return fail(LORA_ERR_DTYPE, "%s: dtype %d is neither LORA_F32 (0) nor LORA_BF16 (1)", what, dtype);
  return LORA_OK;
}

int check_rows(const char *what, int32_t dtype, const char *name, const void *p, uint32_t stride, uint64_t width, uint32_t n) {
  const uint32_t unit = dtype == LORA_BF16 ? 8 : 4;
  if (stride < width)
    return fail(LORA_ERR_STRIDE, "%s: %s row stride %u < its row of %llu elements", what, name, stride, (unsigned long long)width);
  if (stride > (uint32_t)INT_MAX)
    return fail(LORA_ERR_STRIDE, "%s: %s row stride %u exceeds %d", what, name, stride, INT_MAX);
  if (stride % unit)
    return fail(LORA_ERR_UNSUPPORTED, "%s: %s row stride %u must be a multiple of %u", what, name, stride, unit);
  if (n && !p) return fail(LORA_ERR_NULL_PTR, "%s: %s must be non-NULL", what, name);
  if (n && !aligned16(p)) return fail(LORA_ERR_UNSUPPORTED, "%s: %s %p must be 16-byte aligned", what, name, p);
  return LORA_OK;
}

}  // namespace lora

namespace {

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// The cache and the sequences of a call of n rows; fills *d.
int check_kv(const char *what, const lora_kv_cache *c, const lora_kv_seqs *s, uint32_t n, KvDev *d) {
  if (!c || !s) return fail(LORA_ERR_NULL_PTR, "%s: cache %p and seqs %p must be non-NULL", what, (const void *)c, (const void *)s);
  if (c->n_pages == 0 || c->n_kv_heads == 0)
    return fail(LORA_ERR_SHAPE, "%s: cache of n_pages %u, n_kv_heads %u: both must be >= 1", what, c->n_pages, c->n_kv_heads);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return fail(LORA_ERR_UNSUPPORTED, "%s: head_dim %u is none of 64, 128, 256", what, c->head_dim);
  int shift = 4;
  while (shift < 7 && (1u << shift) != c->page_tokens) ++shift;
  if ((1u << shift) != c->page_tokens)
    return fail(LORA_ERR_UNSUPPORTED, "%s: page_tokens %u is none of 16, 32, 64, 128", what, c->page_tokens);
  if (c->n_kv_heads > 65535 || (uint64_t)c->n_pages * c->n_kv_heads * (c->page_tokens / 16) > (uint64_t)INT_MAX)
    return fail(LORA_ERR_SHAPE, "%s: cache of n_pages %u x n_kv_heads %u x page_tokens %u holds more than 2^31 - 1 groups "
                "of 16 tokens, or more than 65535 heads", what, c->n_pages, c->n_kv_heads, c->page_tokens);
  if (n > kMaxRows)
    return fail(LORA_ERR_SHAPE, "%s: n %u rows exceeds the limit %u", what, n, kMaxRows);
  if (s->n_seqs > kMaxRows || (n && s->n_seqs == 0))
    return fail(LORA_ERR_SHAPE, "%s: n_seqs %u must be in 1..%u for n %u rows", what, s->n_seqs, kMaxRows, n);
  if (n && (s->max_pages == 0 || (uint64_t)s->max_pages * c->page_tokens > (uint64_t)(INT_MAX - 64)))
    return fail(LORA_ERR_SHAPE, "%s: max_pages %u x page_tokens %u must be in 1..%d tokens", what, s->max_pages,
                c->page_tokens, INT_MAX - 64);
  if (s->table_stride < s->max_pages)
    return fail(LORA_ERR_STRIDE, "%s: table_stride %u < max_pages %u", what, s->table_stride, s->max_pages);
  if (n == 0) return LORA_OK;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale)
    return fail(LORA_ERR_NULL_PTR, "%s: cache k %p, v %p, k_scale %p, v_scale %p must be non-NULL", what, c->k, c->v,
                (const void *)c->k_scale, (const void *)c->v_scale);
  if (!s->page_table || !s->row_indptr || !s->kv_len)
    return fail(LORA_ERR_NULL_PTR, "%s: page_table %p, row_indptr %p, kv_len %p must be non-NULL", what,
                (const void *)s->page_table, (const void *)s->row_indptr, (const void *)s->kv_len);
  if (!aligned16(c->k) || !aligned16(c->v))
    return fail(LORA_ERR_UNSUPPORTED, "%s: cache k %p and v %p must be 16-byte aligned", what, c->k, c->v);
  d->k = (uint8_t *)c->k;
  d->v = (uint8_t *)c->v;
  d->ke = c->k_scale;
  d->ve = c->v_scale;
  d->n_pages = (int)std::min<uint32_t>(c->n_pages, INT_MAX);
  d->H = (int)c->n_kv_heads;
  d->page_shift = shift;
  d->table = s->page_table;
  d->table_stride = (int)s->table_stride;
  d->max_pages = (int)s->max_pages;
  d->indptr = s->row_indptr;
  d->kv_len = s->kv_len;
  d->n_seqs = (int)s->n_seqs;
  d->n = (int)n;
  return LORA_OK;
}

// Which forms an attention call launches.  Sequences of up to
// kAttendNarrowCols columns take the narrow form, longer ones the wide form
// or its wider units.  max_rows bounds every sequence's rows and with n also
// from below; where it leaves one form, that form takes every sequence, so
// that a wrong bound costs time only.
struct AttendPlan {
  struct Part {
    AttendForm form;
    size_t records, sums;  // offsets in the workspace, after a place for the slots in use
    int slots;
    bool split;  // a unit may be cut into chunks
  } part[2];
  int parts;
  bool split;  // of either
  size_t total;
};
AttendPlan attend_plan(const lora_kv_cache *c, const lora_kv_seqs *s, int32_t dtype, uint32_t n_heads, uint32_t n) {
  AttendPlan p{};
  const int dim = (int)c->head_dim;
  const uint64_t G = std::max<uint64_t>(1, n_heads / std::max(1u, c->n_kv_heads));
  const uint64_t most = s->max_rows ? std::min(s->max_rows, n) : n;
  const uint64_t others = (uint64_t)(s->n_seqs ? s->n_seqs - 1 : 0) * most;
  const uint64_t least = n > others ? n - others : 0;
  // a table that holds no more tiles than a chunk's least splits nothing
  const uint64_t tiles = ((uint64_t)s->max_pages * c->page_tokens + 63) / 64;
  p.total = 256;
  auto add = [&](AttendForm f) {
    AttendPlan::Part &q = p.part[p.parts++];
    q.form = f;
    q.slots = attend_slots(dim, dtype, f);
    q.records = p.total;
    q.sums = q.records + up256(q.slots * sizeof(AttendRecord));
    p.total = q.sums + up256((size_t)q.slots * attend_cols(f) * (dim + 3) * 4);
    q.split = tiles > (uint64_t)attend_min_tiles(f);
    p.split |= q.split;
  };
  const bool wide = most * G > (uint64_t)kAttendNarrowCols;
  if (wide) add(dtype == LORA_BF16 && dim <= 128 && most * G > (uint64_t)kAttendWideCols ? kWider : kWide);
  if (!wide || least * G <= (uint64_t)kAttendNarrowCols) add(kNarrow);
  return p;
}

}  // namespace

extern "C" {

int lora_kv_write(const lora_kv_cache *cache, const lora_kv_seqs *seqs, int32_t dtype, const void *k, uint32_t k_row_stride,
                  const void *v, uint32_t v_row_stride, uint32_t n, void *stream) {
  clear_err();
  const char *what = "lora_kv_write";
  KvDev d{};
  if (int e = check_type(what, dtype)) return e;
  if (int e = check_kv(what, cache, seqs, n, &d)) return e;
  const uint64_t row = (uint64_t)cache->n_kv_heads * cache->head_dim;
  if (int e = check_rows(what, dtype, "k", k, k_row_stride, row, n)) return e;
  if (int e = check_rows(what, dtype, "v", v, v_row_stride, row, n)) return e;
  if (n == 0) return LORA_OK;
  if (int e = check_device(what)) return e;
  hipStream_t st = (hipStream_t)stream;
  return timed(what, st, [&] {
    return launch_kv_write(d, (int)cache->head_dim, dtype, k, (int)k_row_stride, v, (int)v_row_stride, st);
  });
}

int lora_kv_write_rotary(const lora_kv_cache *cache, const lora_kv_seqs *seqs, const lora_rotary *rotary, int32_t dtype,
                         uint32_t n_heads, const void *q, uint32_t q_row_stride, void *q_out, uint32_t q_out_row_stride,
                         const void *k, uint32_t k_row_stride, const void *v, uint32_t v_row_stride, uint32_t n, void *stream) {
  clear_err();
  const char *what = "lora_kv_write_rotary";
  KvDev d{};
  if (int e = check_type(what, dtype)) return e;
  if (int e = check_kv(what, cache, seqs, n, &d)) return e;
  if (!rotary || !rotary->inv_freq)
    return fail(LORA_ERR_NULL_PTR, "%s: rotary %p and its inv_freq must be non-NULL", what, (const void *)rotary);
  if ((uintptr_t)rotary->inv_freq % 4)
    return fail(LORA_ERR_UNSUPPORTED, "%s: inv_freq %p must be aligned to its 4 bytes", what, (const void *)rotary->inv_freq);
  if (rotary->rot_dim == 0 || rotary->rot_dim > cache->head_dim || rotary->rot_dim % 16)
    return fail(LORA_ERR_UNSUPPORTED, "%s: rot_dim %u must be a multiple of 16, at most head_dim %u", what, rotary->rot_dim,
                cache->head_dim);
  if (rotary->interleaved != 0 && rotary->interleaved != 1)
    return fail(LORA_ERR_UNSUPPORTED, "%s: interleaved %d must be 0 or 1", what, rotary->interleaved);
  if (n_heads > 65535) return fail(LORA_ERR_SHAPE, "%s: n_heads %u exceeds 65535", what, n_heads);
  const uint64_t row = (uint64_t)cache->n_kv_heads * cache->head_dim, q_row = (uint64_t)n_heads * cache->head_dim;
  if (n_heads) {
    if (int e = check_rows(what, dtype, "q", q, q_row_stride, q_row, n)) return e;
    if (int e = check_rows(what, dtype, "q_out", q_out, q_out_row_stride, q_row, n)) return e;
    if (n && q == q_out && q_row_stride != q_out_row_stride)
      return fail(LORA_ERR_STRIDE, "%s: in place, q row stride %u and q_out row stride %u must be equal", what, q_row_stride,
                  q_out_row_stride);
  }
  if (int e = check_rows(what, dtype, "k", k, k_row_stride, row, n)) return e;
  if (int e = check_rows(what, dtype, "v", v, v_row_stride, row, n)) return e;
  if (n == 0) return LORA_OK;
  const uint64_t grid = 2ull * kv_max_touched((int)n, (int)seqs->n_seqs, (int)cache->page_tokens) * cache->n_kv_heads +
                        (uint64_t)n_heads * n;
  if (grid > (uint64_t)INT_MAX)
    return fail(LORA_ERR_SHAPE, "%s: n %u rows of n_kv_heads %u and n_heads %u need more than 2^31 - 1 workgroups", what, n,
                cache->n_kv_heads, n_heads);
  if (int e = check_device(what)) return e;
  const RotaryDev rot{rotary->inv_freq, (int)rotary->rot_dim, rotary->interleaved != 0};
  const TurnArgs turn{q, q_out, (int)q_row_stride, (int)q_out_row_stride, (int)n_heads, 0, 0, 0, 0};
  hipStream_t st = (hipStream_t)stream;
  return timed(what, st, [&] {
    return launch_kv_write_rotary(d, rot, turn, (int)cache->head_dim, dtype, k, (int)k_row_stride, v, (int)v_row_stride, st);
  });
}

int lora_kv_read(const lora_kv_cache *cache, const lora_kv_seqs *seqs, int32_t dtype, void *k, uint32_t k_row_stride, void *v,
                 uint32_t v_row_stride, uint32_t n, void *stream) {
  clear_err();
  const char *what = "lora_kv_read";
  KvDev d{};
  if (int e = check_type(what, dtype)) return e;
  if (int e = check_kv(what, cache, seqs, n, &d)) return e;
  const uint64_t row = (uint64_t)cache->n_kv_heads * cache->head_dim;
  if (int e = check_rows(what, dtype, "k", k, k_row_stride, row, n)) return e;
  if (int e = check_rows(what, dtype, "v", v, v_row_stride, row, n)) return e;
  if (n == 0) return LORA_OK;
  if (int e = check_device(what)) return e;
  hipStream_t st = (hipStream_t)stream;
  return timed(what, st, [&] {
    return launch_kv_read(d, (int)cache->head_dim, dtype, k, (int)k_row_stride, v, (int)v_row_stride, st);
  });
}

size_t lora_kv_attend_workspace_bytes(const lora_kv_cache *cache, const lora_kv_seqs *seqs, int32_t dtype, uint32_t n_heads,
                                      uint32_t n) {
  return cache && seqs && n ? attend_plan(cache, seqs, dtype, n_heads, n).total : 0;
}

int lora_kv_attend(const lora_kv_cache *cache, const lora_kv_seqs *seqs, int32_t dtype, uint32_t n_heads, const void *q,
                   uint32_t q_row_stride, float scale, uint32_t window, uint32_t n, void *out, uint32_t out_row_stride,
                   float *lse, void *workspace, size_t workspace_bytes, void *stream) {
  clear_err();
  const char *what = "lora_kv_attend";
  AttendArgs a{};
  if (int e = check_type(what, dtype)) return e;
  if (int e = check_kv(what, cache, seqs, n, &a.kv)) return e;
  if (n_heads == 0 || n_heads > 65535 || n_heads % cache->n_kv_heads)
    return fail(LORA_ERR_SHAPE, "%s: n_heads %u must be a multiple of n_kv_heads %u, at most 65535", what, n_heads,
                cache->n_kv_heads);
  if (!std::isfinite(scale) || !(scale > 0.f))
    return fail(LORA_ERR_SHAPE, "%s: scale %g must be finite and above 0", what, (double)scale);
  if (window > (uint32_t)INT_MAX)
    return fail(LORA_ERR_SHAPE, "%s: window %u exceeds %d", what, window, INT_MAX);
  const uint64_t row = (uint64_t)n_heads * cache->head_dim;
  if (int e = check_rows(what, dtype, "q", q, q_row_stride, row, n)) return e;
  if (int e = check_rows(what, dtype, "out", out, out_row_stride, row, n)) return e;
  if (n == 0) return LORA_OK;
  const AttendPlan p = attend_plan(cache, seqs, dtype, n_heads, n);
  if (!workspace || workspace_bytes < p.total)
    return fail(LORA_ERR_WORKSPACE, "%s: n %u rows of %u heads x %u: workspace %p of %zu bytes, %zu needed", what, n, n_heads,
                cache->head_dim, workspace, workspace_bytes, p.total);
  if (!aligned16(workspace))
    return fail(LORA_ERR_UNSUPPORTED, "%s: workspace %p is not 16-byte aligned", what, workspace);
  if (int e = check_device(what)) return e;
  a.q = q;
  a.q_stride = (int)q_row_stride;
  a.out = out;
  a.out_stride = (int)out_row_stride;
  a.lse = lse;
  a.heads = (int)n_heads;
  a.G = fast_div((int)(n_heads / cache->n_kv_heads));
  a.H = fast_div(a.kv.H);
  a.scale = (float)((double)scale * 1.4426950408889634);
  a.window = (int)window;
  AttendJoin j{};
  j.out = out;
  j.out_stride = a.out_stride;
  j.lse = lse;
  j.heads = a.heads;
  j.G = a.G;
  char *ws = (char *)workspace;
  hipStream_t st = (hipStream_t)stream;
  return timed(what, st, [&] {
    hipError_t e = hipSuccess;
    const int dim = (int)cache->head_dim;
    for (int i = 0; i < p.parts && e == hipSuccess; ++i) {  // the long rows first: the short ones fill in behind them
      const AttendPlan::Part &q = p.part[i];
      a.used = (int *)ws + i;
      a.records = (AttendRecord *)(ws + q.records);
      a.part = (float *)(ws + q.sums);
      a.min_tiles = attend_min_tiles(q.form);
      a.split = q.split;
      a.per_head = std::max(1, attend_target(dim, dtype, q.form) / a.kv.H);
      a.cols_lo = p.parts > 1 && i == 0 ? kAttendNarrowCols : 0;
      a.cols_hi = i == 1 ? kAttendNarrowCols : INT_MAX;
      j.form[i] = {a.records, a.used, a.part, q.slots, attend_cols(q.form)};
      e = launch_attend(a, dim, dtype, q.form, st);
    }
    if (p.split && e == hipSuccess) e = launch_attend_join(j, dim, dtype, p.parts, st);
    return e;
  });
}

size_t lora_token_logprobs_workspace_bytes(int32_t dtype, uint32_t n_vocab, uint32_t n, uint32_t top) {
  if (n == 0 || n > kMaxRows || n_vocab == 0 || n_vocab > LORA_MAX_VOCAB || top > (uint32_t)kScoreMaxTop ||
      (dtype != LORA_F32 && dtype != LORA_BF16))
    return 0;
  const int chunks = score_split((int)n, (int)n_vocab, dtype).chunks;
  return chunks > 1 ? up256((size_t)n * 4) + (size_t)n * chunks * score_record_bytes((int)top) : 0;
}

int lora_token_logprobs(int32_t dtype, uint32_t n_vocab, const void *logits, uint32_t row_stride, const int32_t *token_ids,
                        uint32_t n, uint32_t top, float *logp, float *entropy, int32_t *rank, int32_t *top_ids,
                        float *top_logp, void *workspace, size_t workspace_bytes, void *stream) {
  clear_err();
  const char *what = "lora_token_logprobs";
  if (int e = check_type(what, dtype)) return e;
  if (n_vocab == 0 || n_vocab > LORA_MAX_VOCAB)
    return fail(LORA_ERR_SHAPE, "%s: n_vocab %u must be in 1..%u", what, n_vocab, LORA_MAX_VOCAB);
  if (n > kMaxRows)
    return fail(LORA_ERR_SHAPE, "%s: [n %u x n_vocab %u]: n exceeds the limit %u", what, n, n_vocab, kMaxRows);
  if (top > (uint32_t)kScoreMaxTop || top > n_vocab)
    return fail(LORA_ERR_SHAPE, "%s: top %u must be at most %d and at most n_vocab %u", what, top, kScoreMaxTop, n_vocab);
  if (row_stride < n_vocab)
    return fail(LORA_ERR_STRIDE, "%s: row_stride %u < n_vocab %u", what, row_stride, n_vocab);
  if (n == 0) return LORA_OK;
  if (!logits || !token_ids || !logp || (top && (!top_ids || !top_logp)))
    return fail(LORA_ERR_NULL_PTR, "%s: [n %u x n_vocab %u] top %u: logits %p, token_ids %p, logp %p%s must be non-NULL", what, n,
                n_vocab, top, logits, (const void *)token_ids, (const void *)logp, top ? ", top_ids, top_logp" : "");
  const size_t size = dtype == LORA_F32 ? 4 : 2;
  if ((uintptr_t)logits % size)
    return fail(LORA_ERR_UNSUPPORTED, "%s: logits %p must be aligned to their %zu bytes", what, logits, size);
  const size_t need = lora_token_logprobs_workspace_bytes(dtype, n_vocab, n, top);
  if (need && (!workspace || workspace_bytes < need))
    return fail(LORA_ERR_WORKSPACE, "%s: [n %u x n_vocab %u] top %u: workspace %p of %zu bytes, %zu needed", what, n, n_vocab, top,
                workspace, workspace_bytes, need);
  if (need && !aligned16(workspace))
    return fail(LORA_ERR_UNSUPPORTED, "%s: workspace %p is not 16-byte aligned", what, workspace);
  if (int e = check_device(what)) return e;
  ScoreArgs a{};
  a.logits = logits;
  a.stride = row_stride;
  a.n = (int)n;
  a.n_vocab = (int)n_vocab;
  a.top = (int)top;
  a.ids = token_ids;
  a.logp = logp;
  a.entropy = entropy;
  a.rank = rank;
  a.top_ids = top_ids;
  a.top_logp = top_logp;
  const ScoreSplit split = score_split((int)n, (int)n_vocab, dtype);
  a.chunks = split.chunks;
  a.batches = split.batches;
  a.cnt = (unsigned *)workspace;
  a.part = (float *)((char *)workspace + up256((size_t)n * 4));
  hipStream_t st = (hipStream_t)stream;
  return timed(what, st, [&] { return launch_score(a, dtype, st); });
}

size_t lora_token_sample_workspace_bytes(int32_t dtype, uint32_t n_vocab, uint32_t n) {
  if (n == 0 || n > kMaxRows || n_vocab == 0 || n_vocab > LORA_MAX_VOCAB || (dtype != LORA_F32 && dtype != LORA_BF16)) return 0;
  const int chunks = sample_chunks((int)n, (int)n_vocab, dtype);
  return chunks > 1 ? n * sample_row_bytes(chunks) : 0;
}

int lora_token_sample(int32_t dtype, uint32_t n_vocab, const void *logits, uint32_t row_stride, const float *temperature,
                      const int32_t *top_k, const float *top_p, const float *min_p, const float *uniform, uint32_t n, int32_t *ids,
                      float *logp, void *workspace, size_t workspace_bytes, void *stream) {
  clear_err();
  const char *what = "lora_token_sample";
  if (int e = check_type(what, dtype)) return e;
  if (n_vocab == 0 || n_vocab > LORA_MAX_VOCAB)
    return fail(LORA_ERR_SHAPE, "%s: n_vocab %u must be in 1..%u", what, n_vocab, LORA_MAX_VOCAB);
  if (n > kMaxRows)
    return fail(LORA_ERR_SHAPE, "%s: [n %u x n_vocab %u]: n exceeds the limit %u", what, n, n_vocab, kMaxRows);
  if (row_stride < n_vocab)
    return fail(LORA_ERR_STRIDE, "%s: row_stride %u < n_vocab %u", what, row_stride, n_vocab);
  if (n == 0) return LORA_OK;
  if (!logits || !uniform || !ids)
    return fail(LORA_ERR_NULL_PTR, "%s: [n %u x n_vocab %u]: logits %p, uniform %p, ids %p must be non-NULL", what, n, n_vocab,
                logits, (const void *)uniform, (const void *)ids);
  const size_t size = dtype == LORA_F32 ? 4 : 2;
  if ((uintptr_t)logits % size)
    return fail(LORA_ERR_UNSUPPORTED, "%s: logits %p must be aligned to their %zu bytes", what, logits, size);
  const size_t need = lora_token_sample_workspace_bytes(dtype, n_vocab, n);
  if (need && (!workspace || workspace_bytes < need))
    return fail(LORA_ERR_WORKSPACE, "%s: [n %u x n_vocab %u]: workspace %p of %zu bytes, %zu needed", what, n, n_vocab, workspace,
                workspace_bytes, need);
  if (need && !aligned16(workspace))
    return fail(LORA_ERR_UNSUPPORTED, "%s: workspace %p is not 16-byte aligned", what, workspace);
  if (int e = check_device(what)) return e;
  const SampleArgs a{logits, row_stride, (int)n, (int)n_vocab, temperature, top_p, min_p, top_k, uniform, ids, logp,
                     sample_chunks((int)n, (int)n_vocab, dtype), workspace};
  hipStream_t st = (hipStream_t)stream;
  return timed(what, st, [&] { return launch_sample(a, dtype, st); });
}

}  // extern "C"
