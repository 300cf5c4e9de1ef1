// Argument checks and sizes of include/qpn_decode.h (declared in
// qpn_decode_checks.hpp).
#include "qpn_decode_checks.hpp"

#include <limits.h>
#include <math.h>

#include <algorithm>

#include "qpn_checks.hpp"

namespace qpn {

namespace {

constexpr int64_t kMaxStride = int64_t(1) << 40;  // elements; keeps every 64-bit offset far from its end

constexpr int64_t kMaxGroups = int64_t(1) << 23;  // workgroups of a launch: 2^31 threads

// Whether runs of up to `tokens` tokens go whole, a workgroup each, or the line
// of all tiles is cut into equal shares, which takes a join. Both measured (one
// row of 5 heads a kv head; whole / cut): 8 runs of 512 tokens 7.3 / 9.3 us,
// of 1024 10.5 / 9.4; 128 of 1024 12.7 / 15.6, of 2048 20.7 / 18.4; 512 of
// 1024 17.8 / 31.3, of 4096 58 / 65. They meet near 512 tokens for 8 runs and
// at twice that for four times the runs. (All of equal lengths at their bound. The
// rule knows the bound alone: many runs of which one is long go whole too, and
// that one then takes its workgroup as long as its tiles do.)
bool whole_runs(int64_t tokens, int64_t runs) { return tokens <= 512 || tokens * tokens <= 32768 * runs; }

bool positive(float x) { return isfinite(x) && x > 0.0f; }

bool page_size_ok(int32_t p) { return p == 16 || p == 32 || p == 64 || p == 128 || p == 256; }

bool half_type(int32_t dtype) { return dtype == QPN_DT_F16 || dtype == QPN_DT_BF16; }

bool stride_ok(int64_t s) { return s >= 0 && s <= kMaxStride; }

size_t round16(size_t n) { return (n + 15) & ~size_t(15); }

}  // namespace

int64_t kv4_segment_bytes(int page_size, int head_dim) {
  return static_cast<int64_t>(page_size) * head_dim * 9 / 8;
}

qpn_status check_kv4_cache(const qpn_kv4_cache* c) {
  if (!c) return QPN_ERR_INVALID_ARG;
  if (qpn_kv4_page_bytes(c->page_size, c->kv_heads, c->head_dim) == 0) return QPN_ERR_INVALID_ARG;
  if (c->layers < 1 || c->pages < 0 || c->pages > INT32_MAX) return QPN_ERR_INVALID_ARG;
  if (!positive(c->k_scale) || !positive(c->v_scale)) return QPN_ERR_INVALID_ARG;
  if (c->pages > 0 && (!c->data || !aligned(c->data, 16))) return QPN_ERR_INVALID_ARG;
  return QPN_OK;
}

qpn_status check_kv4_append(const qpn_kv4_cache* c, int32_t layer, const void* k, const void* v, int32_t dtype,
                            int64_t tokens, int64_t k_ts, int64_t k_hs, int64_t v_ts, int64_t v_hs,
                            const int64_t* slots, bool* run) {
  *run = false;
  const qpn_status st = check_kv4_cache(c);
  if (st != QPN_OK) return st;
  if (layer < 0 || layer >= c->layers || !half_type(dtype)) return QPN_ERR_INVALID_ARG;
  if (tokens < 0 || tokens > INT32_MAX) return QPN_ERR_INVALID_ARG;
  if (!stride_ok(k_ts) || !stride_ok(k_hs) || !stride_ok(v_ts) || !stride_ok(v_hs)) return QPN_ERR_INVALID_ARG;
  if (tokens == 0 || c->pages == 0) return QPN_OK;  // no slot exists: every token is skipped
  if (!k || !v || !aligned(k, 2) || !aligned(v, 2) || !slots || !aligned(slots, 8)) return QPN_ERR_INVALID_ARG;
  *run = true;
  return QPN_OK;
}

qpn_status check_kv4_read(const qpn_kv4_cache* c, int32_t layer, const int64_t* slots, int64_t tokens, int32_t dtype,
                          const void* k, const void* v, bool* run) {
  *run = false;
  const qpn_status st = check_kv4_cache(c);
  if (st != QPN_OK) return st;
  if (layer < 0 || layer >= c->layers) return QPN_ERR_INVALID_ARG;
  if (!half_type(dtype) && dtype != QPN_DT_F32) return QPN_ERR_INVALID_ARG;
  if (tokens < 0 || tokens > INT32_MAX) return QPN_ERR_INVALID_ARG;
  if (tokens == 0) return QPN_OK;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || !slots || !aligned(slots, 8)) return QPN_ERR_INVALID_ARG;
  *run = true;  // an empty pool still writes zeros
  return QPN_OK;
}

qpn_status check_kv4_copy_pages(const qpn_kv4_cache* c, const int32_t* src, const int32_t* dst, int64_t count,
                                bool* run) {
  *run = false;
  const qpn_status st = check_kv4_cache(c);
  if (st != QPN_OK) return st;
  if (count < 0 || count > INT32_MAX) return QPN_ERR_INVALID_ARG;
  if (count == 0 || c->pages == 0) return QPN_OK;
  if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4)) return QPN_ERR_INVALID_ARG;
  *run = true;
  return QPN_OK;
}

qpn_status plan_attention(const qpn_kv4_cache* c, const qpn_kv4_attention_args* a, AttentionPlan* p) {
  if (!c || !a || a->reserved != 0) return QPN_ERR_INVALID_ARG;
  if (qpn_kv4_page_bytes(c->page_size, c->kv_heads, c->head_dim) == 0) return QPN_ERR_INVALID_ARG;
  if (a->heads < 1 || a->heads > 65536 || a->heads % c->kv_heads != 0) return QPN_ERR_INVALID_ARG;
  if (a->batch < 0 || a->batch > 65536 || a->rows < 0 || a->max_q_len < 0 || a->max_q_len > 65536)
    return QPN_ERR_INVALID_ARG;
  // positions and token counts stay inside 32 bits with a tile to spare
  if (a->max_kv_len < 0 || a->max_kv_len > (1 << 30) || a->window < 0) return QPN_ERR_INVALID_ARG;
  const int64_t rows = static_cast<int64_t>(std::min(a->max_q_len, a->rows)) * (a->heads / c->kv_heads);
  const int64_t t16 = std::max<int64_t>(1, (rows + 15) / 16);
  const int most = c->head_dim == 256 ? 2 : c->head_dim == 128 ? 3 : 4;
  p->row_tiles = static_cast<int>((t16 + most - 1) / most);
  p->tiles16 = static_cast<int>((t16 + p->row_tiles - 1) / p->row_tiles);
  p->row_tiles = static_cast<int>((t16 + p->tiles16 - 1) / p->tiles16);
  // the tiles of all sequences, row tiles and heads are counted in 32 bits
  const int64_t runs = static_cast<int64_t>(a->batch) * p->row_tiles * c->kv_heads;
  const int64_t tiles = std::max<int64_t>(1, (static_cast<int64_t>(a->max_kv_len) + kTileTokens - 1) / kTileTokens) + 64;
  if (runs > kMaxGroups || runs * tiles > INT32_MAX - (1 << 20)) return QPN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(a->rows) * a->heads > kMaxGroups) return QPN_ERR_UNSUPPORTED;
  p->groups = whole_runs(a->max_kv_len, runs) ? 0 : kComputeUnits * attn_waves_per_simd(c->head_dim, p->tiles16);
  p->min_share = kAttnWaves;
  p->cut_bytes = static_cast<size_t>(p->groups) * 32;
  p->partial_bytes = 2 * static_cast<size_t>(p->groups) * 16 * p->tiles16 * (c->head_dim + 2) * sizeof(float);
  p->total_bytes = a->batch == 0 || a->rows == 0 || p->groups == 0 ? 0 : p->cut_bytes + p->partial_bytes;
  return QPN_OK;
}

qpn_status check_kv4_attention(const qpn_kv4_cache* c, const qpn_kv4_attention_args* a, const void* ws,
                               size_t ws_bytes, AttentionPlan* p, bool* run) {
  *run = false;
  qpn_status st = check_kv4_cache(c);
  if (st != QPN_OK) return st;
  st = plan_attention(c, a, p);
  if (st != QPN_OK) return st;
  if (a->layer < 0 || a->layer >= c->layers || !half_type(a->dtype) || !positive(a->scale)) return QPN_ERR_INVALID_ARG;
  if (!stride_ok(a->q_token_stride) || !stride_ok(a->q_head_stride)) return QPN_ERR_INVALID_ARG;
  if (a->table_stride < 0 || a->table_stride > INT32_MAX) return QPN_ERR_INVALID_ARG;
  if (a->table_stride * c->page_size < a->max_kv_len) return QPN_ERR_INVALID_ARG;
  if (!a->q_start && static_cast<int64_t>(a->batch) * a->max_q_len != a->rows) return QPN_ERR_INVALID_ARG;
  if (a->rows > 0 && a->batch == 0) return QPN_ERR_INVALID_ARG;
  if (a->batch == 0 || a->rows == 0) return QPN_OK;
  if (a->max_q_len == 0) return QPN_ERR_INVALID_ARG;
  if (!a->q || !aligned(a->q, 2) || !a->out || !aligned(a->out, 16)) return QPN_ERR_INVALID_ARG;
  if (a->lse && !aligned(a->lse, 4)) return QPN_ERR_INVALID_ARG;
  if (!a->kv_len || !aligned(a->kv_len, 4)) return QPN_ERR_INVALID_ARG;
  if (a->max_kv_len > 0 && (!a->table || !aligned(a->table, 4))) return QPN_ERR_INVALID_ARG;
  if (a->q_start && !aligned(a->q_start, 4)) return QPN_ERR_INVALID_ARG;
  if (p->total_bytes > 0) {
    if (!ws || !aligned(ws, 16)) return QPN_ERR_INVALID_ARG;
    if (ws_bytes < p->total_bytes) return QPN_ERR_BUFFER_TOO_SMALL;
  }
  *run = true;
  return QPN_OK;
}

bool plan_verify(int32_t batch, int32_t drafts, int32_t vocab, VerifyPlan* p) {
  if (batch < 0 || batch > 65536 || drafts < 0 || drafts > 64 || vocab < 1 || vocab > (1 << 24)) return false;
  p->chunk = 4096;
  p->chunks = (vocab + p->chunk - 1) / p->chunk;
  const size_t rows = static_cast<size_t>(batch) * (2 * drafts + 1);
  // (a launch of 1024-thread workgroups a chunk, too)
  if (rows * p->chunks > static_cast<size_t>(kMaxGroups) ||
      static_cast<size_t>(batch) * p->chunks > static_cast<size_t>(kMaxGroups) / 4)
    return false;
  p->verdict_bytes = static_cast<size_t>(batch) * 32;
  p->stat_bytes = rows * p->chunks * 16;
  p->total_bytes = p->verdict_bytes + p->stat_bytes +
                   round16(static_cast<size_t>(batch) * p->chunks * 3 * sizeof(double));
  return true;
}

qpn_status check_verify(const qpn_verify_args* a, const void* ws, size_t ws_bytes, VerifyPlan* p, bool* run) {
  *run = false;
  if (!a || a->reserved != 0) return QPN_ERR_INVALID_ARG;
  if (!plan_verify(a->batch, a->drafts, a->vocab, p)) return QPN_ERR_INVALID_ARG;
  if (!half_type(a->dtype) && a->dtype != QPN_DT_F32) return QPN_ERR_INVALID_ARG;
  if (a->probabilities != 0 && a->probabilities != 1) return QPN_ERR_INVALID_ARG;
  // probabilities after a filter need their 32 bits, and have no temperature left
  if (a->probabilities && (a->dtype != QPN_DT_F32 || a->temperature)) return QPN_ERR_INVALID_ARG;
  if (!stride_ok(a->target_batch_stride) || !stride_ok(a->target_row_stride) || !stride_ok(a->draft_batch_stride) ||
      !stride_ok(a->draft_row_stride))
    return QPN_ERR_INVALID_ARG;
  if (a->batch == 0) return QPN_OK;
  const uintptr_t size = a->dtype == QPN_DT_F32 ? 4 : 2;
  if (!a->target || !aligned(a->target, size)) return QPN_ERR_INVALID_ARG;
  if (a->draft && !aligned(a->draft, size)) return QPN_ERR_INVALID_ARG;
  if (a->drafts > 0) {
    if (!a->draft_tokens || !aligned(a->draft_tokens, 4)) return QPN_ERR_INVALID_ARG;
    if (!a->u_accept || !aligned(a->u_accept, 4)) return QPN_ERR_INVALID_ARG;
  }
  if (!a->u_sample || !aligned(a->u_sample, 4)) return QPN_ERR_INVALID_ARG;
  if (!aligned(a->num_draft, 4) || !aligned(a->temperature, 4) || !aligned(a->logprobs, 4)) return QPN_ERR_INVALID_ARG;
  if (!a->tokens || !aligned(a->tokens, 4) || !a->accepted || !aligned(a->accepted, 4)) return QPN_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 16)) return QPN_ERR_INVALID_ARG;
  if (ws_bytes < p->total_bytes) return QPN_ERR_BUFFER_TOO_SMALL;
  *run = true;
  return QPN_OK;
}

}  // namespace qpn

extern "C" {

size_t qpn_kv4_page_bytes(int32_t page_size, int32_t kv_heads, int32_t head_dim) {
  if (!qpn::page_size_ok(page_size) || kv_heads < 1 || kv_heads > 1024) return 0;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
  return static_cast<size_t>(qpn::kv4_segment_bytes(page_size, head_dim)) * kv_heads;
}

size_t qpn_kv4_attention_workspace_bytes(const qpn_kv4_cache* cache, const qpn_kv4_attention_args* args) {
  qpn::AttentionPlan p;
  return qpn::plan_attention(cache, args, &p) == QPN_OK ? p.total_bytes : 0;
}

size_t qpn_verify_workspace_bytes(int32_t batch, int32_t drafts, int32_t vocab) {
  qpn::VerifyPlan p;
  return qpn::plan_verify(batch, drafts, vocab, &p) ? p.total_bytes : 0;
}

}  // extern "C"
