// Argument checks and sizes of include/qpn_prompt.h (declared in
// qpn_prompt_checks.hpp).
#include "qpn_prompt_checks.hpp"

#include <limits.h>
#include <math.h>

#include <algorithm>

#include "qpn_checks.hpp"

namespace qpn {

namespace {

constexpr int64_t kMaxStride = int64_t(1) << 40;  // elements; keeps every 64-bit offset far from its end
constexpr int64_t kMaxGroups = int64_t(1) << 23;  // workgroups of a launch: 2^31 threads of 256

bool half_type(int32_t dtype) { return dtype == QPN_DT_F16 || dtype == QPN_DT_BF16; }

int64_t type_size(int32_t dtype) { return dtype == QPN_DT_F32 ? 4 : dtype == QPN_DT_E4M3 ? 1 : 2; }

bool stride_ok(int64_t s) { return s >= 0 && s <= kMaxStride; }

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace

bool plan_fp8_block(int64_t m, int64_t n, int64_t k, Fp8BlockPlan* p) {
  if (m < 0 || m > (1 << 22) || n < 0 || n > (1 << 24) || k < 0 || k > (1 << 20) || k % 16 != 0) return false;
  *p = Fp8BlockPlan{};
  p->blocks = static_cast<int>(ceil_div(k, kScaleBlock));
  p->splits = 1;
  // A wavefront takes all of up to 48 rows, or of up to 64 under a weight of up to 40 M codes
  // (64 rows x 7168 x 5120: 18 us, in tiles 21; x 10240 x 5120: 24.5 and 23, x 5120 x 17408:
  // 41 and 35; 48 rows x 17408 x 5120: 26 and 30).
  if (m <= 48 || (m <= 64 && n * k <= 40 << 20)) {
    p->m_tiles = static_cast<int>(std::max<int64_t>(1, ceil_div(m, 16)));
    p->waves = 4;
    // Up to 256 workgroups of 16 outputs, one a compute unit, share k among more wavefronts (16
    // rows x 2048 x 17408: 12.3 us, with four 15.5; x 4096 x 16384 18.3 and 19.9; with more
    // workgroups four are enough: x 5120 x 17408 21.6 and 20.1).
    if (ceil_div(n, 16) <= kComputeUnits)
      while (p->waves < few_rows_waves(p->m_tiles) && p->blocks >= 8 * p->waves) p->waves *= 2;
  } else {
    // Tiles of 256 x 256, one a compute unit, where they come in whole rounds of 256; the
    // outputs of the last round that would not be full go in tiles of 128 x 128 (2048 x 34816
    // x 5120: 387 us, all in tiles of 256 408, all in tiles of 128 488; 1024 x 16384 x 4096,
    // one whole round: 72 and 84; with less than a round a long k would be better off, too:
    // 2048 x 5120 x 17408 257 us, in its 160 tiles of 256 219). fp32 results take those of 128 always.
    const int64_t m_tiles = ceil_div(m, 256), n_tiles = ceil_div(n, 256), rounds = m_tiles * n_tiles / kComputeUnits;
    if (m >= 256 && rounds > 0) {
      const int64_t left = m_tiles * n_tiles - rounds * kComputeUnits;
      p->wide = left > kComputeUnits * 3 / 4 ? n : rounds * kComputeUnits / m_tiles * 256;
      p->wide = std::min(p->wide, n);
    }
    // Tiles of 64 x 64 where there would be fewer of 128 x 128 than compute units (777 x 1795
    // x 1296, 105 or 377 of them: 27 us or 20; 500 x 5120 x 5120, 160 or 640: 43 and 35; 100 x
    // 34816 x 5120, with 272 of 128: 47, with 1088 of 64 59), and the blocks split where even
    // those are few: up to two workgroups a compute unit, or up to four where there are so many
    // blocks that the join is little beside them. In 1, 2, 3, 4, 6 and 8 splits: 200 x 5120 x
    // 17408 (320 tiles of 136 blocks) 81, 57, 55, 62, 63, 67 us; 256 x 4096 x 8192 (256 of 64) 43, 33,
    // 33, 34, 40, 45; 300 x 1024 x 16384 (80 of 128) 78, 48, 38, 34, 30, 31, in the 12 that this takes
    // 33; 100 x 7168 x 5120 (224 of 40) 29, 25, 26, 27, 32, 34; 70 x 2048 x 4096 (64 of 32) 23, 19,
    // 17, 16, 17, 18; not split: 500 x 5120 x 5120 35, 47, 52, 57; 100 x 17408 x 5120 32, 44, 44, 48.
    // Tiles of 128 in their best number of splits: 53 (3), 33 (4), 35 (8), 26 (4), 19 (6).
    int64_t tiles = ceil_div(m, 128) * ceil_div(n, 128);
    p->tile = tiles < kComputeUnits ? 64 : 128;
    if (tiles > kMaxGroups) return false;
    if (p->tile == 64) {
      tiles = ceil_div(m, 64) * ceil_div(n, 64);
      const int64_t groups = (p->blocks >= 64 ? 4 : 2) * kComputeUnits;
      if (tiles <= groups / 2)
        p->splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(groups / std::max<int64_t>(1, tiles), p->blocks / 8)));
    }
  }
  if (ceil_div(n, 16) > kMaxGroups || ceil_div(m * p->blocks, 16) > kMaxGroups) return false;
  p->code_bytes = round256(static_cast<size_t>(m) * k);
  p->scale_bytes = round256(static_cast<size_t>(m) * p->blocks * sizeof(float));
  p->partial_bytes = p->splits > 1 ? static_cast<size_t>(p->splits) * m * n * sizeof(float) : 0;
  p->total_bytes = m == 0 || n == 0 ? 0 : p->code_bytes + p->scale_bytes + p->partial_bytes;
  return true;
}

qpn_status check_fp8_block_quantize(const void* x, int32_t dtype, int64_t rows, int64_t k, int64_t stride,
                                    int32_t block_rows, const uint8_t* codes, int64_t code_stride, const float* scales,
                                    int64_t scale_row_stride, int64_t scale_block_stride, bool* run) {
  *run = false;
  if (!half_type(dtype) && dtype != QPN_DT_F32) return QPN_ERR_INVALID_ARG;
  if (block_rows != 1 && block_rows != kScaleBlock) return QPN_ERR_INVALID_ARG;
  if (rows < 0 || rows > (1 << 24) || k < 0 || k > (1 << 20)) return QPN_ERR_INVALID_ARG;
  if (!stride_ok(stride) || !stride_ok(code_stride) || code_stride < k || !stride_ok(scale_row_stride) ||
      !stride_ok(scale_block_stride))
    return QPN_ERR_INVALID_ARG;
  if (rows == 0 || k == 0) return QPN_OK;
  const int64_t blocks = ceil_div(rows, block_rows) * ceil_div(k, kScaleBlock);
  if ((block_rows == 1 ? ceil_div(blocks, 16) : blocks) > kMaxGroups) return QPN_ERR_UNSUPPORTED;
  if (!x || !aligned(x, type_size(dtype)) || !codes || !scales || !aligned(scales, 4)) return QPN_ERR_INVALID_ARG;
  *run = true;
  return QPN_OK;
}

qpn_status check_fp8_block_gemm(const qpn_fp8_block_gemm_args* a, const void* ws, size_t ws_bytes, Fp8BlockPlan* p,
                                bool* run) {
  *run = false;
  if (!a) return QPN_ERR_INVALID_ARG;
  const bool codes = a->x_dtype == QPN_DT_E4M3;
  if (!codes && !half_type(a->x_dtype) && a->x_dtype != QPN_DT_F32) return QPN_ERR_INVALID_ARG;
  if (!half_type(a->y_dtype) && a->y_dtype != QPN_DT_F32) return QPN_ERR_INVALID_ARG;
  if (!plan_fp8_block(a->m, a->n, a->k, p)) return QPN_ERR_INVALID_ARG;
  // (a row is at most 2^22 bytes from the next, so that a tile's offsets stay inside 31 bits)
  if (!stride_ok(a->x_stride) || (codes && (a->x_stride % 16 != 0 || a->x_stride > (1 << 22)))) return QPN_ERR_INVALID_ARG;
  if (a->w_stride < a->k || a->w_stride % 16 != 0 || a->w_stride > (1 << 22)) return QPN_ERR_INVALID_ARG;
  if (a->y_stride < a->n || !stride_ok(a->y_stride)) return QPN_ERR_INVALID_ARG;
  if (!stride_ok(a->x_scale_row_stride) || !stride_ok(a->x_scale_block_stride) || !stride_ok(a->w_scale_row_stride) ||
      !stride_ok(a->w_scale_block_stride))
    return QPN_ERR_INVALID_ARG;
  if (codes && a->x_scale_row_stride > (1 << 22)) return QPN_ERR_INVALID_ARG;
  if (codes ? a->x_stride < a->k && a->m > 1 : a->x_scales != nullptr) return QPN_ERR_INVALID_ARG;
  if (a->m == 0 || a->n == 0) return QPN_OK;
  if (!a->y || !aligned(a->y, type_size(a->y_dtype))) return QPN_ERR_INVALID_ARG;
  if (a->k > 0) {
    if (!a->x || !aligned(a->x, codes ? 16 : type_size(a->x_dtype))) return QPN_ERR_INVALID_ARG;
    if (codes && (!a->x_scales || !aligned(a->x_scales, 4))) return QPN_ERR_INVALID_ARG;
    if (!a->w || !aligned(a->w, 16) || !a->w_scales || !aligned(a->w_scales, 4)) return QPN_ERR_INVALID_ARG;
  }
  if (p->total_bytes > 0) {
    if (!ws || !aligned(ws, 16)) return QPN_ERR_INVALID_ARG;
    if (ws_bytes < p->total_bytes) return QPN_ERR_BUFFER_TOO_SMALL;
  }
  *run = true;
  return QPN_OK;
}

qpn_status plan_chunk(const qpn_kv4_cache* c, const qpn_kv4_chunk_args* a, ChunkPlan* p) {
  if (!c || !a || a->reserved != 0) return QPN_ERR_INVALID_ARG;
  if (qpn_kv4_page_bytes(c->page_size, c->kv_heads, c->head_dim) == 0) return QPN_ERR_INVALID_ARG;
  if (a->heads < 1 || a->heads > 65536 || a->heads % c->kv_heads != 0) return QPN_ERR_INVALID_ARG;
  if (a->batch < 0 || a->batch > 65536 || a->rows < 0 || a->rows > (1 << 24) || a->max_q_len < 0 ||
      a->max_q_len > (1 << 20))
    return QPN_ERR_INVALID_ARG;
  // positions and token counts stay inside 32 bits with a step to spare
  if (a->max_kv_len < 0 || a->max_kv_len > (1 << 30) || a->window < 0) return QPN_ERR_INVALID_ARG;
  *p = ChunkPlan{};
  if (a->batch == 0 || a->rows == 0) return QPN_OK;
  const int64_t group = a->heads / c->kv_heads, longest = std::min(a->max_q_len, a->rows);
  // a sequence's rows are counted in 32 bits, its cost in sixteenths of a step
  if (longest * group > (1 << 30)) return QPN_ERR_UNSUPPORTED;
  const int64_t tiles = std::min(a->batch * ceil_div(longest * group, kChunkRows), a->rows * group / kChunkRows + a->batch);
  const int64_t units = tiles * c->kv_heads;
  if (units > kMaxGroups) return QPN_ERR_UNSUPPORTED;
  p->tiles = static_cast<int>(tiles);
  // Steps of a run, at most. A run goes whole, a workgroup each, where it is over before a
  // join would be, or where there are many runs of no great length: heads of 256, 828 runs
  // of 18 steps 206 us whole and 275 in equal shares; heads of 128, 2600 runs of up to 152
  // steps 485 us whole and 335 in shares, 640 of 500 steps 2120 and 1720. Short runs of 128
  // elements a head, whole and shared: 8 runs (5 rows) of 2 steps 12.8 and 16.5 us, of 4 15.5 and
  // 18.4, of 6 18.8 and 18.7, of 8 22.3 and 20.3, of 12 29 and 21; 512 runs of 4 steps 19 and 21, of
  // 8 28 and 31, of 17 48 and 51; 96 runs (4 x 60 rows) of 4 18 and 32, of 8 25 and 35, of 12 32 and 37.
  int64_t steps = ceil_div(a->max_kv_len, kChunkTokens) + ceil_div(longest, kChunkTokens);
  if (a->window > 0) steps = std::min(steps, a->window / kChunkTokens + ceil_div(kChunkRows, group * kChunkTokens) + 2);
  const int64_t room = kComputeUnits * chunk_groups_per_unit(c->head_dim);
  const bool whole = steps <= 8 || (steps <= 64 && units >= 3 * room);
  // (shares are not cut below kMinShare of 4 steps each: see there)
  if (!whole) p->groups = static_cast<int>(std::min<int64_t>(room, ceil_div(units * ceil_div(steps, 4), 8) * 8));
  p->cut_bytes = static_cast<size_t>(p->groups) * 32;
  p->total_bytes = p->cut_bytes + static_cast<size_t>(p->groups) * 2 * kChunkRows * (c->head_dim + 2) * sizeof(float);
  return QPN_OK;
}

qpn_status check_kv4_chunk(const qpn_kv4_cache* c, const qpn_kv4_chunk_args* a, const void* ws, size_t ws_bytes,
                           ChunkPlan* p, bool* run) {
  *run = false;
  qpn_status st = check_kv4_cache(c);
  if (st != QPN_OK) return st;
  st = plan_chunk(c, a, p);
  if (st != QPN_OK) return st;
  if (a->layer < 0 || a->layer >= c->layers || !half_type(a->dtype)) return QPN_ERR_INVALID_ARG;
  if (!isfinite(a->scale) || !(a->scale > 0.0f)) return QPN_ERR_INVALID_ARG;
  if (!stride_ok(a->q_token_stride) || !stride_ok(a->q_head_stride) || !stride_ok(a->k_token_stride) ||
      !stride_ok(a->k_head_stride) || !stride_ok(a->v_token_stride) || !stride_ok(a->v_head_stride))
    return QPN_ERR_INVALID_ARG;
  if (a->table_stride < 0 || a->table_stride > INT32_MAX) return QPN_ERR_INVALID_ARG;
  if (a->table_stride * c->page_size < a->max_kv_len) return QPN_ERR_INVALID_ARG;
  if (!a->q_start && static_cast<int64_t>(a->batch) * a->max_q_len != a->rows) return QPN_ERR_INVALID_ARG;
  if (a->rows > 0 && a->batch == 0) return QPN_ERR_INVALID_ARG;
  if (a->batch == 0 || a->rows == 0) return QPN_OK;
  if (a->max_q_len == 0) return QPN_ERR_INVALID_ARG;
  if (!a->q || !aligned(a->q, 2) || !a->k || !aligned(a->k, 2) || !a->v || !aligned(a->v, 2)) return QPN_ERR_INVALID_ARG;
  if (!a->out || !aligned(a->out, 16) || !aligned(a->lse, 4)) return QPN_ERR_INVALID_ARG;
  if (!a->kv_len || !aligned(a->kv_len, 4) || !aligned(a->q_start, 4)) return QPN_ERR_INVALID_ARG;
  if (a->max_kv_len > 0 && (!a->table || !aligned(a->table, 4))) return QPN_ERR_INVALID_ARG;
  if (p->total_bytes > 0) {
    if (!ws || !aligned(ws, 16)) return QPN_ERR_INVALID_ARG;
    if (ws_bytes < p->total_bytes) return QPN_ERR_BUFFER_TOO_SMALL;
  }
  *run = true;
  return QPN_OK;
}

bool plan_logprobs(int32_t rows, int32_t vocab, int32_t top, LogprobsPlan* p) {
  if (rows < 0 || rows > (1 << 20) || vocab < 1 || vocab > (1 << 24) || top < 0 || top > 64 || top > vocab) return false;
  *p = LogprobsPlan{};
  // as many slices as bring 2048 workgroups, 8 for each compute unit (256 rows of 151936 with
  // five first tokens: 45 us, with 512 or 8192 workgroups 47)
  const int64_t wanted = rows > 0 ? ceil_div(2048, rows) : 1;
  const int64_t most = std::min<int64_t>(ceil_div(vocab, kLogprobsStep), top > 0 ? std::min(kLogprobsSlices, kLogprobsKeys / top) : kLogprobsSlices);
  const int64_t length = ceil_div(ceil_div(vocab, std::min(wanted, most)), kLogprobsStep) * kLogprobsStep;
  p->length = static_cast<int>(length);
  p->slices = static_cast<int>(ceil_div(vocab, length));
  p->stat_bytes = round256(static_cast<size_t>(rows) * p->slices * 24);
  p->total_bytes = rows == 0 ? 0 : p->stat_bytes + static_cast<size_t>(rows) * p->slices * top * 8;
  return true;
}

qpn_status check_token_logprobs(const qpn_logprobs_args* a, const void* ws, size_t ws_bytes, LogprobsPlan* p,
                                bool* run) {
  *run = false;
  if (!a) return QPN_ERR_INVALID_ARG;
  if (!plan_logprobs(a->rows, a->vocab, a->top, p)) return QPN_ERR_INVALID_ARG;
  if (!half_type(a->dtype) && a->dtype != QPN_DT_F32) return QPN_ERR_INVALID_ARG;
  if (!stride_ok(a->row_stride)) return QPN_ERR_INVALID_ARG;
  if (!a->tokens && (a->logprobs || a->rank)) return QPN_ERR_INVALID_ARG;
  if (a->rows == 0) return QPN_OK;
  if (!a->logits || !aligned(a->logits, type_size(a->dtype))) return QPN_ERR_INVALID_ARG;
  if (!aligned(a->tokens, 4) || !aligned(a->temperature, 4) || !aligned(a->logprobs, 4) || !aligned(a->entropy, 4) ||
      !aligned(a->rank, 4) || !aligned(a->top_tokens, 4) || !aligned(a->top_logprobs, 4))
    return QPN_ERR_INVALID_ARG;
  if (a->top > 0 && (!a->top_tokens || !a->top_logprobs)) return QPN_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 16)) return QPN_ERR_INVALID_ARG;
  if (ws_bytes < p->total_bytes) return QPN_ERR_BUFFER_TOO_SMALL;
  *run = true;
  return QPN_OK;
}

}  // namespace qpn

extern "C" {

size_t qpn_token_logprobs_workspace_bytes(int32_t rows, int32_t vocab, int32_t top) {
  qpn::LogprobsPlan p;
  return qpn::plan_logprobs(rows, vocab, top, &p) ? p.total_bytes : 0;
}

size_t qpn_kv4_chunk_workspace_bytes(const qpn_kv4_cache* cache, const qpn_kv4_chunk_args* args) {
  qpn::ChunkPlan p;
  return qpn::plan_chunk(cache, args, &p) == QPN_OK ? p.total_bytes : 0;
}

size_t qpn_fp8_block_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  qpn::Fp8BlockPlan p;
  return qpn::plan_fp8_block(m, n, k, &p) ? p.total_bytes : 0;
}

}  // extern "C"
