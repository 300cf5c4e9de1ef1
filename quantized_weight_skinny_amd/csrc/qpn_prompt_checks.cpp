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

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

bool plan_fp8_block(int64_t m, int64_t n, int64_t k, Fp8BlockPlan* p) {
  if (m < 0 || m > (1 << 22) || n < 0 || n > (1 << 24) || k < 0 || k > (1 << 20) || k % 16 != 0) return false;
  *p = Fp8BlockPlan{};
  p->blocks = static_cast<int>(ceil_div(k, kScaleBlock));
  p->splits = 1;
  if (m <= 64) {
    p->m_tiles = static_cast<int>(std::max<int64_t>(1, ceil_div(m, 16)));
    p->waves = 4;
    while (p->waves < (p->m_tiles == 4 ? 8 : 16) && ceil_div(n, 16) * p->waves < 2048 && p->blocks >= 8 * p->waves) p->waves *= 2;
  } else {
    p->tile = m > 128 && ceil_div(m, 256) * ceil_div(n, 256) >= 200 ? 256 : 128;
    const int64_t tiles = ceil_div(m, p->tile) * ceil_div(n, p->tile);
    // (fp32 results take tiles of 128 always)
    if (ceil_div(m, 128) * ceil_div(n, 128) > kMaxGroups) return false;
    if (tiles < 256)
      p->splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(512 / std::max<int64_t>(1, tiles), p->blocks / 8)));
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

}  // namespace qpn

extern "C" {

size_t qpn_fp8_block_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  qpn::Fp8BlockPlan p;
  return qpn::plan_fp8_block(m, n, k, &p) ? p.total_bytes : 0;
}

}  // extern "C"
