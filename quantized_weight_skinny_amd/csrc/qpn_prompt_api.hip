// C ABI of include/qpn_prompt.h: the argument checks of qpn_prompt_checks.cpp
// on the host, then kernel launches on the caller's stream.
#include "../../include/qpn_prompt.h"

#include "qpn_prompt_internal.hpp"

namespace {

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

qpn_status from_hip(hipError_t e) { return e == hipSuccess ? QPN_OK : QPN_ERR_HIP; }

}  // namespace

extern "C" {

qpn_status qpn_fp8_block_quantize(const void* x_dev, int32_t dtype, int64_t rows, int64_t k, int64_t stride,
                                  int32_t block_rows, uint8_t* codes_dev, int64_t code_stride, float* scales_dev,
                                  int64_t scale_row_stride, int64_t scale_block_stride, void* stream) {
  bool run = false;
  const qpn_status st = qpn::check_fp8_block_quantize(x_dev, dtype, rows, k, stride, block_rows, codes_dev, code_stride,
                                                      scales_dev, scale_row_stride, scale_block_stride, &run);
  if (st != QPN_OK || !run) return st;
  return from_hip(qpn::launch_fp8_block_quantize(x_dev, dtype, rows, k, stride, block_rows, codes_dev, code_stride,
                                                 scales_dev, scale_row_stride, scale_block_stride, as_stream(stream)));
}

qpn_status qpn_fp8_block_gemm(const qpn_fp8_block_gemm_args* args, void* workspace_dev, size_t workspace_bytes,
                              void* stream) {
  bool run = false;
  qpn::Fp8BlockPlan plan;
  const qpn_status st = qpn::check_fp8_block_gemm(args, workspace_dev, workspace_bytes, &plan, &run);
  if (st != QPN_OK || !run) return st;
  return from_hip(qpn::launch_fp8_block_gemm(*args, plan, workspace_dev, as_stream(stream)));
}

qpn_status qpn_kv4_chunk_attention(const qpn_kv4_cache* cache, const qpn_kv4_chunk_args* args, void* workspace_dev,
                                   size_t workspace_bytes, void* stream) {
  bool run = false;
  qpn::ChunkPlan plan;
  const qpn_status st = qpn::check_kv4_chunk(cache, args, workspace_dev, workspace_bytes, &plan, &run);
  if (st != QPN_OK || !run) return st;
  return from_hip(qpn::launch_kv4_chunk(*cache, *args, plan, workspace_dev, as_stream(stream)));
}

qpn_status qpn_token_logprobs(const qpn_logprobs_args* args, void* workspace_dev, size_t workspace_bytes,
                              void* stream) {
  bool run = false;
  qpn::LogprobsPlan plan;
  const qpn_status st = qpn::check_token_logprobs(args, workspace_dev, workspace_bytes, &plan, &run);
  if (st != QPN_OK || !run) return st;
  return from_hip(qpn::launch_token_logprobs(*args, plan, workspace_dev, as_stream(stream)));
}

}  // extern "C"
