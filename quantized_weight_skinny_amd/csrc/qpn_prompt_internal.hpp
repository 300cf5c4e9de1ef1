// Host-side launch declarations of the operators of include/qpn_prompt.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qpn_prompt_checks.hpp"

namespace qpn {

hipError_t launch_fp8_block_quantize(const void* x, int32_t dtype, int64_t rows, int64_t k, int64_t stride,
                                     int32_t block_rows, uint8_t* codes, int64_t code_stride, float* scales,
                                     int64_t scale_row_stride, int64_t scale_block_stride, hipStream_t stream);
hipError_t launch_fp8_block_gemm(const qpn_fp8_block_gemm_args& a, const Fp8BlockPlan& p, void* workspace,
                                 hipStream_t stream);
hipError_t launch_kv4_chunk(const qpn_kv4_cache& c, const qpn_kv4_chunk_args& a, const ChunkPlan& p, void* workspace,
                            hipStream_t stream);
hipError_t launch_token_logprobs(const qpn_logprobs_args& a, const LogprobsPlan& p, void* workspace,
                                 hipStream_t stream);

}  // namespace qpn
