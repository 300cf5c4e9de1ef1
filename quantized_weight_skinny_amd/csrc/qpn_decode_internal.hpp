// Host-side launch declarations of the operators of include/qpn_decode.h, and
// the device-side addressing of the 4-bit cache that they share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qpn_decode_checks.hpp"

namespace qpn {

// Byte offset, among the 16 lanes' V codes of four tokens (2 D bytes) of quad
// g, of lane i's: [quad][i][token][D / 32].
template <int DIM>
__device__ __forceinline__ int lane_v(int i, int g) {
  return g * (2 * DIM) + i * (DIM / 8);
}

// fp32 -> fp16 or bf16 bits, nearest with ties to even; NaN stays NaN.
template <bool BF16>
__device__ __forceinline__ uint16_t round16(float x) {
  if constexpr (BF16) {
    const uint32_t b = __float_as_uint(x);
    if ((b & 0x7FFFFFFFu) > 0x7F800000u) return static_cast<uint16_t>((b >> 16) | 0x40u);
    return static_cast<uint16_t>((b + 0x7FFFu + ((b >> 16) & 1u)) >> 16);
  } else {
    return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
  }
}

// fp16 or bf16 bits -> fp32, exact.
template <bool BF16>
__device__ __forceinline__ float widen16(uint32_t bits) {
  if constexpr (BF16)
    return __uint_as_float(bits << 16);
  else
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(bits)));
}

hipError_t launch_kv4_attention(const qpn_kv4_cache& c, const qpn_kv4_attention_args& a, const AttentionPlan& p,
                                void* workspace, hipStream_t stream);
hipError_t launch_kv4_append(const qpn_kv4_cache& c, int32_t layer, const void* k, const void* v, int32_t dtype,
                             int64_t tokens, int64_t k_ts, int64_t k_hs, int64_t v_ts, int64_t v_hs,
                             const int64_t* slots, hipStream_t stream);
hipError_t launch_kv4_read(const qpn_kv4_cache& c, int32_t layer, const int64_t* slots, int64_t tokens, int32_t dtype,
                           void* k, void* v, hipStream_t stream);
hipError_t launch_kv4_copy_pages(const qpn_kv4_cache& c, const int32_t* src, const int32_t* dst, int64_t count,
                                 hipStream_t stream);
hipError_t launch_verify(const qpn_verify_args& a, const VerifyPlan& p, void* workspace, hipStream_t stream);

}  // namespace qpn
