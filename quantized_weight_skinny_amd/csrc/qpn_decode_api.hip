// C ABI of include/qpn_decode.h: the argument checks of qpn_decode_checks.cpp
// on the host, then kernel launches on the caller's stream.
#include "../../include/qpn_decode.h"

#include "qpn_decode_internal.hpp"

namespace {

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

qpn_status from_hip(hipError_t e) { return e == hipSuccess ? QPN_OK : QPN_ERR_HIP; }

}  // namespace

extern "C" {

qpn_status qpn_kv4_append(const qpn_kv4_cache* cache, int32_t layer, const void* k_dev, const void* v_dev,
                          int32_t dtype, int64_t tokens, int64_t k_token_stride, int64_t k_head_stride,
                          int64_t v_token_stride, int64_t v_head_stride, const int64_t* slots_dev, void* stream) {
  bool run = false;
  const qpn_status st = qpn::check_kv4_append(cache, layer, k_dev, v_dev, dtype, tokens, k_token_stride,
                                              k_head_stride, v_token_stride, v_head_stride, slots_dev, &run);
  if (st != QPN_OK || !run) return st;
  return from_hip(qpn::launch_kv4_append(*cache, layer, k_dev, v_dev, dtype, tokens, k_token_stride, k_head_stride,
                                         v_token_stride, v_head_stride, slots_dev, as_stream(stream)));
}

qpn_status qpn_kv4_read(const qpn_kv4_cache* cache, int32_t layer, const int64_t* slots_dev, int64_t tokens,
                        int32_t dtype, void* k_dev, void* v_dev, void* stream) {
  bool run = false;
  const qpn_status st = qpn::check_kv4_read(cache, layer, slots_dev, tokens, dtype, k_dev, v_dev, &run);
  if (st != QPN_OK || !run) return st;
  return from_hip(qpn::launch_kv4_read(*cache, layer, slots_dev, tokens, dtype, k_dev, v_dev, as_stream(stream)));
}

qpn_status qpn_kv4_copy_pages(const qpn_kv4_cache* cache, const int32_t* src_dev, const int32_t* dst_dev,
                              int64_t count, void* stream) {
  bool run = false;
  const qpn_status st = qpn::check_kv4_copy_pages(cache, src_dev, dst_dev, count, &run);
  if (st != QPN_OK || !run) return st;
  return from_hip(qpn::launch_kv4_copy_pages(*cache, src_dev, dst_dev, count, as_stream(stream)));
}

qpn_status qpn_kv4_attention(const qpn_kv4_cache* cache, const qpn_kv4_attention_args* args, void* workspace_dev,
                             size_t workspace_bytes, void* stream) {
  bool run = false;
  qpn::AttentionPlan plan;
  const qpn_status st = qpn::check_kv4_attention(cache, args, workspace_dev, workspace_bytes, &plan, &run);
  if (st != QPN_OK || !run) return st;
  return from_hip(qpn::launch_kv4_attention(*cache, *args, plan, workspace_dev, as_stream(stream)));
}

qpn_status qpn_verify(const qpn_verify_args* args, void* workspace_dev, size_t workspace_bytes, void* stream) {
  bool run = false;
  qpn::VerifyPlan plan;
  const qpn_status st = qpn::check_verify(args, workspace_dev, workspace_bytes, &plan, &run);
  if (st != QPN_OK || !run) return st;
  return from_hip(qpn::launch_verify(*args, plan, workspace_dev, as_stream(stream)));
}

}  // extern "C"
