// Host-side argument checks and sizes of include/qpn_decode.h, in plain C++
// (no HIP), so that they run under sanitizers without a GPU.
#pragma once

#include "../../include/qpn_decode.h"

namespace qpn {

constexpr int kAttnWaves = 4;   // wavefronts a workgroup
constexpr int kTileTokens = 32; // tokens a wavefront takes at a time
constexpr int kComputeUnits = 256;

// Wavefronts of the attention kernel that a SIMD holds, with nq 16-row tiles
// each: 512 / waves registers hold the output (nq * dim / 4 of them) and what
// a step needs; heads of 256 are kept to 2 by their LDS.
constexpr int attn_waves_per_simd(int dim, int nq) {
  return dim == 256 || nq >= (dim == 64 ? 4 : 3) ? 2 : nq * dim <= 128 ? 4 : 3;
}

// The shape of an attention launch, chosen by plan_attention.
struct AttentionPlan {
  int tiles16;    // 16-row query tiles a wavefront holds (template NQ)
  int row_tiles;  // a sequence's row tiles, at most
  int groups;     // workgroups that share the tiles evenly; 0: a workgroup a run, no join
  int min_share;  // tiles a workgroup takes at least
  size_t cut_bytes, partial_bytes, total_bytes;
};

int64_t kv4_segment_bytes(int page_size, int head_dim);
qpn_status check_kv4_cache(const qpn_kv4_cache* c);
qpn_status check_kv4_append(const qpn_kv4_cache* c, int32_t layer, const void* k, const void* v, int32_t dtype,
                            int64_t tokens, int64_t k_ts, int64_t k_hs, int64_t v_ts, int64_t v_hs,
                            const int64_t* slots, bool* run);
qpn_status check_kv4_read(const qpn_kv4_cache* c, int32_t layer, const int64_t* slots, int64_t tokens, int32_t dtype,
                          const void* k, const void* v, bool* run);
qpn_status check_kv4_copy_pages(const qpn_kv4_cache* c, const int32_t* src, const int32_t* dst, int64_t count,
                                bool* run);
// Sizes only (no pointers): what the workspace query and the launch share.
qpn_status plan_attention(const qpn_kv4_cache* c, const qpn_kv4_attention_args* a, AttentionPlan* p);
qpn_status check_kv4_attention(const qpn_kv4_cache* c, const qpn_kv4_attention_args* a, const void* ws,
                               size_t ws_bytes, AttentionPlan* p, bool* run);

// The shape of a verification: every row is cut into `chunks` pieces of
// `chunk` elements.
struct VerifyPlan {
  int chunk, chunks;
  size_t verdict_bytes, stat_bytes, total_bytes;
};

bool plan_verify(int32_t batch, int32_t drafts, int32_t vocab, VerifyPlan* p);
qpn_status check_verify(const qpn_verify_args* a, const void* ws, size_t ws_bytes, VerifyPlan* p, bool* run);

}  // namespace qpn
