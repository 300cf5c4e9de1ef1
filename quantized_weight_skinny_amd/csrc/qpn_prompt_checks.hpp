// Host-side argument checks and sizes of include/qpn_prompt.h, in plain C++
// (no HIP), so that they run under sanitizers without a GPU.
#pragma once

#include "../../include/qpn_prompt.h"
#include "qpn_decode_checks.hpp"

namespace qpn {

constexpr int kScaleBlock = 128;  // elements along k (and rows of a weight) under one scale

// Wavefronts of a few-rows workgroup, at most: two blocks each of both operands
// have to fit LDS.
constexpr int few_rows_waves(int m_tiles) { return m_tiles == 1 ? 16 : m_tiles < 4 ? 8 : 4; }

// The shape of a block product, chosen by plan_fp8_block.
struct Fp8BlockPlan {
  int m_tiles;       // > 0: a wavefront takes all rows, this many tiles of 16; 0: tiles in LDS
  int waves;         // wavefronts of a workgroup that share k (m_tiles > 0)
  int tile;          // 128 or 64: rows and outputs of an LDS tile
  int64_t wide;      // outputs up to here in tiles of 256 x 256 instead (fp32 results: none)
  int splits;        // k ranges, each to partial sums of its own; 1: none
  int blocks;        // ceil(k / 128)
  size_t code_bytes, scale_bytes, partial_bytes, total_bytes;
};

// Sizes only: what the workspace query and the launch share. False: refused.
bool plan_fp8_block(int64_t m, int64_t n, int64_t k, Fp8BlockPlan* p);
qpn_status check_fp8_block_quantize(const void* x, int32_t dtype, int64_t rows, int64_t k, int64_t stride,
                                    int32_t block_rows, const uint8_t* codes, int64_t code_stride, const float* scales,
                                    int64_t scale_row_stride, int64_t scale_block_stride, bool* run);
qpn_status check_fp8_block_gemm(const qpn_fp8_block_gemm_args* a, const void* ws, size_t ws_bytes, Fp8BlockPlan* p,
                                bool* run);

constexpr int kChunkRows = 128;   // query rows (tokens x heads of a group) of a workgroup
constexpr int kChunkTokens = 64;  // tokens it takes at a time

// Workgroups of the attention kernel that a compute unit holds.
constexpr int chunk_groups_per_unit(int dim) { return dim == 256 ? 1 : 2; }

// The shape of a chunk attention.
struct ChunkPlan {
  int tiles;   // row tiles of all sequences, at most
  int groups;  // workgroups that share the work evenly, a multiple of 8; 0: a workgroup a row tile and kv head, no join
  size_t cut_bytes, total_bytes;
};

qpn_status plan_chunk(const qpn_kv4_cache* c, const qpn_kv4_chunk_args* a, ChunkPlan* p);
qpn_status check_kv4_chunk(const qpn_kv4_cache* c, const qpn_kv4_chunk_args* a, const void* ws, size_t ws_bytes,
                           ChunkPlan* p, bool* run);

constexpr int kLogprobsStep = 4096;   // elements of a row that a workgroup takes at a time
constexpr int kLogprobsKeys = 2048;   // first tokens of a row's slices, at most
constexpr int kLogprobsSlices = 128;  // slices of a row, at most

// The shape of token log-probabilities: every row in `slices` of `length`.
struct LogprobsPlan {
  int slices, length;
  size_t stat_bytes, total_bytes;
};

bool plan_logprobs(int32_t rows, int32_t vocab, int32_t top, LogprobsPlan* p);
qpn_status check_token_logprobs(const qpn_logprobs_args* a, const void* ws, size_t ws_bytes, LogprobsPlan* p,
                                bool* run);

}  // namespace qpn
