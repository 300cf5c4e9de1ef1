// Host checks of qpn_prompt_checks.cpp under AddressSanitizer and
// UndefinedBehaviorSanitizer: every plan over wide ranges of sizes, extremes
// among them, satisfies what the kernels assume, and the checks refuse without
// reading through a device pointer. Prints "ok <plans>".
#include <limits.h>
#include <stdio.h>
#include <stdlib.h>

#include <initializer_list>

#include "../../quantized_weight_skinny_amd/csrc/qpn_plan.hpp"
#include "../../quantized_weight_skinny_amd/csrc/qpn_prompt_checks.hpp"

#define CHECK(x)                                             \
  do {                                                       \
    if (!(x)) {                                              \
      fprintf(stderr, "FAILED %s:%d: %s\n", __FILE__, __LINE__, #x); \
      exit(1);                                               \
    }                                                        \
  } while (0)

using qpn::ceil_div;

int main() {
  long plans = 0;
  const int64_t most_groups = int64_t(1) << 23;
  // products
  for (int64_t m : {0, 1, 15, 16, 17, 48, 49, 64, 65, 128, 255, 256, 257, 777, 2048, 70000, 1 << 22})
    for (int64_t n : {0, 1, 16, 17, 130, 5120, 33000, 151936, 1 << 24})
      for (int64_t k : {0, 16, 112, 128, 144, 1296, 17408, 1 << 20}) {
        qpn::Fp8BlockPlan p;
        if (!qpn::plan_fp8_block(m, n, k, &p)) {
          CHECK(qpn_fp8_block_workspace_bytes(m, n, k) == 0);
          continue;
        }
        ++plans;
        CHECK(p.blocks == ceil_div(k, 128) && p.splits >= 1 && (p.splits == 1 || p.splits <= p.blocks));
        CHECK(p.code_bytes >= static_cast<size_t>(m * k) && p.code_bytes % 256 == 0);
        CHECK(p.scale_bytes >= static_cast<size_t>(m * p.blocks * 4) && p.scale_bytes % 256 == 0);
        CHECK(qpn_fp8_block_workspace_bytes(m, n, k) == p.total_bytes);
        CHECK(m > 48 || p.m_tiles > 0);
        CHECK(m <= 64 || p.m_tiles == 0);
        if (p.m_tiles > 0) {
          CHECK(p.m_tiles >= 1 && p.m_tiles <= 4 && p.m_tiles * 16 >= m && p.splits == 1);
          CHECK(p.waves == 4 || p.waves == 8 || p.waves == 16);
          CHECK(p.waves <= qpn::few_rows_waves(p.m_tiles) && ceil_div(n, 16) <= most_groups);
          CHECK(p.waves * 2 * ((1 + p.m_tiles) * 2048 + 256) <= 160 * 1024);  // its LDS
        } else {
          CHECK(p.tile == 64 || p.tile == 128);
          CHECK(ceil_div(m, p.tile) * ceil_div(n, p.tile) + 8 <= most_groups + 8);
          CHECK(p.wide >= 0 && p.wide <= n && (p.wide == n || p.wide % 256 == 0));
          CHECK(p.wide == 0 || (m >= 256 && p.splits == 1 && p.tile == 128));
          CHECK(p.partial_bytes == (p.splits > 1 ? static_cast<size_t>(p.splits) * m * n * 4 : 0));
        }
      }
  for (int64_t k : {8, 24, (1 << 20) + 16, -16}) {
    qpn::Fp8BlockPlan p;
    CHECK(!qpn::plan_fp8_block(4, 4, k, &p));
  }
  // attention
  for (int32_t dim : {64, 128, 256})
    for (int32_t kvh : {1, 2, 8, 1024})
      for (int32_t group : {1, 3, 5, 16, 64})
        for (int32_t ql : {1, 2, 100, 2048, 1 << 20})
          for (int32_t kv : {0, 1, 513, 131072, 1 << 30})
            for (int32_t batch : {0, 1, 7, 65, 65536})
              for (int32_t window : {0, 1, 100, INT32_MAX}) {
                qpn_kv4_cache c{reinterpret_cast<void*>(4096), 1000, 1, 64, kvh, dim, 1.f, 1.f};
                qpn_kv4_chunk_args a{};
                a.heads = static_cast<int64_t>(kvh) * group > 65536 ? 65536 / kvh * kvh : kvh * group;
                a.batch = batch;
                a.rows = static_cast<int64_t>(batch) * ql > (1 << 24) ? 1 << 24 : batch * ql;
                a.max_q_len = ql, a.max_kv_len = kv, a.window = window;
                qpn::ChunkPlan p;
                const qpn_status st = qpn::plan_chunk(&c, &a, &p);
                CHECK(st == QPN_OK || st == QPN_ERR_UNSUPPORTED);
                if (st != QPN_OK) {
                  CHECK(qpn_kv4_chunk_workspace_bytes(&c, &a) == 0);
                  continue;
                }
                ++plans;
                CHECK(qpn_kv4_chunk_workspace_bytes(&c, &a) == p.total_bytes);
                if (batch == 0) {
                  CHECK(p.total_bytes == 0);
                  continue;
                }
                const int64_t group_rows = static_cast<int64_t>(ql < a.rows ? ql : a.rows) * (a.heads / kvh);
                CHECK(static_cast<int64_t>(p.tiles) * 128 >= group_rows && static_cast<int64_t>(p.tiles) * kvh <= most_groups);
                CHECK(p.groups % 8 == 0 && p.groups <= 512);
                CHECK(p.total_bytes == static_cast<size_t>(p.groups) * (32 + 2 * 128 * (static_cast<size_t>(dim) + 2) * 4));
                // a window needs no more workspace than none, which the torch layer asks for
                a.window = 0;
                CHECK(qpn_kv4_chunk_workspace_bytes(&c, &a) >= p.total_bytes);
              }
  // log-probabilities
  for (int32_t rows : {0, 1, 37, 2047, 2048, 2049, 1 << 20})
    for (int32_t vocab : {1, 63, 64, 4096, 4097, 151936, 1 << 24})
      for (int32_t top : {0, 1, 20, 33, 64}) {
        qpn::LogprobsPlan p;
        if (!qpn::plan_logprobs(rows, vocab, top, &p)) {
          CHECK(top > vocab);
          continue;
        }
        ++plans;
        CHECK(p.length % qpn::kLogprobsStep == 0 && static_cast<int64_t>(p.slices) * p.length >= vocab);
        CHECK(static_cast<int64_t>(p.slices - 1) * p.length < vocab && p.slices <= qpn::kLogprobsSlices);
        CHECK(p.slices * top <= qpn::kLogprobsKeys && static_cast<int64_t>(rows) * p.slices <= most_groups);
        CHECK(p.stat_bytes % 8 == 0 && p.stat_bytes >= static_cast<size_t>(rows) * p.slices * 24);
        CHECK(p.total_bytes == (rows ? p.stat_bytes + static_cast<size_t>(rows) * p.slices * top * 8 : 0));
        CHECK(qpn_token_logprobs_workspace_bytes(rows, vocab, top) == p.total_bytes);
      }
  printf("ok %ld\n", plans);
  return 0;
}
