// Host checks of qpn_decode_checks.cpp under AddressSanitizer and
// UndefinedBehaviorSanitizer: every plan over wide ranges of sizes, extremes
// among them, satisfies what the kernels assume, and the checks refuse without
// reading through a device pointer. Prints "ok <plans>".
#include <limits.h>
#include <math.h>
#include <stdio.h>
#include <stdlib.h>

#include "../../quantized_weight_skinny_amd/csrc/qpn_decode_checks.hpp"

#define CHECK(x)                                             \
  do {                                                       \
    if (!(x)) {                                              \
      fprintf(stderr, "FAILED %s:%d: %s\n", __FILE__, __LINE__, #x); \
      exit(1);                                               \
    }                                                        \
  } while (0)

int main() {
  long plans = 0;
  const int32_t dims[] = {64, 128, 256}, heads[] = {1, 2, 8, 1024}, groups[] = {1, 3, 5, 16, 64};
  const int32_t q_lens[] = {1, 2, 8, 16, 100, 65536}, kv_lens[] = {0, 1, 512, 513, 131072, 1 << 30};
  const int32_t batches[] = {0, 1, 7, 64, 65, 4096, 65536}, pages[] = {16, 64, 256};
  for (int32_t dim : dims)
    for (int32_t kvh : heads)
      for (int32_t group : groups)
        for (int32_t ql : q_lens)
          for (int32_t kv : kv_lens)
            for (int32_t batch : batches)
              for (int32_t page : pages) {
                qpn_kv4_cache c{reinterpret_cast<void*>(4096), 1000, 1, page, kvh, dim, 1.f, 1.f};
                qpn_kv4_attention_args a{};
                a.heads = static_cast<int64_t>(kvh) * group > 65536 ? 65536 / kvh * kvh : kvh * group;
                a.batch = batch;
                a.rows = static_cast<int64_t>(batch) * ql > INT32_MAX ? INT32_MAX : batch * ql;
                a.max_q_len = ql, a.max_kv_len = kv;
                qpn::AttentionPlan p;
                const qpn_status st = qpn::plan_attention(&c, &a, &p);
                CHECK(st == QPN_OK || st == QPN_ERR_UNSUPPORTED);
                if (st != QPN_OK) {
                  CHECK(qpn_kv4_attention_workspace_bytes(&c, &a) == 0);
                  continue;
                }
                ++plans;
                const int64_t rows = static_cast<int64_t>(ql < a.rows ? ql : a.rows) * (a.heads / kvh);
                CHECK(p.tiles16 >= 1 && p.tiles16 <= (dim == 256 ? 2 : dim == 128 ? 3 : 4));
                CHECK(static_cast<int64_t>(p.row_tiles) * p.tiles16 * 16 >= rows);
                CHECK(rows == 0 || static_cast<int64_t>(p.row_tiles - 1) * p.tiles16 * 16 < rows);
                CHECK(p.groups == 0 || (p.groups % 256 == 0 && p.groups <= 1024));
                // every position on the line, and groups * share, stay below 2^31
                const int64_t line = static_cast<int64_t>(batch) * p.row_tiles * kvh * ((static_cast<int64_t>(kv) + 31) / 32 + 64);
                CHECK(line + 2 * p.groups + p.min_share * static_cast<int64_t>(p.groups) <= INT32_MAX);
                const size_t piece = static_cast<size_t>(16) * p.tiles16 * (dim + 2) * 4;
                CHECK(p.partial_bytes == 2 * static_cast<size_t>(p.groups) * piece);
                CHECK(p.cut_bytes == static_cast<size_t>(p.groups) * 32);
                CHECK(p.total_bytes == 0 || p.total_bytes == p.cut_bytes + p.partial_bytes);
                CHECK((p.total_bytes == 0) == (p.groups == 0 || batch == 0 || a.rows == 0));
                CHECK(qpn_kv4_attention_workspace_bytes(&c, &a) == p.total_bytes);
              }
  const int32_t vocabs[] = {1, 2, 4095, 4096, 4097, 151936, 1 << 24}, drafts[] = {0, 1, 7, 64};
  for (int32_t vocab : vocabs)
    for (int32_t n : drafts)
      for (int32_t batch : batches) {
        qpn::VerifyPlan p;
        if (!qpn::plan_verify(batch, n, vocab, &p)) {
          CHECK(qpn_verify_workspace_bytes(batch, n, vocab) == 0);
          continue;
        }
        ++plans;
        CHECK(p.chunk == 4096 && static_cast<int64_t>(p.chunks) * p.chunk >= vocab);
        CHECK(static_cast<int64_t>(p.chunks - 1) * p.chunk < vocab);
        const int64_t rows = static_cast<int64_t>(batch) * (2 * n + 1);
        CHECK(rows * p.chunks <= (1 << 23) && static_cast<int64_t>(batch) * p.chunks <= (1 << 21));
        CHECK(p.stat_bytes == static_cast<size_t>(rows) * p.chunks * 16);
        CHECK(p.total_bytes >= p.verdict_bytes + p.stat_bytes + static_cast<size_t>(batch) * p.chunks * 24);
        CHECK(p.verdict_bytes % 16 == 0 && p.stat_bytes % 16 == 0);
      }
  // refusals look at no device pointer (these point nowhere)
  qpn_kv4_cache c{reinterpret_cast<void*>(4096), 10, 2, 64, 8, 128, 1.f, 1.f};
  bool run = true;
  CHECK(qpn::check_kv4_append(&c, 2, reinterpret_cast<void*>(16), reinterpret_cast<void*>(16), QPN_DT_F16, 1, 0, 0, 0, 0,
                              reinterpret_cast<int64_t*>(16), &run) == QPN_ERR_INVALID_ARG && !run);
  CHECK(qpn::check_kv4_append(&c, 1, reinterpret_cast<void*>(16), reinterpret_cast<void*>(16), QPN_DT_F16, 1, 0, 0, 0, 0,
                              reinterpret_cast<int64_t*>(16), &run) == QPN_OK && run);
  CHECK(qpn::check_kv4_copy_pages(&c, nullptr, nullptr, 0, &run) == QPN_OK && !run);
  CHECK(qpn::check_kv4_read(&c, 0, nullptr, 0, QPN_DT_F32, nullptr, nullptr, &run) == QPN_OK && !run);
  c.k_scale = NAN;
  CHECK(qpn::check_kv4_cache(&c) == QPN_ERR_INVALID_ARG);
  CHECK(qpn::check_kv4_cache(nullptr) == QPN_ERR_INVALID_ARG);
  qpn::AttentionPlan ap;
  CHECK(qpn::check_kv4_attention(nullptr, nullptr, nullptr, 0, &ap, &run) == QPN_ERR_INVALID_ARG);
  qpn::VerifyPlan vp;
  CHECK(qpn::check_verify(nullptr, nullptr, 0, &vp, &run) == QPN_ERR_INVALID_ARG);
  printf("ok %ld\n", plans);
  return 0;
}
