// block_checks.cpp - drives the host-only plans of the entry points around a layer over seeded random and extreme
// sizes: every entry and row is some workgroup's, LDS and workspace hold what the kernels write.
// tests/test_block_host.py builds it under the address and undefined-behaviour sanitizers.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <random>

#include "sgmv.h"
#include "sgmv_block_host.h"

using namespace sgmv_host;

static int failures = 0;
#define CHECK(c)                                                                                       \
  do {                                                                                                 \
    if (!(c)) {                                                                                        \
      if (failures < 20) std::fprintf(stderr, "FAIL %s:%d: %s\n", __FILE__, __LINE__, #c);             \
      ++failures;                                                                                      \
    }                                                                                                  \
  } while (0)

static void check_route_plan(int32_t n, int32_t k, int32_t P) {
  size_t bytes = 0;
  if (sgmv_route_workspace_bytes(n, k, P, &bytes) != SGMV_OK) {
    CHECK((int64_t)n * k > SGMV_MAX_LAYER_ROWS || k > SGMV_MAX_TOP_K || P > SGMV_MAX_ROUTE_LORAS);
    return;
  }
  const RoutePlan r = plan_route(n, k, P);
  const int64_t m = (int64_t)n * k, keys = (int64_t)P + 1;
  CHECK(bytes == r.total);
  CHECK(r.waves >= 1 && r.waves <= sgmv::kRouteThreads / 64);
  CHECK((r.waves + 2) * keys <= sgmv::kRouteLds && keys <= sgmv::kRouteLds / 3);
  CHECK(r.tile > 0 && r.tile % (64 * r.waves) == 0);
  CHECK(r.blocks >= 1 && (int64_t)r.blocks * r.tile >= m && (int64_t)(r.blocks - 1) * r.tile < std::max<int64_t>(m, 1));
  CHECK(r.blocks == 1 || (int64_t)r.total >= r.blocks * keys * 4);
  CHECK(r.blocks * keys <= INT32_MAX / 2);
}

static int seen_forward[sgmv::kNormForwardVariants], seen_backward[sgmv::kNormBackwardVariants];

static void check_norm_plan(int32_t n, int32_t w) {
  size_t bytes = 0;
  CHECK(sgmv_layer_norm_workspace_bytes(n, w, &bytes) == SGMV_OK);
  for (int back = 0; back < 2; ++back) {
    const NormPlan p = plan_norm(n, w, back);
    const int variants = back ? sgmv::kNormBackwardVariants : sgmv::kNormForwardVariants;
    CHECK(p.variant >= 0 && p.variant < variants && p.grid >= 1);
    const sgmv::NormVariant v = (back ? sgmv::kNormBackward : sgmv::kNormForward)[p.variant];
    CHECK(v.keep == 0 || v.eights() >= w / 8);
    (back ? seen_backward : seen_forward)[p.variant]++;
    if (!back) {
      CHECK(p.total == 0);
      continue;
    }
    CHECK(bytes == p.total);
    if (n == 0) continue;
    CHECK(p.planes_off + (size_t)p.grid * 2 * w * 4 <= p.total);
    if (v.keep == 0) {
      CHECK(p.stats_off + (size_t)n * 8 <= p.planes_off);
      CHECK((int64_t)p.grid * p.rows_per_block >= n && (int64_t)(p.grid - 1) * p.rows_per_block < n);
      CHECK((w / 8 + 255) / 256 <= 65535);
    }
    CHECK(p.total <= (size_t)n * 8 + ((size_t)80 << 20));  // a fixed budget beside the rows' moments
  }
}

int main() {
  std::mt19937 rng(7);
  const auto log_int = [&](double lo, double hi) {
    return (int32_t)std::exp(std::uniform_real_distribution<double>(std::log(lo), std::log(hi))(rng));
  };
  for (int i = 0; i < 20000; ++i) {
    check_route_plan(log_int(1, 1 << 30), log_int(1, 70), log_int(1, 9000));
    check_norm_plan(log_int(1, 1 << 30), log_int(1, 1 << 17) * 8);
  }
  for (int32_t n : {0, 1, 2047, 2048, 2049, 1 << 24, 1 << 30})
    for (int32_t P : {1, 2, 63, 64, 2498, 2499, 8191, 8192}) check_route_plan(n, 1, P);
  for (int32_t n : {0, 1, 7, 8, 9, 4096, 1 << 30})
    for (int32_t w : {8, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 6144, 6152, 8192, 8200, 12288, 12296, 16384, 16392, 24576, 24584, 1 << 20})
      check_norm_plan(n, w);
  for (int v : seen_forward) CHECK(v > 0);
  for (int v : seen_backward) CHECK(v > 0);
  if (failures) {
    std::fprintf(stderr, "%d failures\n", failures);
    return 1;
  }
  std::puts("block checks ok");
  return 0;
}
