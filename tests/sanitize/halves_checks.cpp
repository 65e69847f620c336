// halves_checks.cpp - drives the plans of the activation's backward call with dZ in two halves (SGMV_DZ_HALVES) over seeded random
// and extreme problems: dX's tiles cover both halves' rows, every area of the workspace ends where the size says, and small
// problems keep the plan that they have without.  tests/test_act_halves_host.py builds it under the sanitizers.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <random>

#include "sgmv.h"
#include "sgmv_layer_host.h"

using namespace sgmv_host;

static int failures = 0;
#define CHECK(c)                                                                                       \
  do {                                                                                                 \
    if (!(c)) {                                                                                        \
      if (failures < 20) std::fprintf(stderr, "FAIL %s:%d: %s\n", __FILE__, __LINE__, #c);             \
      ++failures;                                                                                      \
    }                                                                                                  \
  } while (0)

static void check(const sgmv_problem_t& p) {
  size_t bytes = 0;
  const int32_t op = SGMV_DENSE_ACT_BACKWARD | SGMV_DZ_HALVES;
  const sgmv_status_t st = sgmv_layer_workspace_bytes(&p, op, &bytes);
  if (p.n_rows > SGMV_MAX_LAYER_ROWS / 2) CHECK(st == SGMV_ERR_UNSUPPORTED);
  if (st != SGMV_OK) return;
  for (int act : {SGMV_ACT_NONE, SGMV_ACT_RELU, SGMV_ACT_GELU}) {
    const ActPlan a = plan_act_backward(p, act, true), plain = plan_act_backward(p, act);
    const LayerPlan& l = a.layer;
    CHECK(a.total <= bytes && l.total <= a.planes_off);
    CHECK(a.planes_off + (size_t)a.blocks * p.h_out * 4 <= a.total);
    CHECK(l.halves == (act == SGMV_ACT_NONE ? 1 : 2));
    if (l.halves == plain.layer.halves) {
      CHECK(a.total == plain.total && l.out.cfg == plain.layer.out.cfg && l.out.ksplit == plain.layer.out.ksplit);
      continue;
    }
    if (p.n_rows == 0) continue;
    const int64_t n = p.n_rows, M = 2 * n, steps = ceil_div(p.h_out, sgmv::kDenseK);
    const DensePlan& d = l.out;
    CHECK(d.cfg >= 0 && d.cfg != sgmv::kTile128Wide && d.to_planes);
    CHECK((int64_t)d.tiles_m * sgmv::dense_tile_rows(d.cfg) >= M && (int64_t)(d.tiles_m - 1) * sgmv::dense_tile_rows(d.cfg) < M);
    CHECK((int64_t)d.ksplit * d.ktiles_per_split >= steps);
    CHECK(d.plane_bytes == (size_t)d.ksplit * M * p.h_in * 4 && l.planes_off + d.plane_bytes <= l.total);
    CHECK(l.gate_off[0] + (size_t)M * p.h_out * 2 <= l.total);
    if (l.row_powers) CHECK(l.row_power_off + round_up(n, 32) <= l.total);
    if (l.lora) {
      CHECK(l.up.planes == 2 * l.up.ksplit);
      CHECK(l.thin_off[1][0] + (size_t)l.up.planes * n * p.rank * 4 <= l.total);
    }
  }
}

int main() {
  std::mt19937 rng(13);
  const auto log_int = [&](double lo, double hi) {
    return (int32_t)std::exp(std::uniform_real_distribution<double>(std::log(lo), std::log(hi))(rng));
  };
  const int ranks[] = {8, 16, 32, 64};
  for (int i = 0; i < 4000; ++i) {
    const int32_t n = log_int(1, i % 4 ? 9000 : 1 << 27);
    const int32_t segs = i % 3 ? log_int(1, 300) : 0;
    check(sgmv_problem_t{(int32_t)(rng() % 2), n, log_int(1, 4000) * 8, log_int(1, 4000) * 8, ranks[rng() % 4], log_int(1, 500), segs,
                         segs ? std::min(n, (int32_t)(n / segs + 1 + rng() % 50)) : 0, 0, 0});
  }
  for (int32_t n : {0, 1, 128, 129, 1 << 29, (1 << 29) + 1, 1 << 30})
    for (int32_t h : {8, 2048, 2056, 1 << 20}) check(sgmv_problem_t{SGMV_F16, n, h, h, 16, 1, 0, 0, 0, 0});
  if (failures) {
    std::fprintf(stderr, "%d failures\n", failures);
    return 1;
  }
  std::puts("halves checks ok");
  return 0;
}
