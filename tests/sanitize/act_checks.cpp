// act_checks.cpp - drives the host-only plans of the layer calls with an activation over seeded random and extreme
// problems: the outputs' tiles cover every row, column and step once, 128 x 256 tiles never write planes, the workspace's areas end
// where the size says.  With arguments (rows, h_in, h_out, rank, segments: triples of forward and dX) it prints the tiles chosen.
// tests/test_act_plans.py builds it under the address and undefined-behaviour sanitizers.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
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

static int seen[6];

static void check_dense(const DensePlan& d, int64_t M, int64_t N, int64_t steps) {
  CHECK(d.cfg >= 0 && d.cfg <= sgmv::kTile128Wide);
  CHECK((int64_t)d.tiles_m * sgmv::dense_tile_rows(d.cfg) >= M && (int64_t)(d.tiles_m - 1) * sgmv::dense_tile_rows(d.cfg) < M);
  CHECK((int64_t)d.tiles_n * sgmv::dense_tile_cols(d.cfg) >= N && (int64_t)(d.tiles_n - 1) * sgmv::dense_tile_cols(d.cfg) < N);
  CHECK((int64_t)d.ksplit * d.ktiles_per_split >= steps && (d.ksplit == 1 || (int64_t)(d.ksplit - 1) * d.ktiles_per_split < steps));
  CHECK(d.ksplit == 1 || d.to_planes);
  if (d.cfg == sgmv::kTile128Wide) CHECK(!d.to_planes && d.ksplit == 1);
  ++seen[d.cfg];
}

static void check(const sgmv_problem_t& p) {
  size_t forward = 0, backward = 0;
  if (sgmv_layer_workspace_bytes(&p, SGMV_DENSE_ACT_FORWARD, &forward) != SGMV_OK) return;
  CHECK(sgmv_layer_workspace_bytes(&p, SGMV_DENSE_ACT_BACKWARD, &backward) == SGMV_OK);
  const LayerPlan f = plan_layer(p, SGMV_DENSE_ACT_FORWARD);
  CHECK(forward == f.total && f.halves == 1 && !f.row_powers);
  if (p.n_rows > 0) check_dense(f.out, p.n_rows, p.h_out, ceil_div(p.h_in, sgmv::kDenseK));
  CHECK(!f.one_launch || f.out.to_planes);
  CHECK(f.out.term_spread == (f.out.term_in_tile && f.out.ksplit > 1 ? 1 : 0));
  CHECK(!plan_layer(p, SGMV_DENSE_FORWARD).out.term_spread && !plan_act_backward(p, SGMV_ACT_SILU).layer.out.term_spread);
  for (int act : {SGMV_ACT_NONE, SGMV_ACT_RELU, SGMV_ACT_GELU}) {
    const ActPlan a = plan_act_backward(p, act);
    CHECK(a.total <= backward && a.layer.total <= a.planes_off && a.planes_off % 256 == 0);
    CHECK(a.planes_off + (size_t)a.blocks * p.h_out * 4 <= a.total);
    if (p.n_rows == 0) continue;
    check_dense(a.layer.out, (int64_t)p.n_rows * a.layer.halves, p.h_in, ceil_div(p.h_out, sgmv::kDenseK));
    CHECK((int64_t)a.blocks * a.rows_per_block >= p.n_rows && (int64_t)(a.blocks - 1) * a.rows_per_block < p.n_rows);
    CHECK(a.layer.row_powers == (act != SGMV_ACT_NONE && p.dtype == SGMV_F16));
    if (act != SGMV_ACT_NONE) {
      CHECK(a.layer.gate_off[0] + (size_t)p.n_rows * a.layer.halves * p.h_out * 2 <= a.layer.total);
      if (a.layer.row_powers) CHECK(a.layer.row_power_off + round_up(p.n_rows, 32) <= a.layer.total);
    } else {
      CHECK(a.layer.halves == 1);
    }
    CHECK((p.h_out / 8 + 255) / 256 <= 65535);
  }
}

int main(int argc, char** argv) {
  if (argc > 1) {
    for (int i = 1; i + 4 < argc; i += 5) {
      sgmv_problem_t p{SGMV_BF16, std::atoi(argv[i]), std::atoi(argv[i + 1]), std::atoi(argv[i + 2]), std::atoi(argv[i + 3]), 4,
                       std::atoi(argv[i + 4]), std::atoi(argv[i]), 0, 0};
      if (p.num_segs == 0) p.max_seg_len = 0;
      std::printf("%d %d %d %d\n", plan_layer(p, SGMV_DENSE_ACT_FORWARD).out.cfg, plan_act_backward(p, SGMV_ACT_SILU).layer.out.cfg,
                  plan_layer(p, SGMV_DENSE_ACT_FORWARD).out.term_in_tile, plan_layer(p, SGMV_DENSE_ACT_FORWARD).out.term_spread);
    }
    return 0;
  }
  std::mt19937 rng(11);
  const auto log_int = [&](double lo, double hi) {
    return (int32_t)std::exp(std::uniform_real_distribution<double>(std::log(lo), std::log(hi))(rng));
  };
  const int ranks[] = {8, 16, 32, 64};
  for (int i = 0; i < 4000; ++i) {
    const int32_t n = log_int(1, i % 4 ? 9000 : 1 << 27);
    const int32_t segs = i % 3 ? log_int(1, 300) : 0;
    sgmv_problem_t p{(int32_t)(rng() % 2), n, log_int(1, 4000) * 8, log_int(1, 4000) * 8, ranks[rng() % 4], log_int(1, 500), segs,
                     segs ? std::min(n, (int32_t)(n / segs + 1 + rng() % 50)) : 0, 0, 0};
    check(p);
  }
  for (int32_t n : {0, 1, 3, 4, 5, 64, 65, 128, 129, 1 << 30})
    for (int32_t h : {8, 2048, 2056, 1 << 20}) check(sgmv_problem_t{SGMV_F16, n, h, h, 16, 1, 0, 0, 0, 0});
  for (int c : seen) CHECK(c > 0);
  if (failures) {
    std::fprintf(stderr, "%d failures\n", failures);
    return 1;
  }
  std::puts("act checks ok");
  return 0;
}
