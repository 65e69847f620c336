// layer_checks.cpp - drives the host-only plans of the layer entry points over
// seeded random and extreme problems: every output element and contraction
// step is covered once, the workspace's areas do not overlap and end where the
// size says.  tests/test_layer_sanitizers.py builds it with the library's
// host-only sources under the address and undefined-behaviour sanitizers.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <random>
#include <utility>
#include <vector>

#include "sgmv.h"
#include "sgmv_layer_host.h"

using namespace sgmv_host;

static int failures = 0;
#define CHECK(c)                                                          \
  do {                                                                    \
    if (!(c)) {                                                           \
      if (failures < 20) std::fprintf(stderr, "FAIL %s:%d: %s\n", __FILE__, __LINE__, #c); \
      ++failures;                                                         \
    }                                                                     \
  } while (0)

static int seen_cfg[5], seen_split, seen_one_launch, seen_in_tile;

static void check_dense(const DensePlan& d, int64_t M, int64_t N, int64_t steps, int cols) {
  CHECK(d.cfg >= 0 && d.cfg <= 4);
  CHECK((int64_t)d.tiles_m * sgmv::dense_tile_rows(d.cfg) >= M);
  CHECK((int64_t)(d.tiles_m - 1) * sgmv::dense_tile_rows(d.cfg) < std::max<int64_t>(M, 1));
  const int64_t c = sgmv::dense_tile_cols(d.cfg) / cols;
  CHECK((int64_t)d.tiles_n * c >= N && (int64_t)(d.tiles_n - 1) * c < N);
  CHECK(d.ksplit >= 1 && d.ksplit <= 16 && d.ktiles_per_split >= 1);
  CHECK((int64_t)d.ksplit * d.ktiles_per_split >= steps);
  CHECK(d.ksplit == 1 || (int64_t)(d.ksplit - 1) * d.ktiles_per_split < steps);  // no empty split
  ++seen_cfg[d.cfg];
  seen_split += d.ksplit > 1;
}

static void check_problem(const sgmv_problem_t& p, int op) {
  size_t bytes = 0;
  if (sgmv_layer_workspace_bytes(&p, op, &bytes) != SGMV_OK) {
    CHECK(sgmv_check_problem(&p) != SGMV_OK || p.n_rows > SGMV_MAX_LAYER_ROWS);
    return;
  }
  const LayerPlan l = plan_layer(p, op);
  CHECK(bytes == l.total);
  const bool back = layer_backward(op), gated = layer_gated(op);
  const int64_t n = p.n_rows;
  if (n > 0) {
    const int64_t kt = ceil_div(back ? p.h_out : p.h_in, sgmv::kDenseK) * (op == SGMV_GATED_BACKWARD ? 2 : 1);
    check_dense(l.out, n * l.halves, back ? p.h_in : p.h_out, kt, op == SGMV_GATED_FORWARD ? 2 : 1);
    CHECK(l.out.ksplit == 1 || l.out.to_planes);
    CHECK(l.halves == 1 || (op == SGMV_GATED_BACKWARD && l.out.to_planes));
    CHECK(!l.lora || l.out.term_in_tile || l.out.to_planes);  // the term is added somewhere
    seen_one_launch += l.one_launch;
    seen_in_tile += l.out.term_in_tile;
  }
  if (back) {
    check_dense(l.dw, p.h_in, p.h_out, ceil_div(n, sgmv::kDenseK), 1);
    CHECK(l.dw.ksplit == 1 && l.dw.cfg <= sgmv::kTile128);
    CHECK(l.nsplit_a >= 1 && l.nsplit_a <= 64 && l.nsplit_b >= 1 && l.nsplit_b <= 64);
  }
  // Areas: each inside the workspace, none over another.
  std::vector<std::pair<size_t, size_t>> area;  // offset, bytes
  const auto add = [&](size_t off, size_t size) {
    if (size > 0) area.push_back({off, size});
  };
  if (l.lora) {
    const size_t v = (size_t)n * p.rank * 4;
    for (int i = 0; i < l.projections; ++i)
      for (int d = 0; d < (back ? 2 : 1); ++d) {
        const ThinPlan& t = d ? l.up : l.down;
        const int64_t K = d ? p.h_out : p.h_in;
        CHECK(t.ksplit >= 1 && t.kc % sgmv::kDenseK == 0 && (int64_t)t.ksplit * t.kc >= K && (int64_t)(t.ksplit - 1) * t.kc < K);
        CHECK(t.units >= 1 && (int64_t)t.units * sgmv::kThinRows >= std::min<int64_t>(n, p.max_seg_len));
        add(l.v_off[d][i], v);
        add(l.half_off[d][i], v);
        add(l.row_scale_off[d][i], (size_t)n * 4);
        const int sum = t.ksplit * (d ? l.halves : 1);
        CHECK(t.planes == (sum > 1 ? sum : 0));
        add(l.thin_off[d][i], (size_t)t.planes * v);
      }
    if (l.one_launch) add(l.row_k_off, (size_t)n * 4);
  }
  if (op == SGMV_GATED_BACKWARD)
    for (int i = 0; i < 2; ++i) add(l.gate_off[i], (size_t)n * l.halves * p.h_out * 2);
  const size_t out = l.out.to_planes ? (size_t)l.out.ksplit * n * l.halves * (back ? p.h_in : p.h_out) * 4 * (gated && !back ? 2 : 1) : 0;
  size_t grads = 0;
  if (back && l.lora) {
    if (l.nsplit_a > 1) grads += (size_t)l.nsplit_a * p.num_loras * p.h_in * p.rank * 4 * l.projections;
    if (l.nsplit_b > 1) grads += (size_t)l.nsplit_b * p.num_loras * p.h_out * p.rank * 4 * l.projections;
  }
  add(l.planes_off, std::max(out, grads));
  std::sort(area.begin(), area.end());
  for (size_t i = 0; i < area.size(); ++i) {
    CHECK(area[i].first % 256 == 0);
    CHECK(area[i].first + area[i].second <= (i + 1 < area.size() ? area[i + 1].first : l.total));
  }
}

int main() {
  std::mt19937_64 rng(7);
  const auto pick = [&](int64_t lo, int64_t hi) {  // spread over the logarithm
    const double u = (double)(rng() >> 11) / 9007199254740992.0;
    double v = (double)lo;
    for (double f = u; v < (double)hi && f > 0; f -= 0.02) v *= 1.0 + 0.02 * 0.69 * 20;
    return std::min<int64_t>(hi, std::max<int64_t>(lo, (int64_t)v));
  };
  const int ranks[] = {8, 16, 32, 64};
  for (int trial = 0; trial < 40000; ++trial) {
    sgmv_problem_t p{};
    p.dtype = (int32_t)(rng() % 2);
    p.n_rows = (int32_t)(rng() % 8 == 0 ? rng() % 40 : pick(1, 1 << 20));
    p.h_in = (int32_t)pick(1, 1 << 17) * 8;
    p.h_out = (int32_t)pick(1, 1 << 17) * 8;
    if (rng() % 4) p.h_in = std::min(p.h_in, 16384), p.h_out = std::min(p.h_out, 16384);
    p.rank = ranks[rng() % 4];
    p.num_loras = (int32_t)pick(1, 5000);
    p.num_segs = p.n_rows ? (int32_t)pick(1, std::max(1, p.n_rows)) : 0;
    p.max_seg_len = p.num_segs ? (int32_t)std::min<int64_t>(p.n_rows, ceil_div(p.n_rows, p.num_segs) + (int64_t)(rng() % 500)) : 0;
    for (int op = 0; op < 4; ++op) check_problem(p, op);
  }
  for (int i = 0; i < 5; ++i) CHECK(seen_cfg[i] > 100);
  CHECK(seen_split > 100 && seen_one_launch > 100 && seen_in_tile > 100);
  if (failures) return 1;
  std::puts("layer checks ok");
  return 0;
}
