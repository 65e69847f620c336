// sgmv_layer_host.cpp - plans, workspace sizes and checks of the layer entry
// points.  No HIP calls.
#include "sgmv_layer_host.h"

#include <algorithm>

namespace sgmv_host {

namespace {

constexpr int64_t kCus = 256;                          // compute units of an MI355X
constexpr int64_t kGradPlaneBytes = (int64_t)256 << 20;  // most the splits of a LoRA gradient may take
// Rows, and values of dG, up to which the gated backward carries dG and dU unrounded (hi + lo halves): a few large
// values' rounding would show in dX and dA, up to 1.7 times the error of an output's own rounding at 5 rows and
// 1.5 times at 77 x 1048, where 1.4 times is what averages out over many.  Few rows are bound by reading W, so
// that twice the rows cost little: 4096 -> 11008, r = 64, 16 rows 68.4 -> 76.5 us; 4096 -> 4096, 64 rows 43 -> 44
// us; but 4096 -> 11008 of 128 rows 82 -> 116.
constexpr int kHalvesRows = 128;
constexpr int64_t kHalvesValues = 1 << 18;

// Whether the tiles' matrix cores add the LoRA term, run by run of rows that share a LoRA (a tile's runs come one
// after another), or the epilogue, row by row from fp32 planes.  Microseconds of either; measured, tiles and
// epilogue: forward, 1024 rows 4096 -> 4096, r = 16: 2 rows a segment 120 and 89 us, 4 rows 84 and 80, 8 rows 65
// and 77; r = 64: 2 rows 200 and 202, 4 rows 131 and 154.  dX, whose epilogue reads A_k row by row: 128 rows,
// r = 64, 4 segments 34 and 84 us, 128 segments 181 and 115; r = 16, 128 segments 128 and 50; 8 rows, r = 16,
// 1 segment 22 and 23, 8 segments 26 and 23; 1024 rows, a LoRA each, r = 16: 210 and 200, r = 64: 338 and 780.
// Decode, forward: the tiles' term costs launches of its own for V, which the epilogue's shares with W's stream:
// 128 gated rows 4096 -> 11008, r = 64, 1 segment 83 and 121 us; 64 rows, 4 segments 82 and 98; 128 rows, r = 16, 81
// and 91; 64 rows, r = 16, 75 and 73; one projection, 128 rows, r = 64, 42 and 47, of 4096 columns 32 and 26.
constexpr int64_t kDecodeRows = 128;
bool tiles_add_term(const sgmv_problem_t& p, bool back, int terms, int64_t N) {
  const double n = p.n_rows;
  const double runs = std::max(1.0, p.num_segs * std::min(1.0, 256.0 / n));  // of one tile
  const double tiles = terms * runs * (p.rank > 32 ? 1.2 : 0.8);
  const double products = terms * n * (double)N * p.rank * 1e-6;
  if (!back && p.n_rows <= kDecodeRows) return tiles + 10.0 < products * (terms > 1 ? 0.3 : 0.2);
  return tiles < 2.0 + products * (back ? 2.0 : 1.0);
}

// Workgroups of a tile shape that run at once on one CU (LDS).
int resident(int cfg) { return cfg <= sgmv::kTile192 || cfg == sgmv::kTile128Wide ? 1 : 2; }

// The model that picks between tile shapes and splits; only ratios matter.
// Large tiles are bound by the matrix cores: microseconds of one contraction
// step of one workgroup on its CU.  Measured, bf16, r = 16: 8192 x 4096 -> 11008 in 6 rounds of 128 steps of
// 256 x 256 tiles 616 us; 2011 x 5120 -> 5120 (r = 64) in one round of 160 steps 142 us of 256 x 256 tiles (160
// workgroups) and 127 us of 192 x 256 (220); 900 rows 4096 -> 4096 in 128 x 128 tiles 50 us (one workgroup a
// CU), 1300 rows 4096 -> 11008 146 us (four), but dX of 5000 rows 11008 -> 4096 590 us (five; 192 rows: 520).
// Without the 192-row tile (it fills rounds that 256 rows leave short) and with it: 1500 rows 4096 -> 11008
// 199 and 166 us; 5000 rows 4096 -> 4096 208 and 174; 2400 gated rows 4096 -> 4096 216 and 179.
// 128 x 256 fills the device where 256 x 256 leave it half empty or split the contraction: without it and with it, forward,
// 2048 rows 4096 -> 4096 81 and 65 us, 1300 rows 5120 -> 5120 81 and 71, 600 rows 4096 -> 11008 68 and 56, 2011 rows
// 11008 -> 4096 172 and 175; dX of 2048 rows 4096 -> 4096 90 and 71, of 1300 rows 5120 -> 5120 90 and 84.
constexpr double kStep256Us = 0.8, kStep192Us = 0.68, kStep128Us = 0.33, kStep128PairUs = 0.3, kStep128WideUs = 0.5;
double step_us(int cfg, int64_t per_cu) {
  if (cfg == sgmv::kTile128Wide) return kStep128WideUs;
  if (cfg == sgmv::kTile256) return kStep256Us;
  if (cfg == sgmv::kTile192) return kStep192Us;
  return per_cu < 2 ? kStep128Us : kStep128PairUs;
}
// The two small ones are bound by streaming B.
constexpr double kStreamBytesPerUs = 5.2e6;  // B of the small tiles, with every slot of the device taken
constexpr double kPlaneBytesPerUs = 4.0e6;   // partial planes, written and read again

DensePlan plan_dense(int64_t M, int64_t N, int64_t steps, int columns_per_n, bool may_split, bool wide128 = false) {
  // columns_per_n: 2 for a gated tile (gate and up columns side by side).  wide128: 128 x 256 tiles may write the outputs.
  DensePlan best;
  double best_cost = -1;
  steps = std::max<int64_t>(steps, 1);
  for (int cfg = sgmv::kTile256; cfg <= (wide128 ? sgmv::kTile128Wide : sgmv::kTile32); ++cfg) {
    const int bm = sgmv::dense_tile_rows(cfg);
    // A tile with more than half of its rows empty only where none is smaller.
    if (cfg <= sgmv::kTile192 && M <= 128) continue;
    if (cfg == sgmv::kTile128Wide && M <= 64) continue;
    if (cfg == sgmv::kTile192 && !may_split) continue;
    if (cfg == sgmv::kTile128 && M <= 64 && may_split) continue;  // dW has no smaller tile
    if (cfg == sgmv::kTile64 && (M <= 32 || M > 64)) continue;
    if (cfg == sgmv::kTile32 && M > 32) continue;
    if (!may_split && cfg > sgmv::kTile128) continue;
    const int64_t tm = ceil_div(M, bm), tn = ceil_div(N, sgmv::dense_tile_cols(cfg) / columns_per_n);
    const int64_t slots = kCus * resident(cfg);
    const int64_t most = may_split && cfg != sgmv::kTile128Wide ? std::max<int64_t>(1, std::min<int64_t>(16, steps / 8)) : 1;
    for (int64_t ks = 1; ks <= most; ++ks) {
      const int64_t per = ceil_div(steps, ks);
      if (ceil_div(steps, per) != ks) continue;
      const int64_t wgs = tm * tn * ks, rounds = ceil_div(wgs, slots);
      double cost;
      if (cfg <= sgmv::kTile128 || cfg == sgmv::kTile128Wide) {
        const int64_t per_cu = ceil_div(wgs, kCus);
        cost = (double)per_cu * (double)per * step_us(cfg, per_cu) + 4.0;
      } else {
        // Gated 4096 -> 11008, one row: 344, 430 and 516 workgroups on 512 slots took 37.8, 34.9 and 39.1 us.
        const double fill = (double)wgs / (double)(rounds * slots);
        cost = (double)steps * sgmv::kDenseK * (double)N * columns_per_n * 2 / kStreamBytesPerUs *
               (fill < 0.5 ? 0.6 / fill : 1.35 - 0.35 * fill);
      }
      if (ks > 1) cost += 3.0 + 2.0 * (double)ks * (double)M * (double)N * columns_per_n * 4 / kPlaneBytesPerUs;
      if (best_cost < 0 || cost < best_cost) {
        best_cost = cost;
        best.cfg = cfg;
        best.tiles_m = (int)tm;
        best.tiles_n = (int)tn;
        best.ksplit = (int)ks;
        best.ktiles_per_split = (int)per;
      }
    }
  }
  return best;
}

// products: that share the launch; summed: whose planes make one V.
ThinPlan plan_thin(const sgmv_problem_t& p, int64_t K, int products, int summed, int64_t workgroups = 1024) {
  ThinPlan t;
  t.units = (int)units_for(p, sgmv::kThinRows, &t.direct);
  // About four workgroups per CU (or as many as said), each of at least 256 contraction steps.
  const int64_t want = ceil_div(workgroups, std::max<int64_t>(1, (int64_t)t.units * products));
  const int64_t ks = std::max<int64_t>(1, std::min<int64_t>(want, ceil_div(K, 256)));
  t.kc = (int)round_up(ceil_div(K, ks), sgmv::kDenseK);
  t.ksplit = (int)ceil_div(K, t.kc);
  t.planes = t.ksplit * summed > 1 ? t.ksplit * summed : 0;
  t.plane_bytes = (size_t)t.planes * p.n_rows * p.rank * sizeof(float);
  return t;
}

// Row splits of one LoRA's gradient over columns C.  All products' tiles share a launch; LoRAs without
// rows leave it at once and have no planes.
int plan_grad_split(const sgmv_problem_t& p, int64_t C, int products) {
  const int64_t used = std::min(p.num_loras, p.num_segs);
  const int64_t wgs = used * products *
                      (ceil_div(p.h_in, sgmv::kLoraGradCols) + ceil_div(p.h_out, sgmv::kLoraGradCols));
  const int64_t fill = ceil_div(768, std::max<int64_t>(1, wgs));
  const int64_t longest = ceil_div(p.max_seg_len, 32 * sgmv::kDenseK);  // one long segment alone
  const int64_t steps = ceil_div(p.n_rows, 4 * sgmv::kDenseK);          // at least four steps each
  // The planes are written and read once each: no more of them than Z has bytes.
  const int64_t cheap = p.n_rows / std::max<int64_t>(1, 4 * used * p.rank);
  const int64_t bytes = (int64_t)p.num_loras * C * p.rank * 4 * products;
  const int64_t n = std::min<int64_t>({std::max(fill, longest), steps, cheap, kGradPlaneBytes / std::max<int64_t>(1, bytes), 64});
  return (int)std::max<int64_t>(1, n);
}

}  // namespace

sgmv_status_t check_layer(const sgmv_problem_t* p) {
  if (!p) return SGMV_ERR_INVALID_ARG;
  const sgmv_status_t st = check_shape(*p);
  if (st != SGMV_OK) return st;
  if (p->n_rows > SGMV_MAX_LAYER_ROWS) return SGMV_ERR_UNSUPPORTED;
  if (nothing_to_do(*p)) return SGMV_OK;
  int direct = 1;
  const int64_t units = units_for(*p, sgmv::kThinRows, &direct);
  return units > SGMV_MAX_LAYER_UNITS || (!direct && p->num_segs > SGMV_MAX_LAYER_LONG_SEGS) ? SGMV_ERR_UNSUPPORTED : SGMV_OK;
}

LayerPlan plan_layer(const sgmv_problem_t& p, int op, bool wide128, bool all_halves) {
  LayerPlan l;
  l.projections = layer_gated(op) ? 2 : 1;
  l.lora = !nothing_to_do(p);
  const int64_t n = p.n_rows;
  l.halves = layer_elementwise(op) && (all_halves || (n <= kHalvesRows && n * p.h_out <= kHalvesValues)) ? 2 : 1;
  const bool back = layer_backward(op);
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (size_t)round_up((int64_t)bytes, 256);
    return here;
  };
  if (l.lora) {
    const size_t v = (size_t)n * p.rank * sizeof(float);
    // The forward call with an activation, beyond decode's rows: half the splits, half the planes to sum.  It rests on two shapes:
    // 2011 rows, K = 11008, r = 64 gain (product and sum 23 + 9 us and 21 + 6), 8192 rows, K = 4096, r = 16 take 30 + 5
    // either way.  (The two products of a backward pass, 4096 rows 4096 -> 11008, r = 16, would lose by it: 35 + 5 and 39 + 5.)
    l.down = plan_thin(p, p.h_in, l.projections, 1, wide128 && !back && n > kDecodeRows ? 512 : 1024);
    if (back) l.up = plan_thin(p, p.h_out, l.projections * l.halves, l.halves);
    for (int i = 0; i < l.projections; ++i) {
      for (int d = 0; d < (back ? 2 : 1); ++d) {
        l.v_off[d][i] = take(v);
        l.half_off[d][i] = take(v);  // two 16-bit halves a value
        l.row_scale_off[d][i] = take((size_t)n * sizeof(float));
        l.thin_off[d][i] = take(d ? l.up.plane_bytes : l.down.plane_bytes);
      }
    }
  }
  if (layer_elementwise(op)) {
    for (int i = 0; i < l.projections; ++i) l.gate_off[i] = take((size_t)n * l.halves * p.h_out * 2);
    l.row_powers = p.dtype == SGMV_F16;
    if (l.row_powers) l.row_power_off = take((size_t)n);
  }
  const int64_t M = n * l.halves, N = back ? p.h_in : p.h_out;
  const bool in_tile = l.lora && tiles_add_term(p, back, l.projections, N);
  const int64_t kt = ceil_div(back ? p.h_out : p.h_in, sgmv::kDenseK);
  const int cols = op == SGMV_GATED_FORWARD ? 2 : 1;
  l.out = plan_dense(M, N, kt * (back ? l.projections : 1), cols, true, wide128 && (!l.lora || in_tile) && l.halves == 1);
  l.out.term_in_tile = in_tile ? 1 : 0;
  // (132 rows 6224 -> 11080, r = 64, 17 segments, in splits: 81 us with all of the term in the first, 55 with its
  // segments shared out.)
  l.out.term_spread = wide128 && in_tile && !back && l.out.ksplit > 1 ? 1 : 0;
  l.out.to_planes = l.out.ksplit > 1 || (l.lora && !in_tile) || l.halves > 1;
  // (The large tiles' workgroups are too big to share a launch with.)
  l.one_launch = l.lora && !back && l.out.to_planes && !in_tile && l.out.cfg > sgmv::kTile192;
  if (l.one_launch) l.row_k_off = take((size_t)n * l.projections * sizeof(int32_t));
  if (l.out.to_planes) l.out.plane_bytes = (size_t)l.out.ksplit * M * N * cols * sizeof(float);
  size_t area = l.out.plane_bytes;
  if (back) {
    l.dw = plan_dense(p.h_in, p.h_out, ceil_div(n, sgmv::kDenseK), 1, false);
    if (l.lora) {
      l.nsplit_a = plan_grad_split(p, p.h_in, l.projections);
      l.nsplit_b = plan_grad_split(p, p.h_out, l.projections);
      const auto bytes = [&](int ns, int64_t C) {
        return ns > 1 ? (size_t)ns * p.num_loras * C * p.rank * sizeof(float) * l.projections : (size_t)0;
      };
      area = std::max(area, bytes(l.nsplit_a, p.h_in) + bytes(l.nsplit_b, p.h_out));
    }
  }
  l.planes_off = take(area);
  l.total = at;
  return l;
}

ActPlan plan_act_backward(const sgmv_problem_t& p, int act, bool all_halves) {
  ActPlan a;
  a.layer = plan_layer(p, act == SGMV_ACT_NONE ? SGMV_DENSE_BACKWARD : SGMV_DENSE_ACT_BACKWARD, true, all_halves);
  // Blocks of rows by 2048 columns: some workgroups a CU, each of four rows and more (their sums are written and read).
  // Whole rows of fp16 have more waves a workgroup: two on a CU.
  const bool whole = p.dtype == SGMV_F16 && act != SGMV_ACT_NONE && p.h_out > 2048 && p.h_out <= sgmv::kActRowCols;
  const int64_t most = whole ? 2 * kCus : ceil_div(6 * kCus, ceil_div(p.h_out, 2048));
  const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>(most, ceil_div(p.n_rows, 4)));
  a.rows_per_block = (int32_t)std::max<int64_t>(1, ceil_div(p.n_rows, blocks));
  a.blocks = (int32_t)ceil_div(p.n_rows, a.rows_per_block);
  a.planes_off = (size_t)round_up((int64_t)a.layer.total, 256);
  a.total = a.planes_off + (size_t)a.blocks * p.h_out * sizeof(float);
  return a;
}

}  // namespace sgmv_host

using namespace sgmv_host;

extern "C" {

sgmv_status_t sgmv_layer_workspace_bytes(const sgmv_problem_t* p, int32_t op, size_t* bytes) {
  const sgmv_status_t st = check_layer(p);
  if (st != SGMV_OK) return st;
  if (!bytes) return SGMV_ERR_INVALID_ARG;
  switch (op) {
    case SGMV_DENSE_FORWARD:
    case SGMV_DENSE_BACKWARD:
    case SGMV_GATED_FORWARD:
    case SGMV_GATED_BACKWARD:
    case SGMV_DENSE_ACT_FORWARD: *bytes = plan_layer(*p, op).total; break;
    case SGMV_DENSE_ACT_BACKWARD:  // of any activation
      *bytes = std::max(plan_act_backward(*p, SGMV_ACT_NONE).total, plan_act_backward(*p, SGMV_ACT_SILU).total);
      break;
    case SGMV_DENSE_ACT_BACKWARD | SGMV_DZ_HALVES:
      if (!halves_fit(*p)) return SGMV_ERR_UNSUPPORTED;
      *bytes = std::max(plan_act_backward(*p, SGMV_ACT_NONE, true).total, plan_act_backward(*p, SGMV_ACT_SILU, true).total);
      break;
    default: return SGMV_ERR_INVALID_ARG;
  }
  return SGMV_OK;
}

}  // extern "C"
