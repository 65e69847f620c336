// sgmv_layer_host.h - host-only plans and workspace layout of the layer entry
// points (plain C++, no HIP).
#pragma once

#include "sgmv_host.h"
#include "sgmv_layer_shapes.h"

namespace sgmv_host {

// One dense product: output M x N per projection, `steps` contraction steps of kDenseK.
struct DensePlan {
  int cfg = sgmv::kTile256;
  int tiles_m = 0, tiles_n = 0;
  int ksplit = 1;
  int ktiles_per_split = 1;
  int to_planes = 0;     // fp32 planes and an epilogue launch
  int term_in_tile = 0;  // the tiles add the LoRA term
  int term_spread = 0;   // all splits of a tile share it (forward calls with an activation)
  size_t plane_bytes = 0;
};

struct ThinPlan {
  int units = 0, direct = 1, ksplit = 1, kc = 128;
  int planes = 0;          // partial planes of one V (0: written at once)
  size_t plane_bytes = 0;  // of them
};

struct LayerPlan {
  bool lora = false;
  int projections = 1;
  DensePlan out;       // forward, or dX
  int halves = 1;      // 2: dG and dU, or dZ, are kept as hi and lo halves, 2 n rows (few rows, or on request)
  bool one_launch = false;  // the thin products run in the dense product's launch, the epilogue sums their planes
  DensePlan dw;        // dW
  ThinPlan down;       // V = s_k X @ A_k        (K = h_in)
  ThinPlan up;         // dV = s_k dY @ B_k^T    (K = h_out)
  int nsplit_a = 1, nsplit_b = 1;  // row splits of the gradients of A_k and B_k
  // Byte offsets into the workspace.
  // [0][i]: V of projection i, [1][i]: dV; as fp32, as 16-bit halves, the halves' row scales, partial planes.
  size_t v_off[2][2] = {}, half_off[2][2] = {}, row_scale_off[2][2] = {}, thin_off[2][2] = {};
  bool row_powers = false;  // dG and dU are kept divided by a power of two per row (fp16)
  size_t gate_off[2] = {0, 0}, row_power_off = 0, row_k_off = 0;
  size_t planes_off = 0;  // partial planes of the dense product, then of the LoRA gradients (never both live)
  size_t total = 0;
};

inline bool layer_gated(int op) { return op == SGMV_GATED_FORWARD || op == SGMV_GATED_BACKWARD; }
inline bool layer_backward(int op) {
  return op == SGMV_DENSE_BACKWARD || op == SGMV_GATED_BACKWARD || op == SGMV_DENSE_ACT_BACKWARD;
}
// The backward pass starts from elementwise products of its own (dG and dU, dZ).
inline bool layer_elementwise(int op) { return op == SGMV_GATED_BACKWARD || op == SGMV_DENSE_ACT_BACKWARD; }
// The shape's checks, the rows that the tiles' 32-bit row numbers reach, the units that one launch holds (a
// workgroup each; a launch has fewer than 2^32 threads), and the segments that every unit may walk.
sgmv_status_t check_layer(const sgmv_problem_t* p);
// wide128: 128 x 256 tiles too (the calls with an activation).
inline bool layer_act(int op) { return op == SGMV_DENSE_ACT_FORWARD || op == SGMV_DENSE_ACT_BACKWARD; }
// all_halves: the elementwise products are kept as two halves at any size (SGMV_DZ_HALVES).
LayerPlan plan_layer(const sgmv_problem_t& p, int op, bool wide128, bool all_halves = false);
inline LayerPlan plan_layer(const sgmv_problem_t& p, int op) { return plan_layer(p, op, layer_act(op)); }

// The backward call of a dense layer with an activation: the layer's plan (without an activation it is the plain dense
// layer's) and the planes of the bias's gradient behind its workspace.
struct ActPlan {
  LayerPlan layer;
  int32_t rows_per_block = 1, blocks = 1;
  size_t planes_off = 0, total = 0;
};
// all_halves: as of plan_layer; at most half of SGMV_MAX_LAYER_ROWS rows then (dX's product has 2 n).
ActPlan plan_act_backward(const sgmv_problem_t& p, int act, bool all_halves = false);
inline bool halves_fit(const sgmv_problem_t& p) { return p.n_rows <= SGMV_MAX_LAYER_ROWS / 2; }

}  // namespace sgmv_host
