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
  int halves = 1;      // 2: the gated backward keeps dG and dU as hi and lo halves, 2 n rows (few rows)
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
inline bool layer_backward(int op) { return op == SGMV_DENSE_BACKWARD || op == SGMV_GATED_BACKWARD; }
// The shape's checks, the rows that the tiles' 32-bit row numbers reach, the units that one launch holds (a
// workgroup each; a launch has fewer than 2^32 threads), and the segments that every unit may walk.
sgmv_status_t check_layer(const sgmv_problem_t* p);
LayerPlan plan_layer(const sgmv_problem_t& p, int op);

}  // namespace sgmv_host
