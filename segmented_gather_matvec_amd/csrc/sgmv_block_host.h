// sgmv_block_host.h - host-only plans and checks of the entry points around a layer (plain C++, no HIP).
#pragma once

#include "sgmv_block_shapes.h"
#include "sgmv_host.h"

namespace sgmv_host {

struct RoutePlan {
  int32_t blocks = 1, tile = 0, waves = 1;
  size_t total = 0;  // workspace bytes
};
// n_rows, top_k, num_loras within their limits.
sgmv_status_t check_route(int32_t n_rows, int32_t top_k, int32_t num_loras);
RoutePlan plan_route(int32_t n_rows, int32_t top_k, int32_t num_loras);

// Rows of `width` values in a 16-bit format.
sgmv_status_t check_rows(int32_t dtype, int32_t n_rows, int32_t top_k, int32_t width);

struct NormPlan {
  int32_t variant = 0, grid = 1;
  int32_t rows_per_block = 0;
  size_t planes_off = 0, stats_off = 0, total = 0;
};
NormPlan plan_norm(int32_t n_rows, int32_t width, bool back);

}  // namespace sgmv_host
