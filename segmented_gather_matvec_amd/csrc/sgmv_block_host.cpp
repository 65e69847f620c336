// sgmv_block_host.cpp - plans, workspace sizes and checks of the entry points around a layer.  No HIP calls.
#include "sgmv_block_host.h"

#include <algorithm>

namespace sgmv_host {

namespace {

constexpr int64_t kCus = 256;                 // compute units of an MI355X
constexpr int kRouteWaves = 16;
constexpr int64_t kRouteTile = 2048;          // entries of a workgroup, at least
constexpr int64_t kRouteCounts = 1 << 16;     // counts that every workgroup reads, at most

}  // namespace

sgmv_status_t check_route(int32_t n_rows, int32_t top_k, int32_t num_loras) {
  if (n_rows < 0 || top_k < 1 || num_loras < 1) return SGMV_ERR_INVALID_ARG;
  if (top_k > SGMV_MAX_TOP_K || num_loras > SGMV_MAX_ROUTE_LORAS) return SGMV_ERR_UNSUPPORTED;
  return (int64_t)n_rows * top_k > SGMV_MAX_LAYER_ROWS ? SGMV_ERR_UNSUPPORTED : SGMV_OK;
}

RoutePlan plan_route(int32_t n_rows, int32_t top_k, int32_t num_loras) {
  RoutePlan r;
  const int64_t m = (int64_t)n_rows * top_k, keys = (int64_t)num_loras + 1;
  r.waves = (int32_t)std::max<int64_t>(1, std::min<int64_t>(kRouteWaves, sgmv::kRouteLds / keys - 2));
  const int64_t most = std::max<int64_t>(1, kRouteCounts / keys);
  const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>(most, ceil_div(m, kRouteTile)));
  r.tile = (int32_t)round_up(std::max<int64_t>(1, ceil_div(m, blocks)), 64 * r.waves);
  r.blocks = (int32_t)std::max<int64_t>(1, ceil_div(m, r.tile));
  r.total = r.blocks > 1 ? (size_t)round_up(r.blocks * keys * 4, 256) : 0;
  return r;
}

sgmv_status_t check_rows(int32_t dtype, int32_t n_rows, int32_t top_k, int32_t width) {
  if (n_rows < 0 || top_k < 1 || width < 1) return SGMV_ERR_INVALID_ARG;
  if (dtype != SGMV_F16 && dtype != SGMV_BF16) return SGMV_ERR_UNSUPPORTED;
  if (width % 8 != 0 || width > SGMV_MAX_HIDDEN || top_k > SGMV_MAX_TOP_K) return SGMV_ERR_UNSUPPORTED;
  return (int64_t)n_rows * top_k > SGMV_MAX_LAYER_ROWS ? SGMV_ERR_UNSUPPORTED : SGMV_OK;
}

NormPlan plan_norm(int32_t n_rows, int32_t width, bool back) {
  NormPlan p;
  const int w8 = width / 8;
  const sgmv::NormVariant* v = back ? sgmv::kNormBackward : sgmv::kNormForward;
  const int last = (back ? sgmv::kNormBackwardVariants : sgmv::kNormForwardVariants) - 1;
  while (p.variant < last && w8 > v[p.variant].eights()) ++p.variant;
  const sgmv::NormVariant& s = v[p.variant];
  const int64_t groups = std::max<int64_t>(1, ceil_div(n_rows, s.rows));
  if (!back) {
    p.grid = (int32_t)std::min<int64_t>(groups, kCus * s.per_cu);
    return p;
  }
  if (s.keep > 0) {
    p.grid = (int32_t)std::min<int64_t>(groups, kCus * s.per_cu);
  } else {
    // Wide rows: (column chunks) x (row blocks).
    const int64_t chunks = ceil_div(width, sgmv::kNormWideCols);
    const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>(ceil_div(1024, chunks), ceil_div(n_rows, 4)));
    p.rows_per_block = (int32_t)std::max<int64_t>(1, ceil_div(n_rows, blocks));
    p.grid = (int32_t)std::max<int64_t>(1, ceil_div(n_rows, p.rows_per_block));
    p.stats_off = 0;
    p.planes_off = (size_t)round_up((int64_t)n_rows * 8, 256);
  }
  p.total = p.planes_off + (size_t)round_up((int64_t)p.grid * 2 * width * 4, 256);
  if (n_rows == 0) p.total = 0;
  return p;
}

}  // namespace sgmv_host

using namespace sgmv_host;

extern "C" {

sgmv_status_t sgmv_route_workspace_bytes(int32_t n_rows, int32_t top_k, int32_t num_loras, size_t* bytes) {
  const sgmv_status_t st = check_route(n_rows, top_k, num_loras);
  if (st != SGMV_OK) return st;
  if (!bytes) return SGMV_ERR_INVALID_ARG;
  *bytes = plan_route(n_rows, top_k, num_loras).total;
  return SGMV_OK;
}

sgmv_status_t sgmv_layer_norm_workspace_bytes(int32_t n_rows, int32_t width, size_t* bytes) {
  const sgmv_status_t st = check_rows(SGMV_F16, n_rows, 1, width);
  if (st != SGMV_OK) return st;
  if (!bytes) return SGMV_ERR_INVALID_ARG;
  *bytes = plan_norm(n_rows, width, true).total;
  return SGMV_OK;
}

}  // extern "C"
