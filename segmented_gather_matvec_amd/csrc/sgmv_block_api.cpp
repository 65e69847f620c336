// sgmv_block_api.cpp - the entry points around a layer (rows sorted by LoRA and back, layer norm): argument checks and
// launches.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/sgmv.h"
#include "sgmv_block.h"
#include "sgmv_block_host.h"

namespace {

using namespace sgmv_host;

bool misaligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }
const uint16_t* half(const void* p) { return static_cast<const uint16_t*>(p); }
uint16_t* half(void* p) { return static_cast<uint16_t*>(p); }
sgmv_status_t status(hipError_t e) { return e == hipSuccess ? SGMV_OK : SGMV_ERR_HIP; }

sgmv_status_t check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (need > 0 && (!ws || ws_bytes < need)) return SGMV_ERR_WORKSPACE;
  return misaligned(ws, 16) ? SGMV_ERR_UNSUPPORTED : SGMV_OK;
}

}  // namespace

extern "C" {

sgmv_status_t sgmv_route_rows(int32_t n_rows, int32_t top_k, int32_t num_loras, const int32_t* ids, int32_t* perm,
                              int32_t* slots, int32_t* seg_indptr, int32_t* lora_idx, void* ws, size_t ws_bytes,
                              void* stream) {
  sgmv_status_t st = check_route(n_rows, top_k, num_loras);
  if (st != SGMV_OK) return st;
  if (n_rows > 0 && !ids) return SGMV_ERR_INVALID_ARG;
  if (misaligned(ids, 4) || misaligned(perm, 4) || misaligned(slots, 4) || misaligned(seg_indptr, 4) || misaligned(lora_idx, 4))
    return SGMV_ERR_UNSUPPORTED;
  const RoutePlan plan = plan_route(n_rows, top_k, num_loras);
  st = check_ws(ws, ws_bytes, plan.total);
  if (st != SGMV_OK) return st;
  sgmv::RouteParams p{};
  p.ids = ids;
  p.perm = perm;
  p.slots = slots;
  p.seg_indptr = seg_indptr;
  p.lora_idx = lora_idx;
  p.counts = static_cast<int32_t*>(ws);
  p.m = n_rows * top_k;
  p.num_loras = num_loras;
  p.blocks = plan.blocks;
  p.tile = plan.tile;
  p.waves = plan.waves;
  return status(sgmv::launch_route(p, static_cast<hipStream_t>(stream)));
}

sgmv_status_t sgmv_dispatch_rows(int32_t dtype, int32_t n_rows, int32_t top_k, int32_t width, const void* X,
                                 const int32_t* slots, void* Xs, void* stream) {
  const sgmv_status_t st = check_rows(dtype, n_rows, top_k, width);
  if (st != SGMV_OK) return st;
  if (n_rows == 0) return SGMV_OK;
  if (!X || !slots || !Xs) return SGMV_ERR_INVALID_ARG;
  if (misaligned(X, 16) || misaligned(slots, 4) || misaligned(Xs, 16)) return SGMV_ERR_UNSUPPORTED;
  sgmv::RowsParams p{};
  p.X = half(X);
  p.slots = slots;
  p.out = half(Xs);
  p.n = n_rows;
  p.top_k = top_k;
  p.w8 = width / 8;
  return status(sgmv::launch_dispatch(p, static_cast<hipStream_t>(stream)));
}

sgmv_status_t sgmv_combine_rows(int32_t dtype, int32_t n_rows, int32_t top_k, int32_t width, const void* Ys,
                                const int32_t* slots, const float* weights, const void* residual, void* Y, void* stream) {
  const sgmv_status_t st = check_rows(dtype, n_rows, top_k, width);
  if (st != SGMV_OK) return st;
  if (n_rows == 0) return SGMV_OK;
  if (!Ys || !slots || !Y) return SGMV_ERR_INVALID_ARG;
  if (misaligned(Ys, 16) || misaligned(slots, 4) || misaligned(weights, 4) || misaligned(residual, 16) || misaligned(Y, 16))
    return SGMV_ERR_UNSUPPORTED;
  sgmv::RowsParams p{};
  p.X = half(Ys);
  p.R = half(residual);
  p.slots = slots;
  p.weights = weights;
  p.out = half(Y);
  p.n = n_rows;
  p.top_k = top_k;
  p.w8 = width / 8;
  return status(sgmv::launch_combine(dtype, p, static_cast<hipStream_t>(stream)));
}

sgmv_status_t sgmv_combine_rows_backward(int32_t dtype, int32_t n_rows, int32_t top_k, int32_t width, const void* dY,
                                         const void* Ys, const int32_t* slots, const float* weights, void* dYs,
                                         float* dweights, void* stream) {
  const sgmv_status_t st = check_rows(dtype, n_rows, top_k, width);
  if (st != SGMV_OK) return st;
  if (n_rows == 0) return SGMV_OK;
  if (!dY || !slots || (dweights && !Ys)) return SGMV_ERR_INVALID_ARG;
  if (misaligned(dY, 16) || misaligned(Ys, 16) || misaligned(slots, 4) || misaligned(weights, 4) || misaligned(dYs, 16) ||
      misaligned(dweights, 4))
    return SGMV_ERR_UNSUPPORTED;
  sgmv::RowsParams p{};
  p.X = half(dY);
  p.Ys = half(Ys);
  p.slots = slots;
  p.weights = weights;
  p.out = half(dYs);
  p.dweights = dweights;
  p.n = n_rows;
  p.top_k = top_k;
  p.w8 = width / 8;
  return status(sgmv::launch_combine_backward(dtype, p, static_cast<hipStream_t>(stream)));
}

sgmv_status_t sgmv_layer_norm_apply(int32_t dtype, int32_t n_rows, int32_t width, const void* X, const void* gamma,
                                    const void* beta, float eps, void* Y, float* mean, float* rstd, void* stream) {
  const sgmv_status_t st = check_rows(dtype, n_rows, 1, width);
  if (st != SGMV_OK) return st;
  if (!(eps >= 0.f) || std::isinf(eps)) return SGMV_ERR_INVALID_ARG;
  if (n_rows == 0) return SGMV_OK;
  if (!X || !Y) return SGMV_ERR_INVALID_ARG;
  if (misaligned(X, 16) || misaligned(gamma, 16) || misaligned(beta, 16) || misaligned(Y, 16) || misaligned(mean, 4) ||
      misaligned(rstd, 4))
    return SGMV_ERR_UNSUPPORTED;
  const NormPlan plan = plan_norm(n_rows, width, false);
  sgmv::NormParams p{};
  p.X = half(X);
  p.gamma = half(gamma);
  p.beta = half(beta);
  p.Y = half(Y);
  p.mean = mean;
  p.rstd = rstd;
  p.eps = eps;
  p.n = n_rows;
  p.w8 = width / 8;
  p.variant = plan.variant;
  p.grid = plan.grid;
  return status(sgmv::launch_layer_norm(dtype, p, static_cast<hipStream_t>(stream)));
}

sgmv_status_t sgmv_layer_norm_backward(int32_t dtype, int32_t n_rows, int32_t width, const void* X, const void* gamma,
                                       const float* mean, const float* rstd, const void* dY, const void* beyond, void* dX,
                                       void* dgamma, void* dbeta, int32_t accumulate, void* ws, size_t ws_bytes,
                                       void* stream) {
  sgmv_status_t st = check_rows(dtype, n_rows, 1, width);
  if (st != SGMV_OK) return st;
  if (accumulate != 0 && accumulate != 1) return SGMV_ERR_INVALID_ARG;
  if (n_rows > 0 && (!X || !mean || !rstd || !dY)) return SGMV_ERR_INVALID_ARG;
  if (misaligned(X, 16) || misaligned(gamma, 16) || misaligned(mean, 4) || misaligned(rstd, 4) || misaligned(dY, 16) ||
      misaligned(beyond, 16) || misaligned(dX, 16) || misaligned(dgamma, 16) || misaligned(dbeta, 16))
    return SGMV_ERR_UNSUPPORTED;
  const NormPlan plan = plan_norm(n_rows, width, true);
  st = check_ws(ws, ws_bytes, plan.total);
  if (st != SGMV_OK) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const bool sums = dgamma || dbeta;
  sgmv::NormParams p{};
  p.X = half(X);
  p.gamma = half(gamma);
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  p.dY = half(dY);
  p.beyond = half(beyond);
  p.dX = half(dX);
  p.planes = sums ? reinterpret_cast<float*>(static_cast<char*>(ws) + plan.planes_off) : nullptr;
  p.stats = reinterpret_cast<float*>(static_cast<char*>(ws) + plan.stats_off);
  p.n = n_rows;
  p.w8 = width / 8;
  p.variant = plan.variant;
  p.grid = plan.grid;
  p.rows_per_block = plan.rows_per_block;
  if (n_rows > 0 && (sums || dX)) {
    st = status(sgmv::launch_layer_norm_backward(dtype, p, s));
    if (st != SGMV_OK) return st;
  }
  return status(sgmv::launch_plane_sum(dtype, p.planes, n_rows > 0 ? plan.grid : 0, 2, width, half(dgamma), half(dbeta),
                                       accumulate, s));
}

}  // extern "C"
