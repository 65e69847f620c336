// sgmv_block.h - host-side interface of the kernels around a layer: rows sorted by LoRA and back (sgmv_route.hip)
// and the layer norm (sgmv_norm.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sgmv {

// ---- rows sorted by LoRA

struct RouteParams {
  const int32_t* ids;   // [m] LoRA of each entry; outside [0, num_loras): none, its key is num_loras
  int32_t* perm;        // [m] entry at each sorted place, or null
  int32_t* slots;       // [m] sorted place of each entry, or null
  int32_t* seg_indptr;  // [num_loras + 1], or null
  int32_t* lora_idx;    // [num_loras], or null
  int32_t* counts;      // [blocks][num_loras + 1], of each block's entries (blocks > 1)
  int32_t m, num_loras;
  int32_t blocks;       // workgroups, `tile` entries each
  int32_t tile;         // a multiple of 64 * waves
  int32_t waves;        // of a workgroup that take entries
};
hipError_t launch_route(const RouteParams& p, hipStream_t stream);

// Rows of X or dY [n, 8 w8] and of Xs, Ys, dYs [n * top_k, 8 w8], 16-bit values.
struct RowsParams {
  const uint16_t* X;       // dispatch: X; combine: Ys; combine backward: dY
  const uint16_t* Ys;      // combine backward
  const uint16_t* R;       // combine: residual, or null
  const int32_t* slots;    // [n * top_k]
  const float* weights;    // [n * top_k], or null (1)
  uint16_t* out;           // dispatch: Xs; combine: Y; combine backward: dYs, or null
  float* dweights;         // combine backward: [n * top_k], or null
  int32_t n, top_k, w8;
};
hipError_t launch_dispatch(const RowsParams& p, hipStream_t stream);
hipError_t launch_combine(int dtype, const RowsParams& p, hipStream_t stream);
hipError_t launch_combine_backward(int dtype, const RowsParams& p, hipStream_t stream);

// ---- layer norm of rows of 8 w8 values

struct NormParams {
  const uint16_t* X;
  const uint16_t* gamma;   // or null (1)
  const uint16_t* beta;    // or null (0)
  uint16_t* Y;
  float* mean;             // [n]; forward: written, or null; backward: read
  float* rstd;
  float eps;
  // backward
  const uint16_t* dY;
  const uint16_t* beyond;  // added to dX, or null
  uint16_t* dX;            // or null
  float* planes;           // [grid][2][8 w8] sums of dY * xh and of dY, or null
  float* stats;            // [n][2] means of q and q * xh (wide rows)
  int32_t n, w8;
  int32_t variant;         // of sgmv_host::NormPlan
  int32_t grid;
  int32_t rows_per_block;  // wide backward: rows of one workgroup
};
hipError_t launch_layer_norm(int dtype, const NormParams& p, hipStream_t stream);
hipError_t launch_layer_norm_backward(int dtype, const NormParams& p, hipStream_t stream);

// out[j][c] (+)= sum over planes g of planes[g][j][c], in a fixed order, rounded once; j < count <= 2, c < width (a
// multiple of 8); an output may be null.  planes == 0 writes zeros.
hipError_t launch_plane_sum(int dtype, const float* planes, int64_t count_planes, int32_t count, int32_t width,
                            uint16_t* out0, uint16_t* out1, int32_t accumulate, hipStream_t stream);

}  // namespace sgmv
