// sgmv_layer.h - host-side interface of the layer kernels (sgmv_dense.hip,
// sgmv_lowrank.hip): a shared projection of any number of rows with the LoRA
// term, the gated feed-forward block made of two of them, and their gradients.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sgmv_layer_shapes.h"

namespace sgmv {

// Segment metadata shared by the layer kernels (device arrays, as elsewhere).
struct SegMeta {
  const int32_t* seg_indptr;
  const int32_t* lora_idx;
  int32_t num_segs;   // 0: no LoRA term
  int32_t num_loras;
  int32_t n_rows;
};

// The LoRA side of one projection as a product's epilogue reads it:
//   out[i, c] += sum_j V[i, j] * E_k[j, c]
// forward: V = s_k X @ A_k, E_k = B_k; dX: V = s_k dY @ B_k^T, E_k = A_k^T.
struct LowRankTerm {
  const float* V;          // [v_planes][n_rows][rank] fp32, read by the epilogue kernel (null: no term)
  const uint16_t* V16;     // [n_rows][2][rank] V's hi, then lo halves, read by the tiles (null: no term)
  const float* row_scale;  // fp16: [n_rows] the power of two that V16's rows are divided by (0: a row of zeros)
  const uint64_t* ptrs;    // [num_loras] -> B_k [r_k, N], or A_k [N, r_k] for dX
  const uint64_t* pair;    // [num_loras] -> A_k, or B_k for dX: where that is null there is no term either
  const int32_t* ranks;    // null, or rank of each LoRA
};

enum DenseMode : int {
  kDenseForward = 0,  // Y = X @ W + term                  A: X, B[0]: W
  kDenseGated = 1,    // G, U two forwards, H = act(G) * U A: X, B[0], B[1]: Wg, Wu
  kDenseDx = 2,       // dX = sum_p dY_p @ W_p^T + terms    A[p]: dY_p, B[p]: W_p
  kDenseDw = 3,       // dW_p = X^T @ dY_p                  A[0]: X, B[p]: dY_p, p = blockIdx.y
  kDenseAct = 4       // Z = X @ W + bias + term, Y = act(Z) + residual   A: X, B[0]: W
};

struct DenseParams {
  int32_t M, N, K;       // output rows and columns, contraction length (of one operand pair)
  int32_t lda, ldb;      // row strides (elements) of the operands as stored
  int32_t pairs;         // operand pairs summed (1 or 2); dW: the second is X with the K rows behind B's first K
  int32_t projections;   // dW: projections (grid y)
  int32_t tiles_m, tiles_n;
  int32_t ksplit;        // workgroups sharing one output tile
  int32_t ktiles_per_split;
  int32_t rank;
  int32_t act;
  int32_t accumulate;    // dW: add to what is there
  int32_t to_planes;     // 1: fp32 partial planes instead of the outputs (ksplit > 1, or the epilogue adds a term)
  int32_t term_in_tile;  // 1: split 0 of every tile adds the LoRA term
  int32_t term_spread;   // 1: forward: the splits of a tile share the term's segments, each adding its own to its plane
  int32_t v_planes;      // partial planes of term[].V that the epilogue sums
  const int32_t* row_k;  // [term][n_rows] LoRA of each covered row (see ThinParams); null: the epilogue searches
  const int8_t* row_power;  // null, or [n_rows] (32-byte aligned, readable to the next 32) the powers that the rows of
                            // dX's A (its n_rows further rows too), or dW's B, are divided by (power_of)
  int64_t plane_stride;  // floats between planes of one projection's output (M * N)
  const uint16_t* A[2];
  const uint16_t* B[2];
  uint16_t* out[3];      // forward: Y; gated: G, U (both may be null), H; dX: dX; dW: dW_0, dW_1; act: Y, Z (may be null)
  const uint16_t* bias;      // act: [N], or null
  const uint16_t* residual;  // act: [M, N] (may be Y itself), or null
  float* planes;         // [projection][ksplit][M][N] (gated: projections g, u)
  SegMeta meta;
  LowRankTerm term[2];
};

// Thin products of the LoRA term: V[i, :] = s_k Z[i, :] @ D_k for every covered
// row, with D_k = A_k ([K, r_k]) or B_k^T (B_k [r_k, K], transposed = 1).
struct ThinParams {
  const uint16_t* Z;      // [n_rows, K]
  const uint64_t* ptrs;
  const int32_t* ranks;
  const float* scales;
  float* V;               // null, or [n_rows][rank] fp32
  uint16_t* V16;          // null, or [n_rows][2][rank] hi and lo halves (see LowRankTerm)
  float* row_scale;       // with V16 in fp16: [n_rows]
  float* planes;          // [ksplit][n_rows][rank], written when to_planes
  int32_t to_planes;      // 1: partial planes (ksplit > 1, or a sum over several products)
  int32_t sum_planes;     // planes from `planes` on that make V (0: another product's sum has them)
  int32_t* row_k;         // null, or [n_rows] the LoRA of each covered row (-1: it lacks this matrix), written
  const int8_t* z_power;  // null, or [n_rows] the powers that Z's rows are divided by (power_of): V gets them back
  const int8_t* q_power;  // null, or [n_rows] powers that row_scale takes on, for a product of V16 with such rows
  int32_t K, rank, transposed;
  int32_t units, direct;  // units of <= kThinRows rows of one segment
  int32_t ksplit, kc;     // K per split, a multiple of 32
  SegMeta meta;
};
// cfg: DenseTile of sgmv_layer_shapes.h.
hipError_t launch_dense(int dtype, int mode, int cfg, const DenseParams& p, hipStream_t stream);
// The forward modes' product of at most 128-row tiles together with `count` thin products (of A_k) in one launch;
// their V stays in partial planes, which the epilogue sums.
hipError_t launch_dense_thin(int dtype, int mode, int cfg, const DenseParams& p, const ThinParams* t, int count,
                             hipStream_t stream);
// Sums the partial planes, adds the LoRA term when term_in_tile is 0, applies
// the activation (gated) and writes the outputs.
hipError_t launch_dense_epilogue(int dtype, int mode, const DenseParams& p, hipStream_t stream);

// count products (at most kMaxThin) in one launch; the plane sums follow.
constexpr int kMaxThin = 6;
hipError_t launch_thin(int dtype, const ThinParams* p, int count, hipStream_t stream);

// Gradients of the LoRA matrices, out[c, j] = sum_{rows i of LoRA k} Z[i, c] * Q[i, j]
// stored [C, r_k] (dA_k: Z = X, Q = s_k dY @ B_k^T) or [r_k, C] (dB_k: Z = dY, Q = s_k X @ A_k).
struct LoraGradParams {
  const uint16_t* Z;      // [n_rows, C], or [2 n_rows, C]: hi halves, then lo (passes = 2)
  int32_t passes;
  const uint16_t* Q;      // [n_rows][2][rank] hi and lo halves (see LowRankTerm)
  const float* row_scale; // fp16: of Q's rows
  const uint64_t* out;    // [num_loras] -> gradient (0: not wanted)
  const uint64_t* A;      // [num_loras] -> A_k, B_k: a LoRA with rows that lacks one has no gradient
  const uint64_t* B;
  const int32_t* ranks;
  float* planes;          // [nsplit][num_loras][C][rank] or [nsplit][num_loras][rank][C] (nsplit > 1)
  int32_t C, rank, rank_major;  // rank_major: stored [r_k, C]
  int32_t nsplit;
  int32_t turns;          // of the sum kernel (set by the launch)
  int32_t first, last;    // segments or LoRAs first .. last - 1 are this launch's (set by the launch)
  int32_t by_segment;     // 1 (fewer segments than LoRAs): a workgroup per segment that is its LoRA's first
  int32_t accumulate;
  SegMeta meta;
};
// count gradients (at most 4) in one launch; the plane sums and the zeros of unused LoRAs follow where there are any.
hipError_t launch_lora_grad(int dtype, const LoraGradParams* p, int count, hipStream_t stream);

// dG = dH * U * act'(G), dU = dH * act(G) ([n, F] each), rounded once to the 16-bit format, or (halves) as hi
// halves followed by lo halves.  fp16: every row divided by its power_of(row_power[i]), written.
hipError_t launch_gate_backward(int dtype, int act, bool halves, const uint16_t* G, const uint16_t* U,
                                const uint16_t* dH, uint16_t* dG, uint16_t* dU, int8_t* row_power, int32_t n, int32_t F,
                                hipStream_t stream);

// dZ = dY * act'(Z) ([n, F]), rounded once to the 16-bit format, or (halves) as hi halves followed by lo halves; fp16:
// every row divided by its power_of(row_power[i]), written.  planes: null, or [blocks][F], the column sums of the
// unrounded dZ over each block of rows.  act none: dY's column sums alone.
struct ActBackwardParams {
  const uint16_t* Z;
  const uint16_t* dY;
  uint16_t* dZ;       // null: act none
  int8_t* row_power;  // fp16
  float* planes;
  int32_t n, F, act;
  int32_t halves;
  int32_t rows_per_block;
};
hipError_t launch_act_backward(int dtype, const ActBackwardParams& p, hipStream_t stream);

}  // namespace sgmv
