// sgmv_layer_shapes.h - tile shapes of the layer kernels that the host plan
// needs.  Plain C++ (no HIP).
#pragma once

namespace sgmv {

constexpr int kDenseK = 32;  // contraction length of one tile step

// Output tiles of the dense products (rows x columns; a gated tile's columns
// are half gate, half up).
enum DenseTile : int {
  kTile256 = 0,  // 256 x 256, 8 waves
  kTile192 = 1,  // 192 x 256, 8 waves (not for dW)
  kTile128 = 2,  // 128 x 128, 4 waves
  kTile64 = 3,   // 64 x 256, 4 waves
  kTile32 = 4,   // 32 x 256, 4 waves
  kTile128Wide = 5  // 128 x 256, 8 waves (the calls with an activation: outputs, and dX)
};
constexpr int dense_tile_rows(int t) {
  return t == kTile256 ? 256 : t == kTile192 ? 192 : t == kTile128 || t == kTile128Wide ? 128 : t == kTile64 ? 64 : 32;
}
constexpr int dense_tile_cols(int t) { return t == kTile128 ? 128 : 256; }

constexpr int kThinRows = 64;      // rows of one segment per thin-product workgroup
constexpr int kLoraGradCols = 256; // columns of X or dY per LoRA-gradient workgroup

// fp16 dG and dU of a row are kept divided by 2^(8 b), -kMaxRowPower <= b <= kMaxRowPower; b of a row of zeros.
constexpr int kMaxRowPower = 15, kZeroRow = -128;

// fp16 rows up to this wide are one workgroup's in the activation's backward, which finds their powers on its way.
constexpr int kActRowCols = 16384;

}  // namespace sgmv
