// sgmv_block_shapes.h - shapes of the kernels around a layer that the host plans need.  Plain C++ (no HIP).
#pragma once

namespace sgmv {

constexpr int kRouteThreads = 1024;
constexpr int kRouteLds = 40000;  // 32-bit counters of a workgroup's LDS: one histogram per wave and two more

// A row is held by `waves` waves in registers, `keep` eights a lane; wider rows are read again (keep = 0).
struct NormVariant {
  int waves, keep, rows;  // rows of a workgroup
  constexpr int eights() const { return waves * 64 * keep; }
};
constexpr NormVariant kNormForward[] = {{1, 1, 4}, {1, 2, 4}, {4, 1, 1}, {4, 2, 1}, {4, 3, 1}, {4, 4, 1}, {8, 4, 1}, {16, 3, 1}, {16, 0, 1}};
constexpr NormVariant kNormBackward[] = {{1, 1, 8}, {1, 2, 8}, {4, 1, 2}, {4, 2, 2}, {4, 3, 2}, {8, 2, 1}, {8, 3, 1}, {16, 0, 1}};
constexpr int kNormForwardVariants = 9, kNormBackwardVariants = 8;
constexpr int kNormWideCols = 2048;  // columns of a workgroup of the wide backward

}  // namespace sgmv
