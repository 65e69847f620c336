// sgmv_block_shapes.h - shapes of the kernels around a layer that the host plans need.  Plain C++ (no HIP).
#pragma once

namespace sgmv {

constexpr int kRouteThreads = 1024;
constexpr int kRouteLds = 40000;  // 32-bit counters of a workgroup's LDS: one histogram per wave and two more

// A row is held by `waves` waves in registers, `keep` eights a lane; wider rows are read again (keep = 0).  As many workgroups
// of `rows` rows at a time as run at once, `per_cu` on each CU, walk all rows, asking for the next ones ahead: with a workgroup per row
// 2000 x 11008 took 34 us, now 24, and 4096 x 4096 16.4, now 14.  (Backward: each writes a plane of column sums; two on a CU
// instead of one cost 4096 x 4096 33 -> 37 us.)
struct NormVariant {
  int waves, keep, rows, per_cu;
  constexpr int eights() const { return waves * 64 * keep; }
};
constexpr NormVariant kNormForward[] = {{1, 1, 4, 8}, {1, 2, 4, 5}, {4, 1, 1, 6}, {4, 2, 1, 4}, {4, 3, 1, 3},
                                        {8, 2, 1, 2}, {16, 2, 1, 1}, {16, 3, 1, 1}, {16, 0, 1, 2}};
constexpr NormVariant kNormBackward[] = {{1, 1, 8, 2}, {1, 2, 8, 1}, {4, 1, 2, 2}, {4, 2, 2, 1}, {4, 3, 2, 1},
                                         {8, 2, 1, 1}, {8, 3, 1, 1}, {8, 4, 1, 1}, {16, 0, 1, 0}};
constexpr int kNormForwardVariants = 9, kNormBackwardVariants = 9;
constexpr int kNormWideCols = 2048;  // columns of a workgroup of the wide backward

}  // namespace sgmv
