// sgmv_tile.h - operand tiles of the layer kernels' matrix products: loads
// straight from memory into LDS, and the reads of matrix operands from there.
//
// An operand whose contraction index is contiguous in memory is kept row by
// row, its 16-byte groups at group ^ swizzle_r(row), and read with 128-bit reads.  An operand
// stored the other way round is kept as it lies and read with the
// transposing 64-bit read; the four rows that one 16-lane group reads fall
// into different banks, because group g of row k is stored at g ^ f(k).
#pragma once

#include "sgmv_layer_ops.h"

namespace sgmv {

template <int N>
__device__ inline void wait_loads_and_lds() {
  // All but the N newest of this wave's loads have landed, and its LDS reads are
  // done (the slot they read is refilled after the barrier that follows).
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// Column swizzle of a tile stored [k][cols] (the f(k) above), in 16-byte groups.  Rows of 16 groups and more are
// read without bank conflicts; the 2 to 8 groups of the thin products' D_k leave fewer places to go: 24 to 33% of
// those kernels' LDS cycles are conflicts.
template <int COLS>
__device__ inline int swizzle_k(int k) {
  return (((k & 3) | ((k >> 1) & 4)) << 1) & (COLS / 8 - 1);
}

// Group swizzle of a tile stored [row][32].  A 128-bit read serves lanes 0-3, 12-15 and 20-27 together (and so on, in
// turns of eight): four rows of one residue mod 4, at groups q and q ^ 1.  (row / 4) % 4 itself leaves two of
// them in the same banks, and half of all LDS cycles were conflicts.
__device__ inline int swizzle_r(int row) { return (-(row >> 2)) & 3; }

// One operand tile of R rows (or columns) x 32 contraction steps.
template <int R, int LOADS, bool T>
struct TileLoader {
  static constexpr int PIECES = R / 16;  // of 1 KiB
  uint32_t voff[LOADS];
  uint32_t lds_off[LOADS];  // uniform
  uint32_t g8;              // first contraction index (of 8) of this lane within the step (row-major operand)
  // Uniform: where the next step starts, and how much there is.
  const uint16_t* base;
  int64_t step;
  uint32_t full, tail;  // bytes of a step's descriptor
  int left;             // contraction indices from the next step on
  __device__ inline void init(int wave, int lane, int ld) {
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int L = (wave * LOADS + j) % PIECES;
      lds_off[j] = (uint32_t)L * 512;
      if constexpr (T) {
        constexpr int G = R / 8;  // 16-byte groups per k row
        const int k = L * (64 / G) + lane / G;
        const int g = (lane % G) ^ swizzle_k<R>(k);
        voff[j] = (uint32_t)(k * ld + g * 8) * 2u;
      } else {
        const int r = L * 16 + (lane >> 2);
        voff[j] = (uint32_t)(r * ld + ((lane & 3) ^ swizzle_r(r)) * 8) * 2u;
      }
    }
    g8 = ((lane & 3) ^ swizzle_r(lane >> 2)) * 8;
  }
  // Points at contraction index k0 of an operand with K of them; r0: first row
  // (column) of the tile, rows: how many the matrix has.
  __device__ inline void start(const uint16_t* operand, int ld, int r0, int rows, int k0, int K) {
    left = K - k0;
    if constexpr (T) {
      base = operand + (int64_t)k0 * ld + r0;
      step = (int64_t)kDenseK * ld;
      full = (uint32_t)((kDenseK - 1) * ld + (rows - r0)) * 2u;
      tail = (uint32_t)((((K - 1) & (kDenseK - 1))) * ld + (rows - r0)) * 2u;  // of the last step
    } else {
      base = operand + (int64_t)r0 * ld + k0;
      full = (uint32_t)((rows - r0 < R ? rows - r0 : R) * ld - k0) * 2u;
    }
  }
  // One step of an operand stored with the contraction index as row: `n` rows (0: none, the slot is
  // filled with zeros) from row `row` on, from column r0 of `cols`.
  __device__ inline void issue_rows(const uint16_t* operand, int ld, int r0, int cols, int row, int n,
                                    uint16_t* lds) const {
    static_assert(T, "row-wise steps");
    const uint32_t bytes = n > 0 ? (uint32_t)((n - 1) * ld + (cols - r0)) * 2u : 0u;
    const auto rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(operand + (int64_t)row * ld + r0), 0,
                                                      (int)bytes, kRawBuffer);
#pragma unroll
    for (int j = 0; j < LOADS; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(lds + lds_off[j]), 16, (int)voff[j], 0, 0, 0);
  }
  // Loads the next step into an LDS slot.  Past the last contraction index every
  // lane is out of range: nothing is fetched and the slot is filled with
  // zeros, so that each step counts the same loads.
  __device__ inline void issue(uint16_t* lds) {
    const uint32_t some = left > 0 ? full : 0u;
    if constexpr (T) {
      const uint32_t bytes = left >= kDenseK || left <= 0 ? some : tail;
      const auto rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base), 0, (int)bytes, kRawBuffer);
#pragma unroll
      for (int j = 0; j < LOADS; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(lds + lds_off[j]), 16, (int)voff[j], 0, 0, 0);
      base += step;
    } else {
      const auto rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base), 0, (int)some, kRawBuffer);
      const uint32_t past = (int)g8 < left ? 0u : kOutOfRange;
#pragma unroll
      for (int j = 0; j < LOADS; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(lds + lds_off[j]), 16, (int)(voff[j] | past), 0, 0, 0);
      base += kDenseK;
      full -= 2 * kDenseK;  // the descriptor's end stays where it is
    }
    left -= kDenseK;
  }
};

// Operand of 16 rows (columns) x 32 contraction steps of an LDS tile; tile: its
// first row / column inside the tile (a multiple of 16).
template <int R, bool T>
__device__ inline u32x4 read_operand(const uint16_t* lds, int tile, int lane) {
  const int q = lane >> 4, i = lane & 15;
  if constexpr (T) {
    const int k = q * 8 + (i >> 2);
    const int g = (tile / 8 + ((i & 3) >> 1)) ^ swizzle_k<R>(k);
    const uint16_t* a = lds + k * R + g * 8 + (i & 1) * 4;
    const u32x2 l = read_transposed(a), h = read_transposed(a + 4 * R);  // k + 4 has the same swizzle
    return u32x4{l[0], l[1], h[0], h[1]};
  } else {
    return load_vec(lds + (tile + i) * kDenseK + ((q ^ swizzle_r(i)) << 3));
  }
}

}  // namespace sgmv
