// sgmv_thin.h - the thin products V = s_k Z @ D_k of the layer kernels (D_k =
// A_k or B_k^T), run by their own kernel or by workgroups of a dense product's launch.
#pragma once

#include "sgmv_tile.h"

namespace sgmv {

// Eight ranks c .. c+7 of row `row` of V, as fp32 and / or as hi + lo halves.
// The rank / 8 lanes of one row are neighbours and all come here.
template <class T>
__device__ inline void store_v(const ThinParams& p, int row, int c, float (&v)[8]) {
  if (p.V != nullptr) {
    float* dst = p.V + (int64_t)row * p.rank + c;
    *reinterpret_cast<f32x4*>(dst) = f32x4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4*>(dst + 4) = f32x4{v[4], v[5], v[6], v[7]};
  }
  if (p.V16 == nullptr) return;
  // fp16 halves hold V well only within some binades (above 65504 they overflow, far below 1 the lo
  // half and then the hi half run out of denormals): the row is kept divided by the power 2^(16 b) that
  // brings its largest value to [2^-4, 2^12) (exact), and the reader puts it back.  Steps of 2^16
  // around 1, so that most rows share one.  A row of zeros has the power 0: it goes with any.
  if constexpr (T::kMaxFinite < 1e6f) {
    float big = 0.f, any = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float a = fabsf(v[e]);
      big = fmaxf(big, a < 3.4e38f ? a : 0.f);  // not of infinities and NaN
      any = a == 0.f ? any : 1.f;
    }
    for (int d = 1; d < p.rank / 8; d <<= 1) {
      big = fmaxf(big, shfl_xor(big, d));
      any = fmaxf(any, shfl_xor(any, d));
    }
    int b = (((int)(__float_as_uint(big) >> 23) & 255) - 127 + 4) >> 4;
    b = b < -7 ? -7 : b > 7 ? 7 : b;
    const float up = __uint_as_float((uint32_t)(127 + 16 * b) << 23);
    const float down = __uint_as_float((uint32_t)(127 - 16 * b) << 23);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= down;
    if (c == 0) {
      float s = any * up;
      if (p.q_power != nullptr) {
        // (Clamped far below and beyond anything an fp16 output can show: 0 stands for a row of zeros.)
        const float w = power_of(p.q_power[row]);
        s = s > 0.f && w > 0.f ? fminf(fmaxf(s * w, 0x1p-126f), 0x1p126f) : 0.f;
      }
      p.row_scale[row] = s;
    }
  }
  u32x4 hi, lo;
  split8<T>(v, hi, lo);
  uint16_t* dst = p.V16 + (int64_t)row * 2 * p.rank + c;
  store_vec(dst, hi);
  store_vec(dst + p.rank, lo);
}

// Workgroup (unit, split): up to 64 rows of one segment (16 per wave) times the
// LoRA's D_k over kc contraction steps; both operands stream through a ring of
// LDS slots (sgmv_tile.h).  Bound by reading Z, 128 bytes of 64 rows a step: X [4096, 4096] and dY of
// the same size 26 us (2.6 TB/s), the four products of gated gradients (4096 x 4096 and 4096 x 11008, r = 64) 71 us
// (3.5 TB/s).  64 rows a workgroup, since each LoRA's D_k is read again by every one of them; K is split
// until about four workgroups a CU are there, and the planes' sum (5 to 7 us) follows.
template <int JT>
struct ThinShape {
  static constexpr int COLS = JT * 16, STAGES = JT == 4 ? 3 : 4;  // three or four workgroups per CU
  // A slot: two steps of 32 (the halves of Z's 128-byte lines are asked for together), each Z then D.
  static constexpr int B0 = kThinRows * kDenseK, HALF = (kThinRows + COLS) * kDenseK, SLOT = 2 * HALF;
  static constexpr int RST = COLS + 4;  // row stride of the result in LDS (floats)
  static constexpr int LDS = STAGES * SLOT;
  static_assert(LDS * 2 >= kThinRows * (RST + 1) * 4, "the result and its rows' powers fit the ring");
};

template <class T, int JT, bool TRANSPOSED>
__device__ inline void thin_body(const ThinParams& p, int block, uint16_t* lds) {
  using S = ThinShape<JT>;
  constexpr int COLS = S::COLS, STAGES = S::STAGES, B0 = S::B0, HALF = S::HALF, SLOT = S::SLOT, RST = S::RST;
  constexpr int kPerStep = 4;
  const int t = threadIdx.x;
  const int lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int q = lane >> 4, ml = lane & 15;
  const int u = block / p.ksplit;
  const int g = block - u * p.ksplit;
  const Unit un = resolve_unit<kThinRows>(p.meta.seg_indptr, p.meta.lora_idx, p.meta.num_segs, p.meta.num_loras,
                                          p.meta.n_rows, p.direct, u);
  if (un.L <= 0) return;
  const uint16_t* D = reinterpret_cast<const uint16_t*>(p.ptrs[un.k]);
  const int rk = D != nullptr ? rank_of(p.ranks, p.rank, un.k) : 0;
  const float scale = p.scales != nullptr ? p.scales[un.k] : 1.f;
  const int k0 = g * p.kc;
  const int k1 = p.K < k0 + p.kc ? p.K : k0 + p.kc;
  const int steps = rk > 0 ? (k1 - k0 + 2 * kDenseK - 1) / (2 * kDenseK) : 0;

  // (The rows' powers, asked for ahead of the contraction.)
  const int z_power = T::kMaxFinite < 1e6f && p.z_power != nullptr && t < un.L ? p.z_power[un.r0 + t] : 0;

  if (p.row_k != nullptr && g == 0 && t < un.L) p.row_k[un.r0 + t] = D != nullptr ? un.k : -1;

  f32x4 acc[JT];
#pragma unroll
  for (int j = 0; j < JT; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (steps > 0) {
    TileLoader<kThinRows, 1, false> la;
    TileLoader<COLS, 1, !TRANSPOSED> lb;  // fewer pieces than waves: some load the same piece twice
    const int ldd = TRANSPOSED ? p.K : rk;
    la.init(wave, lane, p.K);
    lb.init(wave, lane, ldd);
    la.start(p.Z + (int64_t)un.r0 * p.K, p.K, 0, un.L, k0, k1);
    lb.start(D, ldd, 0, rk, k0, k1);
    auto issue = [&](uint16_t* slot) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        la.issue(slot + h * HALF);
        lb.issue(slot + h * HALF + B0);
      }
    };
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) issue(lds + s * SLOT);
    int slot = 0;
    for (int s = 0; s < steps; ++s) {
      wait_loads_and_lds<kPerStep*(STAGES - 2)>();
      __builtin_amdgcn_s_barrier();
      issue(lds + (slot == 0 ? STAGES - 1 : slot - 1) * SLOT);  // read in the step before this one
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint16_t* now = lds + slot * SLOT + h * HALF;
        const u32x4 z = read_operand<kThinRows, false>(now, wave * 16, lane);
#pragma unroll
        for (int j = 0; j < JT; ++j)
          acc[j] = mfma<T>(read_operand<COLS, !TRANSPOSED>(now + B0, j * 16, lane), z, acc[j]);
      }
      slot = slot + 1 == STAGES ? 0 : slot + 1;
    }
    wait_loads_and_lds<0>();
  }
  __syncthreads();
  // acc[j][e]: row 16 wave + ml, rank 16 j + 4 q + e.
  float* res = reinterpret_cast<float*>(lds);
  float* row_w = res + kThinRows * RST;
  if (T::kMaxFinite < 1e6f && t < kThinRows) row_w[t] = power_of(z_power);
#pragma unroll
  for (int j = 0; j < JT; ++j) *reinterpret_cast<f32x4*>(&res[(wave * 16 + ml) * RST + j * 16 + q * 4]) = acc[j];
  __syncthreads();
  const int per_row = p.rank / 8;
  for (int x = t; x < un.L * per_row; x += kThreads) {
    const int r = x / per_row, c = (x - r * per_row) * 8;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c < rk ? res[r * RST + c + e] * scale : 0.f;
    if constexpr (T::kMaxFinite < 1e6f) {
      const float w = row_w[r];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= w;
    }
    if (p.to_planes) {
      float* dst = p.planes + ((int64_t)g * p.meta.n_rows + un.r0 + r) * p.rank + c;
      *reinterpret_cast<f32x4*>(dst) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(dst + 4) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
      store_v<T>(p, un.r0 + r, c, v);
    }
  }
}

}  // namespace sgmv
