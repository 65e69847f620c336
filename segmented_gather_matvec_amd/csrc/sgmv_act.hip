// sgmv_act.hip - the elementwise backward of a dense layer's activation (gfx950): dZ = dY * act'(Z), and the bias's
// gradient, the column sums of dZ.
//
// Bound by memory: Z and dY are read once, dZ is written once, and the column sums ride along in registers.  A thread has eight
// columns of a block of rows, four rows of both operands in flight; the blocks' sums are written as planes and
// added up by a launch of their own (no atomics: one order).
// fp16 rows carry a power of two each (as in the gated block's backward): dZ is an operand of the matrix cores,
// and a row whose values are small must not lose them to fp16's denormals.  The power comes from the row's largest |dY|
// (no activation here has a slope beyond 1.13), so where a
// workgroup has whole rows (up to 2048 columns) it finds it on its way; else a launch ahead looks at dY, and the caches keep part of it.
#include <algorithm>

#include "sgmv_layer_ops.h"

namespace sgmv {
namespace {

// Bits of the largest finite magnitude of eight values; 1 (the smallest denormal) for what is neither finite nor 0.
__device__ inline uint32_t largest(const u32x4& v, uint32_t big) {
  float f[8];
  unpack8<F16>(v, f);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t m = __float_as_uint(1.13f * fabsf(f[e]));
    const uint32_t x = m < 0x7f800000u ? m : 1u;
    big = big > x ? big : x;
  }
  return big;
}

// Power of the row whose largest is `big`: 2^(8 b) brings it to [2^7, 2^15).
__device__ inline int power_for(uint32_t big) {
  int e = ((int)(big >> 23) - 127 - 7) >> 3;
  e = e < -kMaxRowPower ? -kMaxRowPower : e > kMaxRowPower ? kMaxRowPower : e;
  return big == 0 ? kZeroRow : e;
}
__device__ inline uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t y = (uint32_t)__shfl_xor((int)v, d, 64);
    v = v > y ? v : y;
  }
  return v;
}

__global__ __launch_bounds__(kThreads) void sgmv_row_power_kernel(const uint16_t* dY, int8_t* power, int n, int f8) {
  __shared__ uint32_t most[kWaves];
  const int t = threadIdx.x;
  for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
    uint32_t big = 0;
#pragma unroll 4
    for (int c = 0; c < f8; c += kThreads)
      big = largest(load_vec(dY + (row * f8 + (c + t < f8 ? c + t : f8 - 1)) * 8), big);
    big = wave_max(big);
    __syncthreads();  // the row before has been read
    if ((t & 63) == 0) most[t >> 6] = big;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) big = big > most[w] ? big : most[w];
    if (t == 0) power[row] = (int8_t)power_for(big);
  }
}

// POWER: the workgroup has whole rows and finds their powers itself.
template <class T, bool HALVES, bool POWER>
__global__ __launch_bounds__(kThreads) void sgmv_act_backward_kernel(ActBackwardParams p) {
  constexpr int U = 4;  // rows in flight
  __shared__ uint32_t most[POWER ? 2 : 1][kWaves][U];
  const bool live = (int)(blockIdx.y * kThreads + threadIdx.x) * 8 < p.F;
  if (!POWER && !live) return;
  const int c = live ? (blockIdx.y * kThreads + threadIdx.x) * 8 : p.F - 8;
  const int64_t r0 = (int64_t)blockIdx.x * p.rows_per_block;
  const int64_t r1 = r0 + p.rows_per_block < p.n ? r0 + p.rows_per_block : p.n;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  int turn = 0;
  for (int64_t row = r0; row < r1; row += U, turn ^= 1) {
    u32x4 z[U], y[U];
    int power[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t o = (row + u < r1 ? row + u : r1 - 1) * p.F + c;
      y[u] = load_stream(p.dY + o);
      if (p.dZ != nullptr) z[u] = load_stream(p.Z + o);
      if (T::kMaxFinite < 1e6f && !POWER && p.dZ != nullptr) power[u] = p.row_power[row + u < r1 ? row + u : r1 - 1];
    }
    if constexpr (POWER) {
      uint32_t big[U];
#pragma unroll
      for (int u = 0; u < U; ++u) big[u] = wave_max(largest(y[u], 0));
      if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int u = 0; u < U; ++u) most[turn][threadIdx.x >> 6][u] = big[u];
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int w = 0; w < kWaves; ++w) big[u] = big[u] > most[turn][w][u] ? big[u] : most[turn][w][u];
        power[u] = power_for(big[u]);
        if (threadIdx.x == 0 && row + u < r1) p.row_power[row + u] = (int8_t)power[u];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (row + u >= r1) continue;
      float d[8];
      unpack8<T>(y[u], d);
      if (p.dZ != nullptr) {
        float zv[8];
        unpack8<T>(z[u], zv);
        act_slopes<8>(p.act, zv, d);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += d[e];
      if (p.dZ == nullptr || (POWER && !live)) continue;
      const int64_t o = (row + u) * p.F + c;
      if constexpr (T::kMaxFinite < 1e6f) {
        const float down = power_of(power[u] == kZeroRow ? 0 : -power[u]);
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] *= down;
      }
      if constexpr (HALVES) {
        u32x4 hi, lo;
        split8<T>(d, hi, lo);
        store_vec(p.dZ + o, hi);
        store_vec(p.dZ + (int64_t)p.n * p.F + o, lo);
      } else {
        store_vec(p.dZ + o, pack8<T>(d));
      }
    }
  }
  if (p.planes == nullptr || (POWER && !live)) return;
  float* const dst = p.planes + (int64_t)blockIdx.x * p.F + c;
  *reinterpret_cast<f32x4*>(dst) = f32x4{sum[0], sum[1], sum[2], sum[3]};
  *reinterpret_cast<f32x4*>(dst + 4) = f32x4{sum[4], sum[5], sum[6], sum[7]};
}

template <class T, bool POWER>
hipError_t launch_act_backward_t(const ActBackwardParams& p, hipStream_t s) {
  const dim3 grid((unsigned)((p.n + p.rows_per_block - 1) / p.rows_per_block),
                  (unsigned)((p.F / 8 + kThreads - 1) / kThreads));
  if (POWER && grid.y != 1) return hipErrorInvalidValue;
  if (p.halves)
    hipLaunchKernelGGL((sgmv_act_backward_kernel<T, true, POWER>), grid, dim3(kThreads), 0, s, p);
  else
    hipLaunchKernelGGL((sgmv_act_backward_kernel<T, false, POWER>), grid, dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_act_backward(int dtype, const ActBackwardParams& p, hipStream_t stream) {
  if (p.n <= 0 || (p.dZ == nullptr && p.planes == nullptr)) return hipSuccess;
  if (p.rows_per_block < 1) return hipErrorInvalidValue;
  if (dtype == 1) return launch_act_backward_t<BF16, false>(p, stream);
  if (p.dZ != nullptr && p.F <= kThreads * 8) return launch_act_backward_t<F16, true>(p, stream);
  if (p.dZ != nullptr) {
    hipLaunchKernelGGL(sgmv_row_power_kernel, dim3((unsigned)std::min(p.n, 8192)), dim3(kThreads), 0, stream, p.dY, p.row_power,
                       p.n, p.F / 8);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return launch_act_backward_t<F16, false>(p, stream);
}

}  // namespace sgmv
