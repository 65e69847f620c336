// sgmv_act.hip - the elementwise backward of a dense layer's activation (gfx950): dZ = dY * act'(Z), and the bias's
// gradient, the column sums of dZ.
//
// Bound by memory: Z and dY are read once, dZ is written once, and the column sums ride along in registers.  A thread has eight
// columns of a block of rows, four rows of both operands in flight; the blocks' sums are written as planes and
// added up by a launch of their own (no atomics: one order).
// fp16 rows carry a power of two each (as in the gated block's backward): dZ is an operand of the matrix cores,
// and a row whose values are small must not lose them to fp16's denormals.  The power comes from the row's largest |dY|
// (no activation here has a slope beyond 1.13), so a
// workgroup that has whole rows (up to 16384 columns) finds it on its way (4096 rows of 4096, 8192 and
// 11008: 33, 51 and 110 us with the bias's sums; with a launch ahead that looks at dY, as wider rows have it, 43, 70 and 122).
#include <algorithm>

#include "sgmv_layer_ops.h"

namespace sgmv {
namespace {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
// Two running maxima, of the even and the odd columns, of fp16 magnitudes as integers; what is neither finite nor 0 counts as
// the smallest denormal.
__device__ inline uint32_t largest(const u32x4& v, uint32_t big) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t m = v[w] & 0x7fff7fffu;
    const uint32_t odd = ((m + 0x04000400u) >> 15) & 0x00010001u;  // infinities and NaN (no carry between the halves)
    const uint32_t x = (m & ~(odd * 0xffffu)) | odd;
    big = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, big), __builtin_bit_cast(u16x2, x)));
  }
  return big;
}
// fp32 bits of 1.13 times the larger of the two.
__device__ inline uint32_t largest_bits(uint32_t big) {
  const uint32_t a = big & 0xffffu, b = big >> 16;
  return __float_as_uint(1.13f * F16::one((uint16_t)(a > b ? a : b)));
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
    big = wave_max(largest_bits(big));
    __syncthreads();  // the row before has been read
    if ((t & 63) == 0) most[t >> 6] = big;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) big = big > most[w] ? big : most[w];
    if (t == 0) power[row] = (int8_t)power_for(big);
  }
}

// Workgroup: a block of rows by THREADS x KEEP eights of columns, U rows in flight.  POWER: it has whole rows and finds
// their powers itself.
template <class T, bool HALVES, bool POWER, int THREADS, int KEEP, int U>
__global__ __launch_bounds__(THREADS) void sgmv_act_backward_kernel(ActBackwardParams p) {
  constexpr int WAVES = THREADS / 64;
  __shared__ uint32_t most[POWER ? 2 : 1][WAVES][U];
  const int t = threadIdx.x;
  bool live[KEEP];
  int c[KEEP];
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    const int x = ((int)blockIdx.y * KEEP + k) * THREADS + t;
    live[k] = x * 8 < p.F;
    c[k] = live[k] ? x * 8 : p.F - 8;
  }
  if (!POWER && !live[0]) return;
  const int64_t r0 = (int64_t)blockIdx.x * p.rows_per_block;
  const int64_t r1 = r0 + p.rows_per_block < p.n ? r0 + p.rows_per_block : p.n;
  float sum[KEEP][8];
#pragma unroll
  for (int k = 0; k < KEEP; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[k][e] = 0.f;
  u32x4 nz[U][KEEP], ny[U][KEEP];
  const auto ask = [&](int64_t row) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = row + u < r1 ? row + u : r1 - 1;
#pragma unroll
      for (int k = 0; k < KEEP; ++k) {
        ny[u][k] = load_stream(p.dY + at * p.F + c[k]);
        if (p.dZ != nullptr) nz[u][k] = load_stream(p.Z + at * p.F + c[k]);
      }
    }
  };
  if (POWER) ask(r0);
  int turn = 0;
  for (int64_t row = r0; row < r1; row += U, turn ^= 1) {
    u32x4 z[U][KEEP], y[U][KEEP];
    int power[U];
    if (!POWER) ask(row);
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int k = 0; k < KEEP; ++k) {
        y[u][k] = ny[u][k];
        z[u][k] = nz[u][k];
      }
      const int64_t at = row + u < r1 ? row + u : r1 - 1;
      power[u] = T::kMaxFinite < 1e6f && !POWER && p.dZ != nullptr ? p.row_power[at] : 0;
    }
    if (POWER && row + U < r1) ask(row + U);  // ahead of this rows' barrier
    if constexpr (POWER) {
      uint32_t big[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        big[u] = 0;
#pragma unroll
        for (int k = 0; k < KEEP; ++k) big[u] = largest(y[u][k], big[u]);
        big[u] = wave_max(largest_bits(big[u]));
        if ((t & 63) == 0) most[turn][t >> 6][u] = big[u];
      }
      __syncthreads();  // (the other half's readers are past the barrier before)
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int w = 0; w < WAVES; ++w) big[u] = big[u] > most[turn][w][u] ? big[u] : most[turn][w][u];
        power[u] = power_for(big[u]);
        if (t == 0 && row + u < r1) p.row_power[row + u] = (int8_t)power[u];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (row + u >= r1) continue;
#pragma unroll
      for (int k = 0; k < KEEP; ++k) {
        float d[8];
        unpack8<T>(y[u][k], d);
        if (p.dZ != nullptr) {
          float zv[8];
          unpack8<T>(z[u][k], zv);
          act_slopes<8>(p.act, zv, d);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[k][e] += d[e];
        if (p.dZ == nullptr || !live[k]) continue;
        const int64_t o = (row + u) * p.F + c[k];
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
  }
  if (p.planes == nullptr) return;
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    if (!live[k]) continue;
    float* const dst = p.planes + (int64_t)blockIdx.x * p.F + c[k];
    *reinterpret_cast<f32x4*>(dst) = f32x4{sum[k][0], sum[k][1], sum[k][2], sum[k][3]};
    *reinterpret_cast<f32x4*>(dst + 4) = f32x4{sum[k][4], sum[k][5], sum[k][6], sum[k][7]};
  }
}

template <class T, bool POWER, int THREADS, int KEEP, int U>
hipError_t launch_act_backward_t(const ActBackwardParams& p, hipStream_t s) {
  const int per = THREADS * KEEP * 8;
  const dim3 grid((unsigned)((p.n + p.rows_per_block - 1) / p.rows_per_block), (unsigned)((p.F + per - 1) / per));
  if (POWER && grid.y != 1) return hipErrorInvalidValue;
  if (p.halves)
    hipLaunchKernelGGL((sgmv_act_backward_kernel<T, true, POWER, THREADS, KEEP, U>), grid, dim3(THREADS), 0, s, p);
  else
    hipLaunchKernelGGL((sgmv_act_backward_kernel<T, false, POWER, THREADS, KEEP, U>), grid, dim3(THREADS), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_act_backward(int dtype, const ActBackwardParams& p, hipStream_t stream) {
  if (p.n <= 0 || (p.dZ == nullptr && p.planes == nullptr)) return hipSuccess;
  if (p.rows_per_block < 1) return hipErrorInvalidValue;
  if (dtype == 1) return launch_act_backward_t<BF16, false, kThreads, 1, 4>(p, stream);
  if (p.dZ == nullptr) return launch_act_backward_t<F16, false, kThreads, 1, 4>(p, stream);
  if (p.F <= 2048) return launch_act_backward_t<F16, true, 256, 1, 2>(p, stream);
  if (p.F <= 4096) return launch_act_backward_t<F16, true, 256, 2, 1>(p, stream);
  if (p.F <= 8192) return launch_act_backward_t<F16, true, 512, 2, 1>(p, stream);
  if (p.F <= kActRowCols) return launch_act_backward_t<F16, true, 1024, 2, 1>(p, stream);
  hipLaunchKernelGGL(sgmv_row_power_kernel, dim3((unsigned)std::min(p.n, 8192)), dim3(kThreads), 0, stream, p.dY, p.row_power,
                     p.n, p.F / 8);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_act_backward_t<F16, false, kThreads, 1, 4>(p, stream);
}

}  // namespace sgmv
