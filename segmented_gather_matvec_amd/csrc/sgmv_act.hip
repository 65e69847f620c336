// sgmv_act.hip - the elementwise backward of a dense layer's activation (gfx950): dZ = dY * act'(Z), and the bias's
// gradient, the column sums of dZ.
//
// Bound by memory: Z and dY are read once, dZ is written once, and the column sums ride along in registers; the blocks' sums
// are written as planes and added up by a launch of their own (no atomics: one order).  bf16, 8192 x 11008 with the bias's
// gradient: 100 us relu, 104 to 109 the others (5.2 TB/s; the sums alone, without an activation, 37).  dZ takes
// ordinary stores, not those past the caches: the products of the same call read it next.
// fp16 rows carry a power of two each (as in the gated block's backward): dZ is an operand of the matrix cores,
// and a row whose values are small must not lose them to fp16's denormals.  The power comes from the row's largest |dY|
// (no activation here has a slope beyond 1.13).  Rows of up to 16384 columns are one workgroup's, which finds it on its way; wider ones
// have a launch ahead that looks at dY (4096 rows of 4096, 8192 and 11008 with the bias's sums: 32, 50 and 96 us, and 43, 70 and
// 122 that way).
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

// Any width: a thread has eight columns of a block of rows, U in flight (fp16: the rows' powers are there already).
template <class T, bool HALVES>
__global__ __launch_bounds__(kThreads) void sgmv_act_backward_kernel(ActBackwardParams p) {
  constexpr int U = 4;  // rows in flight
  const int c = (blockIdx.y * kThreads + threadIdx.x) * 8;
  if (c >= p.F) return;
  const int64_t r0 = (int64_t)blockIdx.x * p.rows_per_block;
  const int64_t r1 = r0 + p.rows_per_block < p.n ? r0 + p.rows_per_block : p.n;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int64_t row = r0; row < r1; row += U) {
    u32x4 z[U], y[U];
    int power[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t o = (row + u < r1 ? row + u : r1 - 1) * p.F + c;
      y[u] = load_stream(p.dY + o);
      if (p.dZ != nullptr) z[u] = load_stream(p.Z + o);
      if (T::kMaxFinite < 1e6f && p.dZ != nullptr) power[u] = p.row_power[row + u < r1 ? row + u : r1 - 1];
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
      if (p.dZ == nullptr) continue;
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
  if (p.planes == nullptr) return;
  float* const dst = p.planes + (int64_t)blockIdx.x * p.F + c;
  *reinterpret_cast<f32x4*>(dst) = f32x4{sum[0], sum[1], sum[2], sum[3]};
  *reinterpret_cast<f32x4*>(dst + 4) = f32x4{sum[4], sum[5], sum[6], sum[7]};
}

// fp16 rows up to THREADS x KEEP eights wide: a workgroup has whole rows of a block, U at a time, and finds their powers
// itself; the next ones are asked for ahead of the barrier that this costs.
template <bool HALVES, int THREADS, int KEEP, int U>
__global__ __launch_bounds__(THREADS) void sgmv_act_backward_rows_kernel(ActBackwardParams p) {
  using T = F16;
  constexpr int WAVES = THREADS / 64;
  __shared__ uint32_t most[2][WAVES][U];
  const int t = threadIdx.x;
  bool live[KEEP];
  int c[KEEP];
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    const int x = k * THREADS + t;
    live[k] = x * 8 < p.F;
    c[k] = live[k] ? x * 8 : p.F - 8;
  }
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
        nz[u][k] = load_stream(p.Z + at * p.F + c[k]);
      }
    }
  };
  ask(r0);
  int turn = 0;
  for (int64_t row = r0; row < r1; row += U, turn ^= 1) {
    u32x4 z[U][KEEP], y[U][KEEP];
    int power[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int k = 0; k < KEEP; ++k) {
        y[u][k] = ny[u][k];
        z[u][k] = nz[u][k];
      }
    }
    if (row + U < r1) ask(row + U);
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
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (row + u >= r1) continue;
#pragma unroll
      for (int k = 0; k < KEEP; ++k) {
        float d[8];
        unpack8<T>(y[u][k], d);
        float zv[8];
        unpack8<T>(z[u][k], zv);
        act_slopes<8>(p.act, zv, d);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[k][e] += d[e];
        if (!live[k]) continue;
        const int64_t o = (row + u) * p.F + c[k];
        const float down = power_of(power[u] == kZeroRow ? 0 : -power[u]);
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] *= down;
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

dim3 act_grid(const ActBackwardParams& p, int columns) {
  return dim3((unsigned)((p.n + p.rows_per_block - 1) / p.rows_per_block), (unsigned)((p.F + columns - 1) / columns));
}

template <class T>
hipError_t launch_act_columns(const ActBackwardParams& p, hipStream_t s) {
  const dim3 grid = act_grid(p, kThreads * 8);
  if (p.halves)
    hipLaunchKernelGGL((sgmv_act_backward_kernel<T, true>), grid, dim3(kThreads), 0, s, p);
  else
    hipLaunchKernelGGL((sgmv_act_backward_kernel<T, false>), grid, dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

template <int THREADS, int KEEP, int U>
hipError_t launch_act_rows(const ActBackwardParams& p, hipStream_t s) {
  const dim3 grid = act_grid(p, THREADS * KEEP * 8);
  if (grid.y != 1) return hipErrorInvalidValue;
  if (p.halves)
    hipLaunchKernelGGL((sgmv_act_backward_rows_kernel<true, THREADS, KEEP, U>), grid, dim3(THREADS), 0, s, p);
  else
    hipLaunchKernelGGL((sgmv_act_backward_rows_kernel<false, THREADS, KEEP, U>), grid, dim3(THREADS), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_act_backward(int dtype, const ActBackwardParams& p, hipStream_t stream) {
  if (p.n <= 0 || (p.dZ == nullptr && p.planes == nullptr)) return hipSuccess;
  if (p.rows_per_block < 1) return hipErrorInvalidValue;
  if (dtype == 1) return launch_act_columns<BF16>(p, stream);
  if (p.dZ == nullptr) return launch_act_columns<F16>(p, stream);
  if (p.F <= 2048) return launch_act_rows<256, 1, 2>(p, stream);
  if (p.F <= 4096) return launch_act_rows<256, 2, 1>(p, stream);
  if (p.F <= 8192) return launch_act_rows<512, 2, 1>(p, stream);
  if (p.F <= kActRowCols) return launch_act_rows<1024, 2, 1>(p, stream);
  hipLaunchKernelGGL(sgmv_row_power_kernel, dim3((unsigned)std::min(p.n, 8192)), dim3(kThreads), 0, stream, p.dY, p.row_power,
                     p.n, p.F / 8);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_act_columns<F16>(p, stream);
}

}  // namespace sgmv
