// sgmv_norm.hip - layer norm of 16-bit rows and its gradients (gfx950), and the sums of partial planes.
//
//     y  = (x - mean) r gamma + beta,                     r = (mean((x - mean)^2) + eps)^-1/2
//     dx = r (q - mean(q) - xh mean(q xh)) [+ beyond],    xh = (x - mean) r,  q = dy gamma
//     dgamma = sum_i dy xh,   dbeta = sum_i dy
// Everything between a load and a store is fp32; the variance is the mean of squares about the mean, from values
// that are still in registers (a sum of squares about 0 would lose them to a large mean).
// Bound by memory: x (and dy) are read once, y (dx) is written once.  A row is held in registers by one wave (up to 1024
// values) or by 4 to 16, so that every lane has up to four 16-byte loads in flight and the next row's are asked
// for before this row's sums.  Rows beyond that (24576 values, of the gradients 16384) are read again.
#include <algorithm>

#include "sgmv_block.h"
#include "sgmv_block_shapes.h"
#include "sgmv_layer_ops.h"

namespace sgmv {
namespace {

// Sums of N values over the W waves of a row; red: [2][W][N] of LDS, `turn` says which half.
template <int W, int N>
__device__ inline void row_sums(float (&v)[N], float (*red)[W][N], int turn, int t) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v[n] += shfl_xor(v[n], d);
  }
  if constexpr (W > 1) {
    if ((t & 63) == 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) red[turn][t >> 6][n] = v[n];
    }
    __syncthreads();  // (the other half's readers are past the barrier before)
#pragma unroll
    for (int n = 0; n < N; ++n) {
      v[n] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) v[n] += red[turn][w][n];
    }
  }
}

__device__ inline void fill8(float (&f)[8], float v) {
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = v;
}

template <class T, int W, int KEEP>
__global__ __launch_bounds__(W * 64 > kThreads ? W * 64 : kThreads) void sgmv_layer_norm_kernel(NormParams p) {
  constexpr int TPR = W * 64, ROWS = TPR < kThreads ? kThreads / TPR : 1;
  static_assert(W == 1 || ROWS == 1, "a wave or a workgroup per row");
  __shared__ float red[2][W][1];
  const int t = (int)threadIdx.x % TPR;
  const float count = (float)(p.w8 * 8);
  int c[KEEP];
  bool live[KEEP];
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    live[k] = k * TPR + t < p.w8;
    c[k] = live[k] ? (k * TPR + t) * 8 : (p.w8 - 1) * 8;
  }
  const int64_t step = (int64_t)gridDim.x * ROWS, width = (int64_t)p.w8 * 8;
  int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
  if (row >= p.n) return;  // (ROWS > 1: a wave of its own)
  u32x4 next[KEEP], g[KEEP], b[KEEP];
#pragma unroll
  for (int k = 0; k < KEEP; ++k) next[k] = load_stream(p.X + row * width + c[k]);
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    if (p.gamma != nullptr) g[k] = load_vec(p.gamma + c[k]);
    if (p.beta != nullptr) b[k] = load_vec(p.beta + c[k]);
  }
  for (; row < p.n; row += step) {
    float x[KEEP][8];
#pragma unroll
    for (int k = 0; k < KEEP; ++k) unpack8<T>(next[k], x[k]);
    const int64_t ahead = row + step < p.n ? row + step : row;
#pragma unroll
    for (int k = 0; k < KEEP; ++k) next[k] = load_stream(p.X + ahead * width + c[k]);
    float s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < KEEP; ++k) {
      float a = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) a += x[k][e];
      s[0] += live[k] ? a : 0.f;
    }
    row_sums<W, 1>(s, red, 0, t);
    // (A division: the mean of equal values is that value, since a row that fits here has fewer than 2^12 eights, and their
    // number times the 11 bits of a value is exact.)
    const float mean = s[0] / count;
    s[0] = 0.f;
#pragma unroll
    for (int k = 0; k < KEEP; ++k) {
      float a = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[k][e] -= mean;
        a = __builtin_fmaf(x[k][e], x[k][e], a);
      }
      s[0] += live[k] ? a : 0.f;
    }
    row_sums<W, 1>(s, red, 1, t);
    const float r = 1.f / sqrtf(s[0] / count + p.eps);
    if (t == 0) {
      if (p.mean != nullptr) p.mean[row] = mean;
      if (p.rstd != nullptr) p.rstd[row] = r;
    }
#pragma unroll
    for (int k = 0; k < KEEP; ++k) {
      float f[8];
      fill8(f, 1.f);
      if (p.gamma != nullptr) unpack8<T>(g[k], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[k][e] *= r;
      if (p.beta != nullptr) {
        float h[8];
        unpack8<T>(b[k], h);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[k][e] = __builtin_fmaf(x[k][e], f[e], h[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[k][e] *= f[e];
      }
      if (live[k]) store_stream(p.Y + row * width + c[k], pack8<T>(x[k]));
    }
  }
}

// Rows beyond what 16 waves hold: read three times, the last two from the caches.  Sums of so many values round even where all
// are alike (100008 equal fp16 values: 63 of 200 such rows had a mean beside their value, which made normalised values of up to
// 0.78 where 0 is right), so the second pass also sums what is left about the first mean: that corrects the mean, exactly where
// all values are alike, and the mean of squares about it.
template <class T>
__global__ __launch_bounds__(1024) void sgmv_layer_norm_wide_kernel(NormParams p) {
  constexpr int TPR = 1024, W = TPR / 64;
  __shared__ float red_first[2][W][1], red_rest[2][W][2];  // (two barriers a row: one half of each is enough)
  const int t = threadIdx.x;
  const float count = (float)(p.w8 * 8);
  for (int64_t row = blockIdx.x; row < p.n; row += gridDim.x) {
    const uint16_t* const x = p.X + row * p.w8 * 8;
    float total[1] = {0.f};
#pragma unroll 4
    for (int k = t; k < p.w8; k += TPR) {
      float v[8], a = 0.f;
      unpack8<T>(load_vec(x + (int64_t)k * 8), v);
#pragma unroll
      for (int e = 0; e < 8; ++e) a += v[e];
      total[0] += a;
    }
    row_sums<W, 1>(total, red_first, 0, t);
    const float first = total[0] / count;
    float s[2] = {0.f, 0.f};
#pragma unroll 4
    for (int k = t; k < p.w8; k += TPR) {
      float v[8], a = 0.f, b = 0.f;
      unpack8<T>(load_vec(x + (int64_t)k * 8), v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = v[e] - first;
        a = __builtin_fmaf(d, d, a);
        b += d;
      }
      s[0] += a;
      s[1] += b;
    }
    row_sums<W, 2>(s, red_rest, 0, t);
    float rest = s[1] / count, var = s[0] / count;
    rest = rest - rest == 0.f ? rest : 0.f;  // (infinities, or a sum beyond fp32: the mean stays infinite)
    const float mean = first + rest;
    var = __builtin_fmaf(-rest, rest, var);
    const float r = 1.f / sqrtf((var < 0.f ? 0.f : var) + p.eps);  // (NaN stays)
    if (t == 0) {
      if (p.mean != nullptr) p.mean[row] = mean;
      if (p.rstd != nullptr) p.rstd[row] = r;
    }
#pragma unroll 2
    for (int k = t; k < p.w8; k += TPR) {
      float v[8], g[8], b[8];
      unpack8<T>(load_vec(x + (int64_t)k * 8), v);
      fill8(g, 1.f);
      fill8(b, 0.f);
      if (p.gamma != nullptr) unpack8<T>(load_vec(p.gamma + k * 8), g);
      if (p.beta != nullptr) unpack8<T>(load_vec(p.beta + k * 8), b);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf((v[e] - mean) * r, g[e], b[e]);
      store_vec(p.Y + (row * p.w8 + k) * 8, pack8<T>(v));
    }
  }
}

// ---------------------------------------------------------------- gradients
// Workgroup: ROWS rows at a time, W waves each, every grid-th group of rows; the columns' sums stay in registers
// over all of them, are joined through LDS at the end and written as one plane per workgroup (no atomics: one order).
template <class T, int W, int KEEP, int ROWS>
__global__ __launch_bounds__(W * 64 * ROWS) void sgmv_layer_norm_backward_kernel(NormParams p) {
  constexpr int TPR = W * 64;
  // The next row is asked for before this one's sums, and gamma stays in registers.  Four eights a lane leave none for that: no row
  // ahead, and each thread keeps its gamma in LDS (read again from memory 1500 x 16384 took 60 us instead of 55).
  constexpr bool AHEAD = KEEP < 4;
  __shared__ u32x4 own[AHEAD ? 1 : KEEP][AHEAD ? 1 : TPR];
  __shared__ float red[ROWS][2][W][2];
  __shared__ float joined[ROWS > 1 ? ROWS / 2 : 1][2][ROWS > 1 ? TPR * KEEP * 8 : 1];
  const int t = (int)threadIdx.x % TPR;
  const int sub = __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
  const float count = (float)(p.w8 * 8);
  const int64_t width = (int64_t)p.w8 * 8, step = (int64_t)gridDim.x * ROWS;
  int c[KEEP];
  bool live[KEEP];
  u32x4 g[KEEP];
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    live[k] = k * TPR + t < p.w8;
    c[k] = live[k] ? (k * TPR + t) * 8 : (p.w8 - 1) * 8;
    if (p.gamma != nullptr) (AHEAD ? g[k] : own[k][t]) = load_vec(p.gamma + c[k]);
  }
  float sg[KEEP][8], sb[KEEP][8];
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    fill8(sg[k], 0.f);
    fill8(sb[k], 0.f);
  }
  u32x4 nx[KEEP], ny[KEEP];
  float nmean, nr;
  const auto ask = [&](int64_t row) {
    const int64_t at = row < p.n ? row : p.n - 1;
    nmean = p.mean[at];
    nr = p.rstd[at];
#pragma unroll
    for (int k = 0; k < KEEP; ++k) {
      nx[k] = load_stream(p.X + at * width + c[k]);
      ny[k] = load_stream(p.dY + at * width + c[k]);
    }
  };
  int64_t row = (int64_t)blockIdx.x * ROWS + sub;
  if (AHEAD) ask(row);
  int turn = 0;
  for (int64_t group = (int64_t)blockIdx.x * ROWS; group < p.n; group += step, row += step, turn ^= 1) {
    const bool on = ROWS == 1 || row < p.n;
    if (!AHEAD) ask(row);
    u32x4 x[KEEP], y[KEEP], past[KEEP];
    const float mean = nmean, r = nr;
#pragma unroll
    for (int k = 0; k < KEEP; ++k) {
      x[k] = nx[k];
      // (Zeros past the row's end and for rows past the last: they add nothing.  x is then the last eight, or the
      // last row, again: what is not finite there is in the same sums already.)
#pragma unroll
      for (int w = 0; w < 4; ++w) y[k][w] = on && live[k] ? ny[k][w] : 0u;
      if (p.beyond != nullptr) past[k] = load_stream(p.beyond + (on ? row : p.n - 1) * width + c[k]);
    }
    if (AHEAD && group + step < p.n) ask(row + step);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < KEEP; ++k) {
      float xv[8], yv[8], gv[8];
      unpack8<T>(x[k], xv);
      unpack8<T>(y[k], yv);
      fill8(gv, 1.f);
      if (p.gamma != nullptr) unpack8<T>(AHEAD ? g[k] : own[k][t], gv);
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xh = (xv[e] - mean) * r, q = yv[e] * gv[e];
        a += q;
        b = __builtin_fmaf(q, xh, b);
        sg[k][e] = __builtin_fmaf(yv[e], xh, sg[k][e]);
        sb[k][e] += yv[e];
      }
      s[0] += a;
      s[1] += b;
    }
    if (p.dX == nullptr) continue;  // (uniform)
    row_sums<W, 2>(s, red[sub], turn, t);
    const float m0 = s[0] / count, m1 = s[1] / count;
#pragma unroll
    for (int k = 0; k < KEEP; ++k) {
      float xv[8], yv[8], gv[8], d[8];
      unpack8<T>(x[k], xv);
      unpack8<T>(y[k], yv);
      fill8(gv, 1.f);
      if (p.gamma != nullptr) unpack8<T>(AHEAD ? g[k] : own[k][t], gv);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xh = (xv[e] - mean) * r, q = yv[e] * gv[e];
        d[e] = r * (q - m0 - xh * m1);
      }
      if (p.beyond != nullptr) {
        float o[8];
        unpack8<T>(past[k], o);
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] += o[e];
      }
      if (on && live[k]) store_stream(p.dX + row * width + c[k], pack8<T>(d));
    }
  }
  if (p.planes == nullptr) return;
  // The rows' sums of the workgroup, halves onto halves.
  if constexpr (ROWS > 1) {
#pragma unroll
    for (int s = ROWS / 2; s > 0; s /= 2) {
      __syncthreads();
      if (sub >= s && sub < 2 * s) {
#pragma unroll
        for (int k = 0; k < KEEP; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            joined[sub - s][0][(k * 8 + e) * TPR + t] = sg[k][e];
            joined[sub - s][1][(k * 8 + e) * TPR + t] = sb[k][e];
          }
      }
      __syncthreads();
      if (sub < s) {
#pragma unroll
        for (int k = 0; k < KEEP; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            sg[k][e] += joined[sub][0][(k * 8 + e) * TPR + t];
            sb[k][e] += joined[sub][1][(k * 8 + e) * TPR + t];
          }
      }
    }
  }
  if (sub > 0) return;
  float* const plane = p.planes + (int64_t)blockIdx.x * 2 * width;
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    if (!live[k]) continue;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float* dst = plane + half * width + c[k];
      const float(&v)[8] = half ? sb[k] : sg[k];
      *reinterpret_cast<f32x4*>(dst) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(dst + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
  }
}

// Wide rows: the means of q and q xh of every row first,
template <class T>
__global__ __launch_bounds__(1024) void sgmv_layer_norm_stats_kernel(NormParams p) {
  constexpr int TPR = 1024, W = TPR / 64;
  __shared__ float red[2][W][2];
  const int t = threadIdx.x;
  const float count = (float)(p.w8 * 8);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.n; row += gridDim.x, turn ^= 1) {
    const float mean = p.mean[row], r = p.rstd[row];
    float s[2] = {0.f, 0.f};
#pragma unroll 2
    for (int k = t; k < p.w8; k += TPR) {
      float xv[8], yv[8], gv[8];
      unpack8<T>(load_vec(p.X + (row * p.w8 + k) * 8), xv);
      unpack8<T>(load_vec(p.dY + (row * p.w8 + k) * 8), yv);
      fill8(gv, 1.f);
      if (p.gamma != nullptr) unpack8<T>(load_vec(p.gamma + k * 8), gv);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float q = yv[e] * gv[e];
        s[0] += q;
        s[1] = __builtin_fmaf(q, (xv[e] - mean) * r, s[1]);
      }
    }
    row_sums<W, 2>(s, red, turn, t);
    if (t < 2) p.stats[row * 2 + t] = (t ? s[1] : s[0]) / count;
  }
}

// then blocks of rows x 2048 columns, a thread eight columns of all of them.
template <class T>
__global__ __launch_bounds__(kThreads) void sgmv_layer_norm_columns_kernel(NormParams p) {
  const int c8 = blockIdx.y * kThreads + threadIdx.x;
  if (c8 >= p.w8) return;
  const int64_t width = (int64_t)p.w8 * 8, c = (int64_t)c8 * 8;
  const int64_t r0 = (int64_t)blockIdx.x * p.rows_per_block;
  const int64_t r1 = r0 + p.rows_per_block < p.n ? r0 + p.rows_per_block : p.n;
  float sg[8], sb[8], gv[8];
  fill8(sg, 0.f);
  fill8(sb, 0.f);
  fill8(gv, 1.f);
  if (p.gamma != nullptr) unpack8<T>(load_vec(p.gamma + c), gv);
#pragma unroll 2
  for (int64_t row = r0; row < r1; ++row) {
    const float mean = p.mean[row], r = p.rstd[row];
    float xv[8], yv[8];
    unpack8<T>(load_vec(p.X + row * width + c), xv);
    unpack8<T>(load_vec(p.dY + row * width + c), yv);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      xv[e] = (xv[e] - mean) * r;
      sg[e] = __builtin_fmaf(yv[e], xv[e], sg[e]);
      sb[e] += yv[e];
    }
    if (p.dX == nullptr) continue;
    const float m0 = p.stats[row * 2], m1 = p.stats[row * 2 + 1];
    float d[8];
    fill8(d, 0.f);
    if (p.beyond != nullptr) unpack8<T>(load_vec(p.beyond + row * width + c), d);
#pragma unroll
    for (int e = 0; e < 8; ++e) d[e] = r * (yv[e] * gv[e] - m0 - xv[e] * m1) + d[e];
    store_vec(p.dX + row * width + c, pack8<T>(d));
  }
  if (p.planes == nullptr) return;
  float* const dst = p.planes + (int64_t)blockIdx.x * 2 * width + c;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const float(&v)[8] = half ? sb : sg;
    *reinterpret_cast<f32x4*>(dst + half * width) = f32x4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4*>(dst + half * width + 4) = f32x4{v[4], v[5], v[6], v[7]};
  }
}

// ---------------------------------------------------------------- sums of planes
// Workgroup: 64 columns of one output, 16 lanes of four; 64 slices of the planes, joined through LDS in one order.
constexpr int kSumThreads = 1024, kSumCols = 64, kSumSlices = kSumThreads / 16;
template <class T>
__global__ __launch_bounds__(kSumThreads) void sgmv_plane_sum_kernel(const float* planes, int64_t n, int count, int width,
                                                                     uint16_t* out0, uint16_t* out1, int accumulate) {
  __shared__ __attribute__((aligned(16))) float lds[kSumSlices][kSumCols];
  uint16_t* const out = blockIdx.y == 0 ? out0 : out1;
  if (out == nullptr) return;
  const int t = threadIdx.x, slice = t >> 4;
  const int c = blockIdx.x * kSumCols + (t & 15) * 4;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (c < width) {
#pragma unroll 4
    for (int64_t g = slice; g < n; g += kSumSlices) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(planes + (g * count + blockIdx.y) * (int64_t)width + c);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += v[e];
    }
  }
  *reinterpret_cast<f32x4*>(&lds[slice][(t & 15) * 4]) = s;
  __syncthreads();
  const int col = t & 63, part = t >> 6;  // 16 parts of four slices
  float v = 0.f;
#pragma unroll
  for (int x = 0; x < kSumSlices / 16; ++x) v += lds[part * (kSumSlices / 16) + x][col];
  __syncthreads();
  lds[part][col] = v;
  __syncthreads();
  if (t >= kSumCols || blockIdx.x * kSumCols + t >= width) return;
  v = 0.f;
#pragma unroll
  for (int x = 0; x < 16; ++x) v += lds[x][t];
  uint16_t* const dst = out + blockIdx.x * kSumCols + t;
  if (accumulate) v += T::one(*dst);
  *dst = T::round(v);
}

template <class T, int W, int KEEP>
hipError_t launch_norm(const NormParams& p, hipStream_t s) {
  hipLaunchKernelGGL((sgmv_layer_norm_kernel<T, W, KEEP>), dim3((unsigned)p.grid),
                     dim3(W * 64 > kThreads ? W * 64 : kThreads), 0, s, p);
  return hipGetLastError();
}

template <class T>
hipError_t launch_norm_t(const NormParams& p, hipStream_t s) {
  switch (p.variant) {
    case 0: return launch_norm<T, kNormForward[0].waves, kNormForward[0].keep>(p, s);
    case 1: return launch_norm<T, kNormForward[1].waves, kNormForward[1].keep>(p, s);
    case 2: return launch_norm<T, kNormForward[2].waves, kNormForward[2].keep>(p, s);
    case 3: return launch_norm<T, kNormForward[3].waves, kNormForward[3].keep>(p, s);
    case 4: return launch_norm<T, kNormForward[4].waves, kNormForward[4].keep>(p, s);
    case 5: return launch_norm<T, kNormForward[5].waves, kNormForward[5].keep>(p, s);
    case 6: return launch_norm<T, kNormForward[6].waves, kNormForward[6].keep>(p, s);
    case 7: return launch_norm<T, kNormForward[7].waves, kNormForward[7].keep>(p, s);
  }
  hipLaunchKernelGGL((sgmv_layer_norm_wide_kernel<T>), dim3((unsigned)p.grid), dim3(1024), 0, s, p);
  return hipGetLastError();
}

template <class T, int V>
hipError_t launch_norm_back(const NormParams& p, hipStream_t s) {
  constexpr NormVariant v = kNormBackward[V];
  hipLaunchKernelGGL((sgmv_layer_norm_backward_kernel<T, v.waves, v.keep, v.rows>), dim3((unsigned)p.grid),
                     dim3(v.waves * 64 * v.rows), 0, s, p);
  return hipGetLastError();
}

template <class T>
hipError_t launch_norm_back_t(const NormParams& p, hipStream_t s) {
  switch (p.variant) {
    case 0: return launch_norm_back<T, 0>(p, s);
    case 1: return launch_norm_back<T, 1>(p, s);
    case 2: return launch_norm_back<T, 2>(p, s);
    case 3: return launch_norm_back<T, 3>(p, s);
    case 4: return launch_norm_back<T, 4>(p, s);
    case 5: return launch_norm_back<T, 5>(p, s);
    case 6: return launch_norm_back<T, 6>(p, s);
    case 7: return launch_norm_back<T, 7>(p, s);
  }
  if (p.dX != nullptr) {
    hipLaunchKernelGGL((sgmv_layer_norm_stats_kernel<T>), dim3((unsigned)std::min(p.n, 8192)), dim3(1024), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((sgmv_layer_norm_columns_kernel<T>), dim3((unsigned)p.grid, (unsigned)((p.w8 + kThreads - 1) / kThreads)),
                     dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_layer_norm(int dtype, const NormParams& p, hipStream_t stream) {
  if (p.n <= 0) return hipSuccess;
  return dtype == 1 ? launch_norm_t<BF16>(p, stream) : launch_norm_t<F16>(p, stream);
}

hipError_t launch_layer_norm_backward(int dtype, const NormParams& p, hipStream_t stream) {
  if (p.n <= 0) return hipSuccess;
  return dtype == 1 ? launch_norm_back_t<BF16>(p, stream) : launch_norm_back_t<F16>(p, stream);
}

hipError_t launch_plane_sum(int dtype, const float* planes, int64_t count_planes, int32_t count, int32_t width,
                            uint16_t* out0, uint16_t* out1, int32_t accumulate, hipStream_t stream) {
  if (out0 == nullptr && out1 == nullptr) return hipSuccess;
  if (count_planes == 0 && accumulate) return hipSuccess;
  const dim3 grid((unsigned)((width + kSumCols - 1) / kSumCols), (unsigned)count);
  if (dtype == 1)
    hipLaunchKernelGGL((sgmv_plane_sum_kernel<BF16>), grid, dim3(kSumThreads), 0, stream, planes, count_planes, count, width,
                       out0, out1, accumulate);
  else
    hipLaunchKernelGGL((sgmv_plane_sum_kernel<F16>), grid, dim3(kSumThreads), 0, stream, planes, count_planes, count, width,
                       out0, out1, accumulate);
  return hipGetLastError();
}

}  // namespace sgmv
