// sgmv_lowrank.hip - the LoRA side of a layer and of its gradients (gfx950):
// thin products with A_k and B_k^T, the gradients of A_k and B_k, and the
// gated block's elementwise backward.
//
// With y = x@W + s_k (x@A_k)@B_k (LoRA paragraph of the Punica README, page
// "Punica：多 LoRA 模型统一服务框架", with LoRA's scale), V = s_k x@A_k and
// dV = s_k dy@B_k^T:
//     dx  += dV @ A_k^T,   dA_k = sum_i x_i^T dV_i,   dB_k = sum_i V_i^T dy_i.
// All of them read a [rows, thousands] operand once and are bound by memory.
#include "sgmv_tile.h"

namespace sgmv {
namespace {

// ---------------------------------------------------------------- thin products
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
  // fp16 halves hold V only below 65504: a row with a value beyond 32768 is kept
  // scaled down by a power of two (exact), which the reader puts back.
  if constexpr (T::kMaxFinite < 1e6f) {
    float big = 0.f, up = 1.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) big = fmaxf(big, fabsf(v[e]));
    for (int d = 1; d < p.rank / 8; d <<= 1) big = fmaxf(big, shfl_xor(big, d));
    if (big > 32768.f && big < 3.4e38f) {
      const int e = ((int)(__float_as_uint(big) >> 23) & 255) - 127 - 14;  // 1 .. 113
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);
      up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
      for (int x = 0; x < 8; ++x) v[x] *= down;
    }
    if (c == 0) p.row_scale[row] = up;
  }
  u32x4 hi, lo;
  split8<T>(v, hi, lo);
  uint16_t* dst = p.V16 + (int64_t)row * 2 * p.rank + c;
  store_vec(dst, hi);
  store_vec(dst + p.rank, lo);
}

// Workgroup (unit, split): up to 64 rows of one segment (16 per wave) times the
// LoRA's D_k over kc contraction steps; both operands stream through a ring of
// LDS slots (sgmv_tile.h).  Bound by reading Z.
template <class T, int JT, bool TRANSPOSED>
__global__ __launch_bounds__(kThreads) void sgmv_thin_kernel(ThinParams p0, ThinParams p1) {
  const ThinParams& p = blockIdx.y ? p1 : p0;
  constexpr int COLS = JT * 16, STAGES = 6, kPerStep = 2;
  constexpr int B0 = kThinRows * kDenseK, SLOT = (kThinRows + COLS) * kDenseK;
  constexpr int RST = COLS + 4;  // row stride of the result in LDS (floats)
  static_assert(STAGES * SLOT * 2 >= kThinRows * RST * 4, "the result fits the ring");
  __shared__ __attribute__((aligned(1024))) uint16_t lds[STAGES * SLOT];
  const int t = threadIdx.x;
  const int lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int q = lane >> 4, ml = lane & 15;
  const int u = (int)blockIdx.x / p.ksplit;
  const int g = (int)blockIdx.x - u * p.ksplit;
  const Unit un = resolve_unit<kThinRows>(p.meta.seg_indptr, p.meta.lora_idx, p.meta.num_segs, p.meta.num_loras,
                                          p.meta.n_rows, p.direct, u);
  if (un.L <= 0) return;
  const uint16_t* D = reinterpret_cast<const uint16_t*>(p.ptrs[un.k]);
  const int rk = D != nullptr ? rank_of(p.ranks, p.rank, un.k) : 0;
  const float scale = p.scales != nullptr ? p.scales[un.k] : 1.f;
  const int k0 = g * p.kc;
  const int k1 = p.K < k0 + p.kc ? p.K : k0 + p.kc;
  const int steps = rk > 0 ? (k1 - k0 + kDenseK - 1) / kDenseK : 0;

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
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
      la.issue(lds + s * SLOT);
      lb.issue(lds + s * SLOT + B0);
    }
    int slot = 0;
    for (int s = 0; s < steps; ++s) {
      wait_loads_and_lds<kPerStep*(STAGES - 2)>();
      __builtin_amdgcn_s_barrier();
      uint16_t* refill = lds + (slot == 0 ? STAGES - 1 : slot - 1) * SLOT;  // read in the step before this one
      la.issue(refill);
      lb.issue(refill + B0);
      const uint16_t* now = lds + slot * SLOT;
      const u32x4 z = read_operand<kThinRows, false>(now, wave * 16, lane);
#pragma unroll
      for (int j = 0; j < JT; ++j)
        acc[j] = mfma<T>(read_operand<COLS, !TRANSPOSED>(now + B0, j * 16, lane), z, acc[j]);
      slot = slot + 1 == STAGES ? 0 : slot + 1;
    }
    wait_loads_and_lds<0>();
  }
  __syncthreads();
  // acc[j][e]: row 16 wave + ml, rank 16 j + 4 q + e.
  float* res = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int j = 0; j < JT; ++j) *reinterpret_cast<f32x4*>(&res[(wave * 16 + ml) * RST + j * 16 + q * 4]) = acc[j];
  __syncthreads();
  const int per_row = p.rank / 8;
  for (int x = t; x < un.L * per_row; x += kThreads) {
    const int r = x / per_row, c = (x - r * per_row) * 8;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c < rk ? res[r * RST + c + e] * scale : 0.f;
    if (p.ksplit > 1) {
      float* dst = p.planes + ((int64_t)g * p.meta.n_rows + un.r0 + r) * p.rank + c;
      *reinterpret_cast<f32x4*>(dst) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(dst + 4) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
      store_v<T>(p, un.r0 + r, c, v);
    }
  }
}

// V = sum of the planes, in plane order (rows no segment covers hold anything;
// nothing reads them).
template <class T>
__global__ __launch_bounds__(kThreads) void sgmv_thin_sum_kernel(ThinParams p0, ThinParams p1) {
  const ThinParams& p = blockIdx.y ? p1 : p0;
  const int per_row = p.rank / 8;
  const int64_t n = (int64_t)p.meta.n_rows * p.rank;
  const int64_t x = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (x * 8 >= n) return;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int g = 0; g < p.ksplit; ++g) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p.planes + g * n + x * 8);
    const f32x4 b = *reinterpret_cast<const f32x4*>(p.planes + g * n + x * 8 + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] += a[e];
      v[4 + e] += b[e];
    }
  }
  store_v<T>(p, (int)(x / per_row), (int)(x % per_row) * 8, v);
}

// ---------------------------------------------------------------- gradients of A_k and B_k
// Workgroup (column tile, LoRA k, split z): 256 columns of Z, 64 per wave;
// walks the rows of every segment of LoRA k in steps of 32, every nsplit-th
// step its own.  The contraction index is the row, so Z's tile is kept as it
// lies and read with the transposing read; Q (fp32) is split into hi + lo
// halves, stored rank by rank.  fp16 halves need |Q| < 65504: the sums run at a
// power-of-two scale that shrinks when a step's Q would not fit.
template <class T, int JT>
__global__ __launch_bounds__(kThreads) void sgmv_lora_grad_kernel(LoraGradParams p0, LoraGradParams p1) {
  const int ctiles = (p0.C + kLoraGradCols - 1) / kLoraGradCols;
  const int k = (int)blockIdx.x / ctiles;
  const LoraGradParams& p = blockIdx.y ? p1 : p0;
  constexpr int ROWS = kLoraGradRows, COLS = kLoraGradCols, ZST = COLS + 16, QST = ROWS + 8;
  __shared__ __attribute__((aligned(16))) uint16_t lds_z[ROWS * ZST];
  __shared__ __attribute__((aligned(16))) uint16_t lds_q[2][JT * 16 * QST];
  __shared__ int lds_lo[kThreads], lds_hi[kThreads];
  __shared__ int lds_count[kWaves];
  __shared__ float lds_max[kWaves];
  const int t = threadIdx.x;
  const int lane = t & 63;
  const int wave = t >> 6;
  const int q = lane >> 4, ml = lane & 15;
  const int c0 = ((int)blockIdx.x - k * ctiles) * COLS;
  const int z = (int)blockIdx.z;
  const int R = p.rank;
  uint16_t* out = reinterpret_cast<uint16_t*>(p.out[k]);
  const int rk = rank_of(p.ranks, R, k);
  if (out == nullptr || rk <= 0) return;

  f32x4 acc[4][JT];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < JT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  float scale = 1.f;  // of the sums (fp16 only)
  bool any = false;   // LoRA k has rows
  int counter = 0;    // steps of 32 rows so far, over all of its segments

  for (int s0 = 0; s0 < p.meta.num_segs; s0 += kThreads) {
    // The window's segments of LoRA k, in order.
    const int s = s0 + t;
    int lo = 0, hi = 0;
    if (s < p.meta.num_segs && p.meta.lora_idx[s] == k) {
      lo = p.meta.seg_indptr[s];
      hi = p.meta.seg_indptr[s + 1];
      hi = hi < p.meta.n_rows ? hi : p.meta.n_rows;
    }
    const bool hit = lo >= 0 && hi > lo;
    const unsigned long long m = __ballot(hit);
    __syncthreads();
    if (lane == 0) lds_count[wave] = __popcll(m);
    __syncthreads();
    int at = __popcll(m & ((1ull << lane) - 1)), count = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      at += w < wave ? lds_count[w] : 0;
      count += lds_count[w];
    }
    if (hit) {
      lds_lo[at] = lo;
      lds_hi[at] = hi;
    }
    __syncthreads();
    any = any || count > 0;
    for (int e = 0; e < count; ++e) {
      const int lo_e = lds_lo[e], hi_e = lds_hi[e];
      const int steps = (hi_e - lo_e + ROWS - 1) / ROWS;
      // First step of this segment that is this split's.
      int st = (z - counter % p.nsplit + p.nsplit) % p.nsplit;
      counter += steps;
      for (; st < steps; st += p.nsplit) {
        const int r0 = lo_e + st * ROWS;
        const int L = hi_e - r0 < ROWS ? hi_e - r0 : ROWS;
        // Z: 32 rows x 32 vectors of 8 columns, 4 per thread; rows past the segment are zero.
        u32x4 zv[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int r = (t >> 5) + 8 * x, c = c0 + (t & 31) * 8;
          const bool ok = r < L && c < p.C;
          zv[x] = load_vec(p.Z + (ok ? (int64_t)(r0 + r) * p.C + c : 0));
          if (!ok) zv[x] = u32x4{0u, 0u, 0u, 0u};
        }
        // Q: 32 rows x R values; thread t takes row t % 32, ranks (t / 32) * 2 JT ...
        float qv[2 * JT];
        float big = 0.f;
#pragma unroll
        for (int x = 0; x < 2 * JT; ++x) {
          const int r = t & 31, j = (t >> 5) * 2 * JT + x;
          const bool ok = r < L && j < rk;
          const float v = p.Q[ok ? (int64_t)(r0 + r) * R + j : 0];
          qv[x] = ok ? v : 0.f;
          big = fmaxf(big, fabsf(qv[x]));
        }
        if constexpr (T::kMaxFinite < 1e6f) {
#pragma unroll
          for (int d = 1; d < 64; d <<= 1) big = fmaxf(big, shfl_xor(big, d));
          if (lane == 0) lds_max[wave] = big;
        }
        __syncthreads();  // the last step's tiles are read, the maxima are in
        if constexpr (T::kMaxFinite < 1e6f) {
          big = 0.f;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) big = fmaxf(big, lds_max[w]);
          if (big * scale > 32768.f && big < 3.4e38f) {
            const int ex = ((int)(__float_as_uint(big) >> 23) & 255) - 127 - 14;
            const float next = __uint_as_float((uint32_t)(127 - ex) << 23);
            const float f = next / scale;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int j = 0; j < JT; ++j) acc[i][j] *= f;
            scale = next;
          }
#pragma unroll
          for (int x = 0; x < 2 * JT; ++x) qv[x] *= scale;
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) store_vec(&lds_z[((t >> 5) + 8 * x) * ZST + (t & 31) * 8], zv[x]);
#pragma unroll
        for (int x = 0; x < 2 * JT; ++x) {
          uint16_t h, l;
          split_hi_lo<T>(qv[x], h, l);
          const int a = ((t >> 5) * 2 * JT + x) * QST + (t & 31);
          lds_q[0][a] = h;
          lds_q[1][a] = l;
        }
        __syncthreads();
        u32x4 qh[JT], ql[JT];
#pragma unroll
        for (int j = 0; j < JT; ++j) {
          qh[j] = load_vec(&lds_q[0][(j * 16 + ml) * QST + q * 8]);
          ql[j] = load_vec(&lds_q[1][(j * 16 + ml) * QST + q * 8]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint16_t* a = &lds_z[(q * 8 + (ml >> 2)) * ZST + wave * 64 + i * 16 + (ml & 3) * 4];
          const u32x2 l2 = read_transposed(a), h2 = read_transposed(a + 4 * ZST);
          const u32x4 zf = {l2[0], l2[1], h2[0], h2[1]};
#pragma unroll
          for (int j = 0; j < JT; ++j) {
            // rank_major: lane holds 4 columns of one rank; else 4 ranks of one column
            if (p.rank_major) {
              acc[i][j] = mfma<T>(zf, ql[j], acc[i][j]);
              acc[i][j] = mfma<T>(zf, qh[j], acc[i][j]);
            } else {
              acc[i][j] = mfma<T>(ql[j], zf, acc[i][j]);
              acc[i][j] = mfma<T>(qh[j], zf, acc[i][j]);
            }
          }
        }
      }
    }
    __syncthreads();  // the list is read before the next window overwrites it
  }
  // A LoRA without rows keeps what it has when gradients accumulate.
  if (p.accumulate && !any) return;
  const float inv = 1.f / scale;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < JT; ++j) {
      const int c = c0 + wave * 64 + i * 16 + (p.rank_major ? q * 4 : ml);
      const int r = j * 16 + (p.rank_major ? ml : q * 4);
      if (c >= p.C || r >= rk) continue;
      f32x4 v = acc[i][j];
      if constexpr (T::kMaxFinite < 1e6f) v *= inv;
      if (p.nsplit > 1) {
        float* dst = p.planes + ((int64_t)z * p.meta.num_loras + k) * p.C * R +
                     (p.rank_major ? (int64_t)r * p.C + c : (int64_t)c * R + r);
        *reinterpret_cast<f32x4*>(dst) = v;
      } else {
        uint16_t* dst = out + (p.rank_major ? (int64_t)r * p.C + c : (int64_t)c * rk + r);
        if (p.accumulate) {
          const u32x2 old = *reinterpret_cast<const u32x2*>(dst);
          v[0] += T::lo(old[0]);
          v[1] += T::hi(old[0]);
          v[2] += T::lo(old[1]);
          v[3] += T::hi(old[1]);
        }
        *reinterpret_cast<u32x2*>(dst) =
            u32x2{(uint32_t)T::round(v[0]) | ((uint32_t)T::round(v[1]) << 16),
                  (uint32_t)T::round(v[2]) | ((uint32_t)T::round(v[3]) << 16)};
      }
    }
}

// Sums the splits' planes of one LoRA's gradient (split order), four values per thread.
template <class T>
__global__ __launch_bounds__(kThreads) void sgmv_lora_grad_sum_kernel(LoraGradParams p0, LoraGradParams p1) {
  const int64_t blocks = ((int64_t)p0.C * p0.rank / 4 + kThreads - 1) / kThreads;  // of one LoRA
  const int k = (int)(blockIdx.x / blocks);
  const LoraGradParams& p = blockIdx.y ? p1 : p0;
  const int R = p.rank;
  uint16_t* out = reinterpret_cast<uint16_t*>(p.out[k]);
  const int rk = rank_of(p.ranks, R, k);
  if (out == nullptr || rk <= 0) return;
  if (p.accumulate) {  // a LoRA without rows keeps what it has
    bool any = false;
    for (int s0 = 0; s0 < p.meta.num_segs && !any; s0 += kThreads) {
      const int s = s0 + (int)threadIdx.x;
      const bool hit = s < p.meta.num_segs && p.meta.lora_idx[s] == k && p.meta.seg_indptr[s + 1] > p.meta.seg_indptr[s];
      any = __syncthreads_or(hit);
    }
    if (!any) return;
  }
  const int64_t n = (int64_t)p.C * rk;
  const int64_t o = ((int64_t)(blockIdx.x - k * blocks) * kThreads + threadIdx.x) * 4;  // of the stored gradient
  if (o >= n) return;
  // Planes hold [C][rank] or [rank][C]; the stored [C, r_k] has its own row length.
  const int64_t src = p.rank_major ? o : o / rk * R + o % rk;
  const int64_t stride = (int64_t)p.meta.num_loras * p.C * R;
  const float* pl = p.planes + (int64_t)k * p.C * R + src;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  for (int g = 0; g < p.nsplit; ++g) v += *reinterpret_cast<const f32x4*>(pl + g * stride);
  if (p.accumulate) {
    const u32x2 old = *reinterpret_cast<const u32x2*>(out + o);
    v[0] += T::lo(old[0]);
    v[1] += T::hi(old[0]);
    v[2] += T::lo(old[1]);
    v[3] += T::hi(old[1]);
  }
  *reinterpret_cast<u32x2*>(out + o) = u32x2{(uint32_t)T::round(v[0]) | ((uint32_t)T::round(v[1]) << 16),
                                             (uint32_t)T::round(v[2]) | ((uint32_t)T::round(v[3]) << 16)};
}

// ---------------------------------------------------------------- gated block, elementwise backward
// Eight values per thread; bound by memory (three reads, two writes).  dG and
// dU are the matrix cores' operands of everything that follows, so they are
// rounded to the 16-bit format here, once.
template <class T>
__global__ __launch_bounds__(kThreads) void sgmv_gate_backward_kernel(int act, const uint16_t* G, const uint16_t* U,
                                                                      const uint16_t* dH, uint16_t* dG, uint16_t* dU,
                                                                      int64_t n8) {
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n8; i += (int64_t)gridDim.x * kThreads) {
    float g[8], u[8], h[8], a[8], b[8];
    unpack8<T>(load_stream(G + i * 8), g);
    unpack8<T>(load_stream(U + i * 8), u);
    unpack8<T>(load_stream(dH + i * 8), h);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float value, slope;
      act_both(act, g[e], value, slope);
      a[e] = h[e] * u[e] * slope;
      b[e] = h[e] * value;
    }
    store_vec(dG + i * 8, pack8<T>(a));
    store_vec(dU + i * 8, pack8<T>(b));
  }
}

template <class T, int JT>
hipError_t launch_thin_j(const ThinParams* p, int count, hipStream_t s) {
  const ThinParams& a = p[0];
  const ThinParams& b = p[count - 1];
  const dim3 grid((unsigned)((int64_t)a.units * a.ksplit), (unsigned)count);
  if (a.transposed)
    hipLaunchKernelGGL((sgmv_thin_kernel<T, JT, true>), grid, dim3(kThreads), 0, s, a, b);
  else
    hipLaunchKernelGGL((sgmv_thin_kernel<T, JT, false>), grid, dim3(kThreads), 0, s, a, b);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.ksplit <= 1) return e;
  const int64_t items = (int64_t)a.meta.n_rows * a.rank / 8;
  hipLaunchKernelGGL((sgmv_thin_sum_kernel<T>), dim3((unsigned)((items + kThreads - 1) / kThreads), (unsigned)count),
                     dim3(kThreads), 0, s, a, b);
  return hipGetLastError();
}

template <class T>
hipError_t launch_thin_t(const ThinParams* p, int count, hipStream_t s) {
  switch (p[0].rank) {
    case 8:
    case 16: return launch_thin_j<T, 1>(p, count, s);
    case 32: return launch_thin_j<T, 2>(p, count, s);
    case 64: return launch_thin_j<T, 4>(p, count, s);
  }
  return hipErrorInvalidValue;
}

template <class T>
hipError_t launch_lora_grad_t(const LoraGradParams* p, int count, hipStream_t s) {
  const LoraGradParams& a = p[0];
  const LoraGradParams& b = p[count - 1];
  const int64_t tiles = (int64_t)((a.C + kLoraGradCols - 1) / kLoraGradCols) * a.meta.num_loras;
  const int64_t blocks = ((int64_t)a.C * a.rank / 4 + kThreads - 1) / kThreads * a.meta.num_loras;
  if (tiles > 0x7fffffff || blocks > 0x7fffffff) return hipErrorInvalidValue;
  const dim3 grid((unsigned)tiles, (unsigned)count, (unsigned)a.nsplit);
  switch (a.rank) {
    case 8:
    case 16: hipLaunchKernelGGL((sgmv_lora_grad_kernel<T, 1>), grid, dim3(kThreads), 0, s, a, b); break;
    case 32: hipLaunchKernelGGL((sgmv_lora_grad_kernel<T, 2>), grid, dim3(kThreads), 0, s, a, b); break;
    case 64: hipLaunchKernelGGL((sgmv_lora_grad_kernel<T, 4>), grid, dim3(kThreads), 0, s, a, b); break;
    default: return hipErrorInvalidValue;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.nsplit <= 1) return e;
  hipLaunchKernelGGL((sgmv_lora_grad_sum_kernel<T>), dim3((unsigned)blocks, (unsigned)count), dim3(kThreads), 0, s, a,
                     b);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_thin(int dtype, const ThinParams* p, int count, hipStream_t stream) {
  if (count < 1 || p[0].units <= 0) return hipSuccess;
  return dtype == 1 ? launch_thin_t<BF16>(p, count, stream) : launch_thin_t<F16>(p, count, stream);
}

hipError_t launch_lora_grad(int dtype, const LoraGradParams* p, int count, hipStream_t stream) {
  if (count < 1 || p[0].meta.num_loras <= 0) return hipSuccess;
  return dtype == 1 ? launch_lora_grad_t<BF16>(p, count, stream) : launch_lora_grad_t<F16>(p, count, stream);
}

hipError_t launch_gate_backward(int dtype, int act, const uint16_t* G, const uint16_t* U, const uint16_t* dH,
                                uint16_t* dG, uint16_t* dU, int64_t n, hipStream_t stream) {
  const int64_t n8 = n / 8;
  if (n8 <= 0) return hipSuccess;
  const unsigned grid = (unsigned)(n8 < (int64_t)kThreads * 8192 ? (n8 + kThreads - 1) / kThreads : 8192);
  if (dtype == 1)
    hipLaunchKernelGGL((sgmv_gate_backward_kernel<BF16>), dim3(grid), dim3(kThreads), 0, stream, act, G, U, dH, dG, dU, n8);
  else
    hipLaunchKernelGGL((sgmv_gate_backward_kernel<F16>), dim3(grid), dim3(kThreads), 0, stream, act, G, U, dH, dG, dU, n8);
  return hipGetLastError();
}

}  // namespace sgmv
