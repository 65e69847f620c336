// sgmv_lowrank.hip - the LoRA side of a layer and of its gradients (gfx950):
// thin products with A_k and B_k^T, the gradients of A_k and B_k, and the
// gated block's elementwise backward.
//
// With y = x@W + s_k (x@A_k)@B_k (LoRA paragraph of the Punica README, page
// "Punica：多 LoRA 模型统一服务框架", with LoRA's scale), V = s_k x@A_k and
// dV = s_k dy@B_k^T:
//     dx  += dV @ A_k^T,   dA_k = sum_i x_i^T dV_i,   dB_k = sum_i V_i^T dy_i.
// All of them read a [rows, thousands] operand once and are bound by memory.
#include <algorithm>

#include "sgmv_thin.h"

namespace sgmv {
namespace {

// ---------------------------------------------------------------- thin products
// The products of one launch (grid y).
struct ThinBatch {
  ThinParams p[kMaxThin];
};

template <class T, int JT>
__global__ __launch_bounds__(kThreads) void sgmv_thin_kernel(ThinBatch batch) {
  __shared__ __attribute__((aligned(1024))) uint16_t lds[ThinShape<JT>::LDS];
  const ThinParams& p = batch.p[blockIdx.y];
  if ((int)blockIdx.x >= p.units * p.ksplit) return;
  if (p.transposed)
    thin_body<T, JT, true>(p, (int)blockIdx.x, lds);
  else
    thin_body<T, JT, false>(p, (int)blockIdx.x, lds);
}

// V = sum of the planes, in plane order (rows no segment covers hold anything;
// nothing reads them).
template <class T>
__global__ __launch_bounds__(kThreads) void sgmv_thin_sum_kernel(ThinBatch batch) {
  const ThinParams& p = batch.p[blockIdx.y];
  if (p.sum_planes < 1) return;  // written by the product itself, or part of another's sum
  constexpr int kBatch = 8;   // planes in flight
  const int per_row = p.rank / 8;
  const int64_t n = (int64_t)p.meta.n_rows * p.rank;
  const int64_t x = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (x * 8 >= n) return;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int g0 = 0; g0 < p.sum_planes; g0 += kBatch) {
    f32x4 a[kBatch], b[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const float* src = p.planes + (g0 + u < p.sum_planes ? g0 + u : p.sum_planes - 1) * n + x * 8;
      a[u] = *reinterpret_cast<const f32x4*>(src);
      b[u] = *reinterpret_cast<const f32x4*>(src + 4);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const bool live = g0 + u < p.sum_planes;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = live ? v[e] + a[u][e] : v[e];
        v[4 + e] = live ? v[4 + e] + b[u][e] : v[4 + e];
      }
    }
  }
  store_v<T>(p, (int)(x / per_row), (int)(x % per_row) * 8, v);
}

// ---------------------------------------------------------------- gradients of A_k and B_k
// Workgroup (column tile, LoRA k, split z): 256 columns of Z, 64 per wave; walks
// the rows of every segment of LoRA k in steps of 32, every nsplit-th step its
// own.  The contraction index is the row, so both operands (Z, and V16's rows
// [hi | lo]) are kept as they lie and read with the transposing read; they
// stream through a ring of LDS slots (sgmv_tile.h).  Bound by reading Z, 512 bytes of 32 rows a step: 4096 rows
// of 4096 and 4096 columns, r = 16, 24 us (2.8 TB/s); the four gradients of a gated layer 4096 -> 11008 at
// r = 64, 94 us (2.6 TB/s).  V16 comes from L2 once per column tile: at 256 columns and r = 64 half as many
// bytes as Z.  Splits of the rows fill the device when there are few LoRAs; their planes are not atomics, so that sums keep
// one order.
// fp16 rows of V16 are kept divided by a power of two each (store_v), and rows of different powers may not
// meet in a product (bringing one row to another's power would cost it bits): the matrix cores sum rows of one power, and where it
// changes, their sum joins the total in fp32.  A step whose rows differ is multiplied once per power, the other rows
// masked to zeros.  Most steps have one power and cost a comparison.
// Up to four gradients in one launch (grid y).
struct LoraGradBatch {
  LoraGradParams p[4];
};

template <class T, int R>
struct LoraGradShape {
  static constexpr bool F16T = T::kMaxFinite < 1e6f;
  static constexpr int ROWS = kDenseK, COLS = kLoraGradCols, QC = 2 * R, JT = R < 16 ? 1 : R / 16;
  static constexpr int STAGES = R >= 32 ? 3 : 4;
  static constexpr int B0 = COLS * ROWS, S0 = B0 + QC * ROWS, SLOT = S0 + (F16T ? 128 : 0);  // Z, V16, row scales
  static constexpr int LIST = 2 * kThreads + kWaves;  // ints: the segments of one window
  static_assert(2 * (STAGES * SLOT * 2 + LIST * 4) <= 160 << 10, "two workgroups per CU");
};

// All bits set where x is 0, else none.
__device__ inline uint32_t is_zero(uint32_t x) { return (x < 1u ? x : 1u) - 1u; }
// The largest value of lanes l, l + 16, l + 32, l + 48 (the same for all l): uniform.
__device__ inline uint32_t max_over_q(uint32_t x) {
#pragma unroll
  for (int d = 16; d < 64; d <<= 1) {
    const uint32_t y = (uint32_t)__shfl_xor((int)x, d, 64);
    x = x > y ? x : y;
  }
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)x);
}

// RANK_MAJOR: a lane ends up with 4 columns of one rank; else with 4 ranks of one column.
template <class T, int R, bool RANK_MAJOR>
__device__ inline void lora_grad_body(const LoraGradParams& p, uint16_t* lds, int* lds_lo, int* lds_hi, int* lds_count) {
  using S = LoraGradShape<T, R>;
  constexpr bool F16T = S::F16T;
  constexpr int ROWS = S::ROWS, COLS = S::COLS, QC = S::QC, JT = S::JT, STAGES = S::STAGES;
  constexpr int B0 = S::B0, S0 = S::S0, SLOT = S::SLOT;
  constexpr int LZ = COLS / 16 / kWaves, LQ = QC / 16 < kWaves ? 1 : QC / 16 / kWaves;
  constexpr int kPerStep = LZ + LQ + (F16T ? 1 : 0);
  const int ctiles = (p.C + COLS - 1) / COLS;
  const int tile = (int)blockIdx.x % ctiles, item = p.first + (int)blockIdx.x / ctiles;
  if (item >= p.last || (int)blockIdx.z >= p.nsplit) return;
  const int k = p.by_segment ? p.meta.lora_idx[item] : item;
  if (k < 0 || k >= p.meta.num_loras) return;
  const int t = threadIdx.x;
  const int lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int q = lane >> 4, ml = lane & 15;
  const int c0 = tile * COLS;
  const int z = (int)blockIdx.z;
  uint16_t* out = reinterpret_cast<uint16_t*>(p.out[k]);
  const int rk = rank_of(p.ranks, R, k);
  if (out == nullptr || rk <= 0) return;

  TileLoader<COLS, LZ, true> lz;
  TileLoader<QC, LQ, true> lq;
  lz.init(wave, lane, p.C);
  lq.init(wave, lane, QC);
  f32x4 acc[4][JT];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < JT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  // fp16: what acc is to be multiplied by, and the sums of other powers.
  float unit = 0.f;
  f32x4 total[F16T ? 4 : 1][F16T ? JT : 1];
#pragma unroll
  for (int i = 0; i < (F16T ? 4 : 1); ++i)
#pragma unroll
    for (int j = 0; j < (F16T ? JT : 1); ++j) total[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto fold = [&](float next) {
    if constexpr (F16T) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < JT; ++j) {
#pragma unroll
          for (int e = 0; e < 4; ++e) total[i][j][e] = __builtin_fmaf(acc[i][j][e], unit, total[i][j][e]);
          acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
      unit = next;
    }
  };
  // acc += the products of a slot's rows; lane q holds rows 8 q .. 8 q + 7, two to a word of `mask`.
  auto multiply = [&](const uint16_t* now, const u32x4& mask) {
    u32x4 zf[4], qf[QC / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) zf[i] = read_operand<COLS, true>(now, wave * 64 + i * 16, lane);
#pragma unroll
    for (int j = 0; j < QC / 16; ++j) qf[j] = read_operand<QC, true>(now + B0, j * 16, lane);
    if constexpr (F16T) {
#pragma unroll
      for (int i = 0; i < 4; ++i) zf[i] &= mask;  // both: an infinity times a masked zero is NaN
#pragma unroll
      for (int j = 0; j < QC / 16; ++j) qf[j] &= mask;
    }
#pragma unroll
    for (int j = QC / 16 - 1; j >= 0; --j)  // lo halves first
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[i][j % JT] = RANK_MAJOR ? mfma<T>(zf[i], qf[j], acc[i][j % JT]) : mfma<T>(qf[j], zf[i], acc[i][j % JT]);
  };
  bool any = false;  // LoRA k has rows
  int counter = 0;   // steps of 32 rows so far, over all of its segments

  for (int s0 = 0; s0 < p.meta.num_segs; s0 += kThreads) {
    // The window's segments of LoRA k, in order.
    const int s = s0 + t;
    const int sc = s < p.meta.num_segs ? s : p.meta.num_segs - 1;
    // (k as a lane's value: its pointers come with the lane's other loads.)
    int k_lane = k;
    asm("" : "+v"(k_lane));
    const uint64_t A = p.A[k_lane], B = p.B[k_lane];
    const int id = p.meta.lora_idx[sc], lo = p.meta.seg_indptr[sc];
    int hi = p.meta.seg_indptr[sc + 1];
    hi = hi < p.meta.n_rows ? hi : p.meta.n_rows;
    const bool same = s < p.meta.num_segs && id == k;
    const bool hit = same && lo >= 0 && hi > lo;
    const unsigned long long m = __ballot(hit);
    // By segment: another workgroup has the LoRA if an earlier segment is its.
    if (__syncthreads_or(p.by_segment && same && s < item)) return;
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
    count = __builtin_amdgcn_readfirstlane(count);
    any = any || count > 0;
    // Rows, but a matrix is missing: no gradient.  (Entries of LoRAs without rows are not used.)
    if (any && (__ballot(A == 0 || B == 0) != 0)) return;
    // This split's steps of the window, in order: step st of segment e, which has `steps`.
    int st_first = z - counter % p.nsplit, mine = 0;
    if (st_first < 0) st_first += p.nsplit;
    {
      int all = 0;
      for (int x = lane; x < count; x += 64) all += (lds_hi[x] - lds_lo[x] + ROWS - 1) / ROWS;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) all += __shfl_xor(all, d, 64);
      all = __builtin_amdgcn_readfirstlane(all);
      mine = all > st_first ? (all - st_first + p.nsplit - 1) / p.nsplit : 0;
      counter += all;
    }
    for (int pass = 0; pass < p.passes; ++pass) {
      const uint16_t* Z = p.Z + (int64_t)pass * p.meta.n_rows * p.C;
      int e = -1, st = st_first, row = 0, end = 0, steps = 0;
      auto issue = [&](uint16_t* slot) {
        while (st >= steps && e < count) {  // on to the segment that holds step st
          st -= steps;
          steps = 0;
          if (++e < count) {
            row = __builtin_amdgcn_readfirstlane(lds_lo[e]);
            end = __builtin_amdgcn_readfirstlane(lds_hi[e]);
            steps = (end - row + ROWS - 1) / ROWS;
          }
        }
        const int r0 = e < count ? row + st * ROWS : 0;
        const int n = e < count ? (end - r0 < ROWS ? end - r0 : ROWS) : 0;
        lz.issue_rows(Z, p.C, c0, p.C, r0, n, slot);
        lq.issue_rows(p.Q, QC, 0, QC, r0, n, slot + B0);
        if constexpr (F16T) {
          const auto rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(p.row_scale + r0), 0, n * 4, kRawBuffer);
          __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(slot + S0), 4, lane * 4, 0, 0, 0);
        }
        st += p.nsplit;
      };
      if (mine > 0) {
#pragma unroll
        for (int x = 0; x < STAGES - 1; ++x) issue(lds + x * SLOT);
        int slot = 0;
        for (int x = 0; x < mine; ++x) {
          wait_loads_and_lds<kPerStep*(STAGES - 2)>();
          __builtin_amdgcn_s_barrier();
          issue(lds + (slot == 0 ? STAGES - 1 : slot - 1) * SLOT);
          const uint16_t* now = lds + slot * SLOT;
          // Powers as bits (positive floats compare like integers; arithmetic instead of conditions, whose many scalar
          // masks would spill).
          bool mixed = false;  // a row of another power than the sums'
          uint32_t u[8];
          if constexpr (F16T) {
            const uint32_t* sp = reinterpret_cast<const uint32_t*>(now + S0) + q * 8;
            const u32x4 u0 = *reinterpret_cast<const u32x4*>(sp), u1 = *reinterpret_cast<const u32x4*>(sp + 4);
            uint32_t other = 0;
#pragma unroll
            for (int r = 0; r < 8; ++r) {
              u[r] = r < 4 ? u0[r & 3] : u1[r & 3];
              other |= (u[r] ^ __float_as_uint(unit)) & ~is_zero(u[r]);
            }
            mixed = __ballot(other != 0) != 0;
          }
          // Once, or power by power, largest first; rows of zeros (and past the segment) go with the first.
          uint32_t later = 0;
          u32x4 mask = {~0u, ~0u, ~0u, ~0u};
          do {
            if (mixed) {
              uint32_t next = 0;
#pragma unroll
              for (int r = 0; r < 8; ++r) next = next > u[r] ? next : u[r];
              next = max_over_q(next);
              if (next == 0) break;
              if (next != __float_as_uint(unit)) fold(__uint_as_float(next));
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                uint32_t m[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  m[h] = is_zero(u[2 * w + h] ^ next) | is_zero(u[2 * w + h] | later);
                  u[2 * w + h] &= ~m[h];  // done
                }
                mask[w] = (m[0] & 0xffffu) | (m[1] & 0xffff0000u);
              }
              later = 1;
            }
            multiply(now, mask);
          } while (mixed);
          slot = slot + 1 == STAGES ? 0 : slot + 1;
        }
        wait_loads_and_lds<0>();
      }
      __syncthreads();  // the list and the slots are read before the next pass or window overwrites them
    }
  }
  fold(0.f);
  // A LoRA without rows: zeros, written by split 0, or what it has when gradients accumulate.
  if (!any && (p.accumulate || z > 0)) return;
  const bool planes = p.nsplit > 1 && any;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < JT; ++j) {
      const int c = c0 + wave * 64 + i * 16 + (RANK_MAJOR ? q * 4 : ml);
      const int r = j * 16 + (RANK_MAJOR ? ml : q * 4);
      f32x4 v;
      if constexpr (F16T)
        v = total[i][j];
      else
        v = acc[i][j];
      if constexpr (R == 8) {  // ranks 8..15 are the lo halves' sums of ranks 0..7
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] += RANK_MAJOR ? shfl_xor(v[x], 8) : shfl_xor(v[x], 32);
      }
      if (c >= p.C || r >= rk) continue;
      if (planes) {
        float* dst = p.planes + ((int64_t)z * p.meta.num_loras + k) * p.C * R +
                     (RANK_MAJOR ? (int64_t)r * p.C + c : (int64_t)c * R + r);
        *reinterpret_cast<f32x4*>(dst) = v;
      } else {
        uint16_t* dst = out + (RANK_MAJOR ? (int64_t)r * p.C + c : (int64_t)c * rk + r);
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

template <class T, int R>
__global__ __launch_bounds__(kThreads, 2) void sgmv_lora_grad_kernel(LoraGradBatch batch) {
  using S = LoraGradShape<T, R>;
  __shared__ __attribute__((aligned(1024))) uint16_t lds[S::STAGES * S::SLOT];
  __shared__ int lds_lo[kThreads], lds_hi[kThreads];
  __shared__ int lds_count[kWaves];
  const LoraGradParams& p = batch.p[blockIdx.y];
  if (p.rank_major)
    lora_grad_body<T, R, true>(p, lds, lds_lo, lds_hi, lds_count);
  else
    lora_grad_body<T, R, false>(p, lds, lds_lo, lds_hi, lds_count);
}

// Sums the splits' planes of one LoRA's gradient (split order), and writes the zeros of LoRAs that no
// workgroup has seen: p.turns times four values per thread.  Many turns only where workgroups abound: eight took 19 us for
// six planes of 8 gradients of 4096 x 16 (64 workgroups), one takes 6; and one took 45 us instead of 25 for
// 57 LoRAs' zeros (the search for the LoRA's segments outweighed them).
__host__ __device__ constexpr int64_t sum_blocks(int64_t C, int64_t rank, int turns) {  // of one LoRA
  return (C * rank / 4 + kThreads * turns - 1) / (kThreads * turns);
}
template <class T>
__global__ __launch_bounds__(kThreads) void sgmv_lora_grad_sum_kernel(LoraGradBatch batch) {
  const LoraGradParams& p = batch.p[blockIdx.y];
  const int64_t blocks = sum_blocks(p.C, p.rank, p.turns);
  const int k = p.first + (int)(blockIdx.x / blocks);
  const int64_t block = blockIdx.x % blocks;
  if (k >= p.last) return;
  const int R = p.rank;
  uint16_t* out = reinterpret_cast<uint16_t*>(p.out[k]);
  const int rk = rank_of(p.ranks, R, k);
  if (out == nullptr || rk <= 0) return;
  // A LoRA without rows has no planes; by segment, one without a segment has not been seen at all.
  bool rows = false, seen = false;
  for (int s0 = 0; s0 < p.meta.num_segs && !rows; s0 += kThreads) {
    const int s = s0 + (int)threadIdx.x, sc = s < p.meta.num_segs ? s : p.meta.num_segs - 1;
    const int lo = p.meta.seg_indptr[sc], end = p.meta.seg_indptr[sc + 1];
    const int hi = end < p.meta.n_rows ? end : p.meta.n_rows;
    const bool same = s < p.meta.num_segs && p.meta.lora_idx[sc] == k;
    rows = __syncthreads_or(same && lo >= 0 && hi > lo);
    seen = __syncthreads_or(same) || seen;
  }
  const bool zeros = !seen && p.by_segment && !p.accumulate;
  if (!zeros && (!rows || p.nsplit <= 1 || p.A[k] == 0 || p.B[k] == 0)) return;
  const int64_t n = (int64_t)p.C * rk;
  const int64_t stride = (int64_t)p.meta.num_loras * p.C * R;
  constexpr int kBatch = 8;  // planes in flight
  const int planes = zeros ? 0 : p.nsplit;
  for (int turn = 0; turn < p.turns; ++turn) {
    const int64_t o = ((block * p.turns + turn) * kThreads + threadIdx.x) * 4;
    if (o >= n) return;  // o: of the stored gradient
    // Planes hold [C][rank] or [rank][C]; the stored [C, r_k] has its own row length.
    const float* pl = p.planes + (int64_t)k * p.C * R + (p.rank_major || rk == R ? o : o / rk * R + o % rk);
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    for (int g0 = 0; g0 < planes; g0 += kBatch) {
      f32x4 x[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        x[u] = *reinterpret_cast<const f32x4*>(pl + (g0 + u < planes ? g0 + u : planes - 1) * stride);
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = g0 + u < planes ? v[e] + x[u][e] : v[e];
    }
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
}

// ---------------------------------------------------------------- gated block, elementwise backward
// dG = dH * U * act'(G), dU = dH * act(G).  They are the matrix cores' operands of everything that follows, so they are
// rounded to the 16-bit format here, once.  HALVES (few rows): kept as hi halves and,
// n F values behind them, lo halves, which go through the same products as further rows: those
// are bound by reading W then, and the error of a handful of large values does not average out.
template <class T>
__device__ inline void gate_slopes(int act, const u32x4& G, const u32x4& U, const u32x4& dH, float (&a)[8],
                                   float (&b)[8]) {
  float g[8], u[8], h[8];
  unpack8<T>(G, g);
  unpack8<T>(U, u);
  unpack8<T>(dH, h);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float value, slope;
    act_both(act, g[e], value, slope);
    a[e] = h[e] * u[e] * slope;
    b[e] = h[e] * value;
  }
}
template <class T, bool HALVES>
__device__ inline void store_slopes(const float (&v)[8], uint16_t* dst, int64_t i, int64_t n8) {
  if constexpr (HALVES) {
    u32x4 hi, lo;
    split8<T>(v, hi, lo);
    store_vec(dst + i * 8, hi);
    store_vec(dst + (n8 + i) * 8, lo);
  } else {
    store_vec(dst + i * 8, pack8<T>(v));
  }
}

// bf16: eight values per thread; bound by memory (three reads, two writes: 2048 x 11008 37 us, 6.1 TB/s, part of them from
// the Infinity Cache; with two exponentials per value 50 us).
template <bool HALVES>
__global__ __launch_bounds__(kThreads) void sgmv_gate_backward_kernel(int act, const uint16_t* G, const uint16_t* U,
                                                                      const uint16_t* dH, uint16_t* dG, uint16_t* dU,
                                                                      int64_t n8) {
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n8; i += (int64_t)gridDim.x * kThreads) {
    float a[8], b[8];
    gate_slopes<BF16>(act, load_stream(G + i * 8), load_stream(U + i * 8), load_stream(dH + i * 8), a, b);
    store_slopes<BF16, HALVES>(a, dG, i, n8);
    store_slopes<BF16, HALVES>(b, dU, i, n8);
  }
}

// fp16: |dG| may pass 65504 where the gradients do not, and small values' lo and then hi halves run out of denormals. So a
// row of both is kept divided by a power 2^(8 b) (exact), and the readers put it back.  b brings the row's largest
// |dH| max(1.13 |U|, |G|) to [2^7, 2^15): no |dG| or |dU| is larger, since |act'| <= 1.13 and |act(g)| <= |g|, and it costs
// no exponential; a value then keeps its 11 bits down to 2^-21 of it.  TPR threads share a row, or with few rows
// several workgroups do: each finds the row's power for itself and computes every splits-th piece of TPR eights.
// A thread's first KEEP eights stay in registers meanwhile, the others are read again.
template <bool HALVES, int TPR, int KEEP>
__global__ __launch_bounds__(TPR > kThreads ? TPR : kThreads) void sgmv_gate_backward_rows_kernel(
    int act, const uint16_t* G, const uint16_t* U, const uint16_t* dH, uint16_t* dG, uint16_t* dU, int8_t* power,
    int32_t n, int32_t f8, int32_t splits) {
  constexpr int ROWS = TPR < kThreads ? kThreads / TPR : 1;  // of a workgroup
  static_assert(TPR == 64 || ROWS == 1, "a wave or a workgroup per row");
  __shared__ uint32_t most[TPR / 64];
  const int t = (int)threadIdx.x % TPR;
  const int split = (int)blockIdx.x % splits;
  const int64_t n8 = (int64_t)n * f8;
  const int64_t first = (int64_t)(blockIdx.x / splits) * ROWS + threadIdx.x / TPR;
  for (int64_t row = first; row < n; row += (int64_t)(gridDim.x / splits) * ROWS) {
    const int64_t at = row * f8;
    u32x4 g[KEEP ? KEEP : 1], u[KEEP ? KEEP : 1], h[KEEP ? KEEP : 1];
    // Bits of the largest finite magnitude; 1 (the smallest denormal) for what is neither finite nor 0.
    uint32_t big = 0;
    const auto see = [&](const u32x4& G8, const u32x4& U8, const u32x4& H8) {
      float x[8], y[8], z[8];
      unpack8<F16>(G8, x);
      unpack8<F16>(U8, y);
      unpack8<F16>(H8, z);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t m = __float_as_uint(fabsf(z[e]) * fmaxf(1.13f * fabsf(y[e]), fabsf(x[e])));
        const uint32_t f = m < 0x7f800000u ? m : 1u;
        big = big > f ? big : f;
      }
    };
#pragma unroll
    for (int c = 0; c < KEEP; ++c) {  // (past the end: the row's last eight again, so that all loads are in flight at once)
      const int64_t i = at + (c * TPR + t < f8 ? c * TPR + t : f8 - 1);
      g[c] = load_stream(G + i * 8);
      u[c] = load_stream(U + i * 8);
      h[c] = load_stream(dH + i * 8);
    }
#pragma unroll
    for (int c = 0; c < KEEP; ++c) see(g[c], u[c], h[c]);
#pragma unroll 4
    for (int c = KEEP * TPR; c < f8; c += TPR) {
      const int64_t i = at + (c + t < f8 ? c + t : f8 - 1);
      see(load_vec(G + i * 8), load_vec(U + i * 8), load_vec(dH + i * 8));
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t y = (uint32_t)__shfl_xor((int)big, d, 64);
      big = big > y ? big : y;
    }
    if constexpr (TPR > 64) {
      __syncthreads();  // the row before has been read
      if ((t & 63) == 0) most[t >> 6] = big;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < TPR / 64; ++w) big = big > most[w] ? big : most[w];
    }
    int e = ((int)(big >> 23) - 127 - 7) >> 3;
    e = e < -kMaxRowPower ? -kMaxRowPower : e > kMaxRowPower ? kMaxRowPower : e;
    const float down = power_of(-e);
    if (t == 0 && split == 0) power[row] = (int8_t)(big == 0 ? kZeroRow : e);
    const auto put = [&](const u32x4& G8, const u32x4& U8, const u32x4& H8, int64_t i) {
      float a[8], b[8];
      gate_slopes<F16>(act, G8, U8, H8, a, b);
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        a[x] *= down;
        b[x] *= down;
      }
      store_slopes<F16, HALVES>(a, dG, i, n8);
      store_slopes<F16, HALVES>(b, dU, i, n8);
    };
#pragma unroll
    for (int c = 0; c < KEEP; ++c)
      if (c * TPR + t < f8) put(g[c], u[c], h[c], at + c * TPR + t);
    for (int c = (KEEP + split) * TPR + t; c < f8; c += splits * TPR) {
      const int64_t i = at + c;
      put(load_vec(G + i * 8), load_vec(U + i * 8), load_vec(dH + i * 8), i);
    }
  }
}

template <class T>
hipError_t launch_thin_t(const ThinParams* p, int count, hipStream_t s) {
  ThinBatch batch{};
  int64_t grid = 0;
  bool sums = false;
  for (int i = 0; i < count; ++i) {
    batch.p[i] = p[i];
    grid = std::max(grid, (int64_t)p[i].units * p[i].ksplit);
    sums = sums || p[i].sum_planes > 0;
  }
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  const dim3 g((unsigned)grid, (unsigned)count);
  switch (p[0].rank) {
    case 8:
    case 16: hipLaunchKernelGGL((sgmv_thin_kernel<T, 1>), g, dim3(kThreads), 0, s, batch); break;
    case 32: hipLaunchKernelGGL((sgmv_thin_kernel<T, 2>), g, dim3(kThreads), 0, s, batch); break;
    case 64: hipLaunchKernelGGL((sgmv_thin_kernel<T, 4>), g, dim3(kThreads), 0, s, batch); break;
    default: return hipErrorInvalidValue;
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !sums) return e;
  const int64_t items = (int64_t)p[0].meta.n_rows * p[0].rank / 8;
  hipLaunchKernelGGL((sgmv_thin_sum_kernel<T>), dim3((unsigned)((items + kThreads - 1) / kThreads), (unsigned)count),
                     dim3(kThreads), 0, s, batch);
  return hipGetLastError();
}

// (Segments or LoRAs that take more workgroups than a launch holds, fewer than 2^32 threads, go in several.)
constexpr int64_t kMostWorkgroups = ((int64_t)1 << 32) / kThreads - 1;

template <class T>
hipError_t launch_lora_grad_t(const LoraGradParams* p, int count, hipStream_t s) {
  LoraGradBatch batch{};
  int64_t items = 0, ctiles = 1, quads = 0, blocks = 1;
  int nsplit = 1;
  bool sums = false;
  const int64_t loras = p[0].meta.num_loras;
  for (int i = 0; i < count; ++i) {
    items = std::max<int64_t>(items, p[i].by_segment ? p[i].meta.num_segs : loras);
    ctiles = std::max<int64_t>(ctiles, (p[i].C + kLoraGradCols - 1) / kLoraGradCols);
    nsplit = std::max(nsplit, p[i].nsplit);
    sums = sums || p[i].nsplit > 1 || (p[i].by_segment && !p[i].accumulate);
    quads += loras * sum_blocks(p[i].C, p[i].rank, 1);
  }
  const int turns = (int)std::max<int64_t>(1, std::min<int64_t>(8, quads / 2048));
  for (int i = 0; i < count; ++i) {
    batch.p[i] = p[i];
    batch.p[i].turns = turns;
    blocks = std::max(blocks, sum_blocks(p[i].C, p[i].rank, turns));
  }
  const auto part = [&](int64_t first, int64_t last) {
    for (int i = 0; i < count; ++i) {
      batch.p[i].first = (int32_t)first;
      batch.p[i].last = (int32_t)last;
    }
  };
  const int64_t most = kMostWorkgroups / ctiles;
  for (int64_t first = 0; first < items; first += most) {
    const int64_t n = std::min(most, items - first);
    part(first, first + n);
    const dim3 grid((unsigned)(n * ctiles), (unsigned)count, (unsigned)nsplit);
    switch (p[0].rank) {
      case 8: hipLaunchKernelGGL((sgmv_lora_grad_kernel<T, 8>), grid, dim3(kThreads), 0, s, batch); break;
      case 16: hipLaunchKernelGGL((sgmv_lora_grad_kernel<T, 16>), grid, dim3(kThreads), 0, s, batch); break;
      case 32: hipLaunchKernelGGL((sgmv_lora_grad_kernel<T, 32>), grid, dim3(kThreads), 0, s, batch); break;
      case 64: hipLaunchKernelGGL((sgmv_lora_grad_kernel<T, 64>), grid, dim3(kThreads), 0, s, batch); break;
      default: return hipErrorInvalidValue;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t most_sums = kMostWorkgroups / blocks;
  for (int64_t first = 0; sums && first < loras; first += most_sums) {
    const int64_t n = std::min(most_sums, loras - first);
    part(first, first + n);
    const dim3 grid((unsigned)(n * blocks), (unsigned)count);
    hipLaunchKernelGGL((sgmv_lora_grad_sum_kernel<T>), grid, dim3(kThreads), 0, s, batch);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool HALVES, int TPR, int KEEP>
hipError_t launch_gate_rows(int act, const uint16_t* G, const uint16_t* U, const uint16_t* dH, uint16_t* dG, uint16_t* dU,
                            int8_t* power, int32_t n, int32_t f8, int32_t splits, hipStream_t s) {
  constexpr int rows = TPR < kThreads ? kThreads / TPR : 1;
  const dim3 grid((unsigned)(std::min<int64_t>(((int64_t)n + rows - 1) / rows, 8192) * splits));
  hipLaunchKernelGGL((sgmv_gate_backward_rows_kernel<HALVES, TPR, KEEP>), grid, dim3(TPR < kThreads ? kThreads : TPR), 0, s,
                     act, G, U, dH, dG, dU, power, n, f8, splits);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_thin(int dtype, const ThinParams* p, int count, hipStream_t stream) {
  if (count < 1 || p[0].units <= 0) return hipSuccess;
  if (count > kMaxThin) return hipErrorInvalidValue;
  return dtype == 1 ? launch_thin_t<BF16>(p, count, stream) : launch_thin_t<F16>(p, count, stream);
}

hipError_t launch_lora_grad(int dtype, const LoraGradParams* p, int count, hipStream_t stream) {
  if (count < 1 || p[0].meta.num_loras <= 0) return hipSuccess;
  if (count > 4) return hipErrorInvalidValue;
  return dtype == 1 ? launch_lora_grad_t<BF16>(p, count, stream) : launch_lora_grad_t<F16>(p, count, stream);
}

hipError_t launch_gate_backward(int dtype, int act, bool halves, const uint16_t* G, const uint16_t* U,
                                const uint16_t* dH, uint16_t* dG, uint16_t* dU, int8_t* row_power, int32_t n, int32_t F,
                                hipStream_t stream) {
  const int f8 = F / 8;
  const int64_t n8 = (int64_t)n * f8;
  if (n8 <= 0) return hipSuccess;
  if (dtype == 1) {
    const dim3 grid((unsigned)std::min<int64_t>((n8 + kThreads - 1) / kThreads, 8192));
    if (halves)
      hipLaunchKernelGGL((sgmv_gate_backward_kernel<true>), grid, dim3(kThreads), 0, stream, act, G, U, dH, dG, dU, n8);
    else
      hipLaunchKernelGGL((sgmv_gate_backward_kernel<false>), grid, dim3(kThreads), 0, stream, act, G, U, dH, dG, dU, n8);
    return hipGetLastError();
  }
  const auto rows = [&](auto launch, int splits) {
    return launch(act, G, U, dH, dG, dU, row_power, n, f8, splits, stream);
  };
  // Threads a row, measured on 11008 columns: up to 63 rows several workgroups a row (1 row 6.6 us; one workgroup 12),
  // to 512 rows 1024 threads that hold all (256 rows 12.5 us; 256 threads that read twice 21), beyond, 256
  // threads of up to six eights each (2048 rows 60 us; without rows' powers 55).
  if (halves || n < 64 || (n <= 512 && f8 <= 256)) {
    const int pieces = (f8 + kThreads - 1) / kThreads, splits = std::max(1, std::min(pieces, 1024 / n));
    return halves ? rows(launch_gate_rows<true, 256, 0>, splits) : rows(launch_gate_rows<false, 256, 0>, splits);
  }
  if (n <= 512) return rows(launch_gate_rows<false, 1024, 2>, 1);
  if (f8 <= 256) return rows(launch_gate_rows<false, 64, 4>, 1);
  if (f8 <= 512) return rows(launch_gate_rows<false, 256, 2>, 1);
  if (f8 <= 1024) return rows(launch_gate_rows<false, 256, 4>, 1);
  if (f8 <= 1536) return rows(launch_gate_rows<false, 256, 6>, 1);
  return rows(launch_gate_rows<false, 512, 6>, 1);
}

}  // namespace sgmv
