// sgmv_route.hip - rows sorted by LoRA and back (gfx950): from the LoRA of every (row, choice) the order, its
// inverse and the segments that the library's calls take; rows to their sorted places, and back with weights.
//
// The multi-LoRA paragraph of the Punica README (page "Punica：多 LoRA 模型统一服务框架") binds every row of a
// batch to its own LoRA; the kernels want rows that share one next to each other.  With entries e = i top_k + j,
//     slots[e] = entries of smaller key + earlier entries of the same key     (a stable counting sort; perm is its inverse)
//     Xs[slots[e]] = X[i],   Y[i] = R[i] + sum_j w[e] Ys[slots[e]]
//     dYs[slots[e]] = w[e] dY[i],   dw[e] = <dY[i], Ys[slots[e]]>,   dX[i] = sum_j dXs[slots[e]].
#include <algorithm>

#include "sgmv_block.h"
#include "sgmv_block_shapes.h"
#include "sgmv_layer_ops.h"

namespace sgmv {
namespace {

// ---------------------------------------------------------------- the sort
// One pass over as many keys as there are LoRAs, and one for rows without: no digits, since a histogram of all keys fits
// LDS.  Workgroups count their tiles (first launch, where there are several); each then adds up the
// counts of the tiles before it itself (a launch and a wait less than a scan of its own), and its waves place their
// entries one group of 64 at a time: the lanes of one key find each other by ballots over the key's bits, so that the
// order within a key is the entries' own and no counter's timing shows.
__device__ inline int route_key(const RouteParams& p, int e) {
  const int k = p.ids[e];
  return k >= 0 && k < p.num_loras ? k : p.num_loras;
}

__global__ __launch_bounds__(kRouteThreads) void sgmv_route_count_kernel(RouteParams p) {
  __shared__ int count[kRouteLds / 3];
  const int keys = p.num_loras + 1, t = threadIdx.x;
  for (int k = t; k < keys; k += kRouteThreads) count[k] = 0;
  __syncthreads();
  const int64_t first = (int64_t)blockIdx.x * p.tile;
  const int last = (int)(first + p.tile < p.m ? first + p.tile : p.m);
  for (int64_t e = first + t; e < last; e += kRouteThreads) atomicAdd(&count[route_key(p, (int)e)], 1);
  __syncthreads();
  for (int k = t; k < keys; k += kRouteThreads) p.counts[(int64_t)blockIdx.x * keys + k] = count[k];
}

__global__ __launch_bounds__(kRouteThreads) void sgmv_route_kernel(RouteParams p) {
  __shared__ int lds[kRouteLds];
  __shared__ int wave_sum[kRouteThreads / 64];
  const int keys = p.num_loras + 1, t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  int* const total = lds;          // [keys] entries of each key
  int* const before = lds + keys;  // [keys] of them in earlier tiles
  int* const hist = lds + 2 * keys;  // [waves][keys]
  for (int x = t; x < (p.waves + 2) * keys; x += kRouteThreads) lds[x] = 0;
  __syncthreads();

  // Entries of this wave: a run of whole groups of 64.
  const int per_wave = p.tile / p.waves;
  const int64_t tile = (int64_t)blockIdx.x * p.tile;
  const int64_t first = tile + (int64_t)wave * per_wave;
  const int64_t tile_end = tile + p.tile < p.m ? tile + p.tile : p.m;
  const int64_t last = wave < p.waves ? (first + per_wave < tile_end ? first + per_wave : tile_end) : first;
  int* const mine = hist + wave * keys;
  for (int64_t e = first + lane; e < last; e += 64) atomicAdd(&mine[route_key(p, (int)e)], 1);
  if (p.blocks > 1) {
    // With few keys several threads share one, each with every slices-th tile.  (Sums of integers: their order does not show.)
    int lanes = 64;
    while (lanes < keys && lanes < kRouteThreads) lanes *= 2;
    const int slices = kRouteThreads / lanes;
    for (int k = t & (lanes - 1); k < keys; k += kRouteThreads) {
      int all = 0, early = 0;
#pragma unroll 4
      for (int b = t / lanes; b < p.blocks; b += slices) {
        const int c = p.counts[(int64_t)b * keys + k];
        all += c;
        early += b < (int)blockIdx.x ? c : 0;
      }
      atomicAdd(&total[k], all);
      atomicAdd(&before[k], early);
    }
  }
  __syncthreads();

  // Exclusive scan over the keys: thread t has `per` keys in a row.
  const int per = (keys + kRouteThreads - 1) / kRouteThreads;
  const int k0 = t * per, k1 = k0 + per < keys ? k0 + per : keys;
  int sum = 0;
  for (int k = k0; k < k1; ++k) {
    if (p.blocks == 1) {
      int c = 0;
      for (int w = 0; w < p.waves; ++w) c += hist[w * keys + k];
      total[k] = c;
    }
    sum += total[k];
  }
  int scan = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int up = __shfl_up(scan, d, 64);
    scan += lane >= d ? up : 0;
  }
  if (lane == 63) wave_sum[wave] = scan;
  __syncthreads();
  int at = scan - sum;
  for (int w = 0; w < wave; ++w) at += wave_sum[w];
  for (int k = k0; k < k1; ++k) {
    if (blockIdx.x == 0) {
      if (p.seg_indptr != nullptr) p.seg_indptr[k] = at;
      if (p.lora_idx != nullptr && k < p.num_loras) p.lora_idx[k] = k;
    }
    int place = at + before[k];
    at += total[k];
    for (int w = 0; w < p.waves; ++w) {
      const int c = hist[w * keys + k];
      hist[w * keys + k] = place;
      place += c;
    }
  }
  __syncthreads();
  if (p.perm == nullptr && p.slots == nullptr) return;

  const int bits = 32 - __builtin_clz((unsigned)keys);
  for (int64_t e0 = first; e0 < last; e0 += 64) {
    const bool live = e0 + lane < last;
    const int e = (int)(live ? e0 + lane : last - 1);
    const int key = route_key(p, e);
    unsigned long long same = __ballot(live);
    for (int b = 0; b < bits; ++b) {
      const bool one = (key >> b) & 1;
      const unsigned long long ones = __ballot(one);
      same &= one ? ones : ~ones;
    }
    const int rank = __builtin_popcountll(same & ((1ull << lane) - 1));
    // Every lane reads its key's counter before the first lane of a key moves it on (one wave: LDS accesses
    // keep their order, the fences keep the compiler's).
    const int place = __hip_atomic_load(&mine[key], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT) + rank;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (live && rank == 0)
      __hip_atomic_store(&mine[key], place + (int)__builtin_popcountll(same), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    // (Counts that another call wrote over, or ids that changed under way, must not become places elsewhere.)
    if (live && place >= 0 && place < p.m) {
      if (p.perm != nullptr) p.perm[place] = e;
      if (p.slots != nullptr) p.slots[e] = place;
    }
  }
}

// ---------------------------------------------------------------- rows to their places and back
// Bound by memory: every row is read once and written once (dispatch: written top_k times).  L lanes a row (fewer
// than 64 for narrow rows), V vectors of 16 bytes each; wide rows go over several workgroups (grid y).
constexpr int kRowsVec = 4;

// (A place outside the sorted rows, from slots that no sort made, is passed over.)
__device__ inline bool in_range(int slot, int64_t m) { return slot >= 0 && slot < m; }

template <int L, int V>
__global__ __launch_bounds__(kThreads) void sgmv_dispatch_kernel(RowsParams p) {
  constexpr int ROWS = kThreads / L;
  const int lane = threadIdx.x % L;
  const int c0 = blockIdx.y * L * V + lane;
  const int64_t m = (int64_t)p.n * p.top_k;
  for (int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / L; row < p.n; row += (int64_t)gridDim.x * ROWS) {
    u32x4 x[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = c0 + v * L < p.w8 ? c0 + v * L : p.w8 - 1;
      x[v] = load_stream(p.X + (row * p.w8 + c) * 8);
    }
    for (int j = 0; j < p.top_k; ++j) {
      const int slot = p.slots[row * p.top_k + j];
      if (!in_range(slot, m)) continue;
      uint16_t* dst = p.out + (int64_t)slot * p.w8 * 8;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (c0 + v * L < p.w8) store_stream(dst + (int64_t)(c0 + v * L) * 8, x[v]);
    }
  }
}

// JB: choices whose rows are asked for together.  V: 4 of a wave's vectors where rows are wide and many (one choice, 16384 rows of 4096:
// 61 us with 2, 49 with 4, and 45 with stores past the caches, which cost two choices 37 -> 43), 2 for a few rows (one row
// 2.5 -> 2.2 us).
template <class T, int L, int V, int JB>
__global__ __launch_bounds__(kThreads) void sgmv_combine_kernel(RowsParams p) {
  constexpr int ROWS = kThreads / L;
  const int lane = threadIdx.x % L;
  const int c0 = blockIdx.y * L * V + lane;
  const int64_t m = (int64_t)p.n * p.top_k;
  for (int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / L; row < p.n; row += (int64_t)gridDim.x * ROWS) {
    float y[V][8];
    int c[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      c[v] = c0 + v * L < p.w8 ? c0 + v * L : p.w8 - 1;
#pragma unroll
      for (int e = 0; e < 8; ++e) y[v][e] = 0.f;
    }
    if (p.R != nullptr) {
#pragma unroll
      for (int v = 0; v < V; ++v) unpack8<T>(load_vec(p.R + (row * p.w8 + c[v]) * 8), y[v]);
    }
    for (int j0 = 0; j0 < p.top_k; j0 += JB) {
      float w[JB];
      int slot[JB];
      u32x4 x[JB][V];
#pragma unroll
      for (int u = 0; u < JB; ++u) {
        const int j = j0 + u < p.top_k ? j0 + u : p.top_k - 1;
        slot[u] = p.slots[row * p.top_k + j];
        w[u] = p.weights != nullptr ? p.weights[row * p.top_k + j] : 1.f;
      }
#pragma unroll
      for (int u = 0; u < JB; ++u) {
        if (j0 + u >= p.top_k || !in_range(slot[u], m)) {
          w[u] = 0.f;
          slot[u] = 0;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) x[u][v] = load_stream(p.X + ((int64_t)slot[u] * p.w8 + c[v]) * 8);
      }
#pragma unroll
      for (int u = 0; u < JB; ++u) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float f[8];
          unpack8<T>(x[u][v], f);
          // (A weight of 0 adds nothing, whatever its row holds.)
#pragma unroll
          for (int e = 0; e < 8; ++e) y[v][e] = w[u] != 0.f ? __builtin_fmaf(w[u], f[e], y[v][e]) : y[v][e];
        }
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (c0 + v * L < p.w8) {
        uint16_t* const dst = p.out + (row * p.w8 + c[v]) * 8;
        JB == 1 ? store_stream(dst, pack8<T>(y[v])) : store_vec(dst, pack8<T>(y[v]));
      }
  }
}

// TPE threads an entry (its dot product needs the whole row): a wave where there are entries enough, fewer lanes for narrow
// rows (131072 entries of 64 values: 60 us with a wave each, 10 with eight lanes).
template <class T, int TPE>
__global__ __launch_bounds__(kThreads) void sgmv_combine_backward_kernel(RowsParams p) {
  constexpr int ENTRIES = kThreads / TPE, V = TPE < 64 ? 1 : 4;
  __shared__ float part[kWaves];
  const int t = threadIdx.x % TPE;
  const int64_t m = (int64_t)p.n * p.top_k;
  for (int64_t e0 = (int64_t)blockIdx.x * ENTRIES; e0 < m; e0 += (int64_t)gridDim.x * ENTRIES) {
    const int64_t e = e0 + (TPE < 64 ? (int)threadIdx.x / TPE : __builtin_amdgcn_readfirstlane(threadIdx.x / TPE));
    float dot = 0.f;
    if (e < m) {
      const int64_t row = e / p.top_k;
      const int slot = p.slots[e];
      const bool there = in_range(slot, m);
      const float w = p.weights != nullptr ? p.weights[e] : 1.f;
      const uint16_t* const dy = p.X + row * p.w8 * 8;
      const uint16_t* const ys = p.dweights != nullptr ? p.Ys + (there ? (int64_t)slot : 0) * p.w8 * 8 : dy;
      uint16_t* const dys = there && p.out != nullptr ? p.out + (int64_t)slot * p.w8 * 8 : nullptr;
      for (int c0 = t; c0 < p.w8; c0 += TPE * V) {
        u32x4 a[V], b[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int c = c0 + v * TPE < p.w8 ? c0 + v * TPE : p.w8 - 1;
          a[v] = load_vec(dy + (int64_t)c * 8);
          b[v] = load_stream(ys + (int64_t)c * 8);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const bool live = c0 + v * TPE < p.w8;
          float f[8], g[8];
          unpack8<T>(a[v], f);
          unpack8<T>(b[v], g);
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            dot = live ? __builtin_fmaf(f[x], g[x], dot) : dot;
            f[x] = w != 0.f ? f[x] * w : 0.f;
          }
          if (live && dys != nullptr) store_stream(dys + (int64_t)(c0 + v * TPE) * 8, pack8<T>(f));
        }
      }
      if (!there) dot = 0.f;
    }
    if (p.dweights == nullptr) continue;
#pragma unroll
    for (int d = 1; d < (TPE < 64 ? TPE : 64); d <<= 1) dot += shfl_xor(dot, d);
    if constexpr (TPE > 64) {
      __syncthreads();  // the entry before has been read
      if ((t & 63) == 0) part[t >> 6] = dot;
      __syncthreads();
      dot = 0.f;
#pragma unroll
      for (int x = 0; x < TPE / 64; ++x) dot += part[x];
    }
    if (t == 0 && e < m) p.dweights[e] = dot;
  }
}

constexpr int64_t kMostBlocks = 8192;

// Lanes of a row: 64, or the power of two that holds it.
int lanes_of(int w8) { return w8 > 32 ? 64 : w8 > 16 ? 32 : w8 > 8 ? 16 : 8; }

dim3 rows_grid(const RowsParams& p, int lanes, int vecs) {
  const int64_t rows = kThreads / lanes, per = (int64_t)lanes * vecs;
  return dim3((unsigned)std::min<int64_t>((p.n + rows - 1) / rows, kMostBlocks), (unsigned)((p.w8 + per - 1) / per));
}

template <class T, int L, int V>
hipError_t launch_combine_l(const RowsParams& p, hipStream_t s) {
  const dim3 grid = rows_grid(p, L, V);
  if (p.top_k == 1)
    hipLaunchKernelGGL((sgmv_combine_kernel<T, L, V, 1>), grid, dim3(kThreads), 0, s, p);
  else if (p.top_k == 2)
    hipLaunchKernelGGL((sgmv_combine_kernel<T, L, V, 2>), grid, dim3(kThreads), 0, s, p);
  else
    hipLaunchKernelGGL((sgmv_combine_kernel<T, L, V, 4>), grid, dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

template <class T>
hipError_t launch_combine_t(const RowsParams& p, hipStream_t s) {
  switch (lanes_of(p.w8)) {
    case 8: return launch_combine_l<T, 8, 1>(p, s);
    case 16: return launch_combine_l<T, 16, 1>(p, s);
    case 32: return launch_combine_l<T, 32, 1>(p, s);
  }
  if (p.w8 <= 64) return launch_combine_l<T, 64, 1>(p, s);
  if (p.w8 <= 128 || (int64_t)p.n * p.w8 < (1 << 18)) return launch_combine_l<T, 64, 2>(p, s);
  return launch_combine_l<T, 64, 4>(p, s);
}

template <class T>
hipError_t launch_combine_backward_t(const RowsParams& p, hipStream_t s) {
  const int64_t m = (int64_t)p.n * p.top_k;
  const int lanes = m < 2048 && p.w8 > 64 ? kThreads : lanes_of(p.w8), per = kThreads / lanes;
  const dim3 grid((unsigned)std::min<int64_t>((m + per - 1) / per, kMostBlocks)), block(kThreads);
  switch (lanes) {
    case 8: hipLaunchKernelGGL((sgmv_combine_backward_kernel<T, 8>), grid, block, 0, s, p); break;
    case 16: hipLaunchKernelGGL((sgmv_combine_backward_kernel<T, 16>), grid, block, 0, s, p); break;
    case 32: hipLaunchKernelGGL((sgmv_combine_backward_kernel<T, 32>), grid, block, 0, s, p); break;
    case 64: hipLaunchKernelGGL((sgmv_combine_backward_kernel<T, 64>), grid, block, 0, s, p); break;
    default: hipLaunchKernelGGL((sgmv_combine_backward_kernel<T, kThreads>), grid, block, 0, s, p);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteParams& p, hipStream_t stream) {
  if (p.blocks > 1) {
    hipLaunchKernelGGL(sgmv_route_count_kernel, dim3((unsigned)p.blocks), dim3(kRouteThreads), 0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(sgmv_route_kernel, dim3((unsigned)p.blocks), dim3(kRouteThreads), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_dispatch(const RowsParams& p, hipStream_t stream) {
  if (p.n <= 0) return hipSuccess;
  const int lanes = lanes_of(p.w8);
  const dim3 grid = rows_grid(p, lanes, lanes == 64 ? kRowsVec : 1);
  switch (lanes) {
    case 8: hipLaunchKernelGGL((sgmv_dispatch_kernel<8, 1>), grid, dim3(kThreads), 0, stream, p); break;
    case 16: hipLaunchKernelGGL((sgmv_dispatch_kernel<16, 1>), grid, dim3(kThreads), 0, stream, p); break;
    case 32: hipLaunchKernelGGL((sgmv_dispatch_kernel<32, 1>), grid, dim3(kThreads), 0, stream, p); break;
    default: hipLaunchKernelGGL((sgmv_dispatch_kernel<64, kRowsVec>), grid, dim3(kThreads), 0, stream, p);
  }
  return hipGetLastError();
}

hipError_t launch_combine(int dtype, const RowsParams& p, hipStream_t stream) {
  if (p.n <= 0) return hipSuccess;
  return dtype == 1 ? launch_combine_t<BF16>(p, stream) : launch_combine_t<F16>(p, stream);
}

hipError_t launch_combine_backward(int dtype, const RowsParams& p, hipStream_t stream) {
  if (p.n <= 0 || (p.out == nullptr && p.dweights == nullptr)) return hipSuccess;
  return dtype == 1 ? launch_combine_backward_t<BF16>(p, stream) : launch_combine_backward_t<F16>(p, stream);
}

}  // namespace sgmv
