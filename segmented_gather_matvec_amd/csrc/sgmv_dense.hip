// sgmv_dense.hip - dense products of a layer with the LoRA term (gfx950), for
// any number of rows.
//
// The LoRA paragraph of the Punica README (page "Punica：多 LoRA 模型统一服务框架")
// gives a row x the output x@W + x@A@B.  Four products share one kernel:
//     forward  Y  = X @ W + V @ B_k                       V = s_k X @ A_k
//     gated    G, U = two forwards, H = act(G) * U
//     dX       dX = sum_p (dY_p @ W_p^T + V_p @ A_{p,k}^T) V_p = s_k dY_p @ B_{p,k}^T
//     dW       dW_p = X^T @ dY_p
// A workgroup owns one output tile and walks the contraction in steps of 32.
// Both operand tiles go from memory straight into LDS (no registers), one ring
// slot per step; lanes past the matrix ask for an offset beyond the buffer
// descriptor and get zeros (sgmv_tile.h has the layouts).  Tiles multiply as
// D^T = B^T A^T, so that a lane ends up with four consecutive columns of one row.
// The LoRA term joins before the output: per run of rows that share a LoRA, V's
// hi + lo 16-bit halves (together 16 or 22 bits of fp32's V) times E_k on the
// matrix cores, added to the accumulators in fp32; outputs are rounded once.
//
// Bound, many rows: the matrix cores, and past them the power limit.  The gated 8192 x 4096 -> 11008 product
// runs 1.32 ms, 1.12 PFLOP/s, with the matrix cores busy in 56% of all cycles at a clock that the load
// holds near 1.9 GHz; a plain library product of the same size reaches 1.24 PFLOP/s.  What it took: both operands of
// a step read from LDS between the products of the step before (1.81 -> 1.60 ms), steps of 32 in a ring of four
// slots instead of 64 in two (1.47), LDS swizzles without bank conflicts (the dX product's GPU cycles
// -6%), the LoRA term from LDS behind one barrier (r = 64, 1777 rows: 520 -> 500 us).
// Tile: 8 waves of 128 x 64 accumulators hold 256 x 256; four waves of 128 x 128 spilled.  256 x 256
// reads each operand from LDS least per product; 192 x 256 fills rounds that 256 rows leave short, and
// 128 x 128 small grids (the host's plan has the figures).
// Few rows: HBM, reading W once.  32 x 256 and 64 x 256 tiles, two workgroups a CU with 64 KiB or more of W's loads in
// flight each: one gated row of 4096 -> 11008 streams 181 MB in 33.6 us, 5.4 TB/s.  Contraction splits
// fill the device there; their fp32 planes stay in the Infinity Cache until the epilogue sums them.
#include "sgmv_thin.h"

namespace sgmv {
namespace {

constexpr int kXcds = 8;
constexpr int kGroupRows = 8;  // row tiles that walk the columns together (they share W tiles in an XCD's L2)

template <int MODE, int BM_, int BN_, int WM_, int WN_, int STAGES_, int WAVES_PER_SIMD_>
struct DenseShape {
  static constexpr int WAVES_PER_SIMD = WAVES_PER_SIMD_;
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, STAGES = STAGES_;
  static constexpr int NW = WM * WN;                  // waves
  static constexpr int TM = BM / WM / 16;             // 16-row tiles per wave
  static constexpr int TN = BN / WN / 16;             // 16-column tiles per wave
  static constexpr bool GATED = MODE == kDenseGated;
  static constexpr bool A_T = MODE == kDenseDw;       // stored with the contraction index as row
  static constexpr bool B_T = MODE != kDenseDx;
  static constexpr int NB = GATED ? 2 : 1;            // column sub-tiles (gate, up)
  static constexpr int C = BN / NB;                   // columns of one sub-tile
  // 1 KiB loads per wave and step.  (A 32-row tile is two of them and a 192-row tile twelve: some
  // are loaded twice, the same bytes, so that every wave counts alike.)
  static constexpr int LA = (BM / 16 + NW - 1) / NW;
  static constexpr int LB = BN / 16 / NW;
  static constexpr int TNP = TN / NB;                 // 16-column tiles of one projection per wave
  static constexpr int SLOT = (BM + BN) * kDenseK;    // halves of one ring slot
  static_assert(LA * 16 * NW >= BM && LB * 16 * NW == BN, "tile loads split evenly over the waves");
  static_assert(TM * 16 * WM == BM && TNP * NB * 16 * WN == BN, "tile splits evenly over the waves");
};

// Loads a step of E_k (columns n0 .. n0 + C of the forward's B_k [r_k, N], or rows of dX's A_k [N, r_k]) as a B
// operand tile: ranks k0 .. k0+31, or, at ranks up to 16, all of them twice, for V's hi and lo halves.
template <int C, int LOADS, bool T>
__device__ inline void issue_e(const uint16_t* E, int rk, int R, int k0, int N, int n0, uint16_t* lds, int wave,
                               int lane) {
  const int cols = N - n0 < C ? N - n0 : C;
  const uint32_t bytes = T ? (uint32_t)((rk - 1) * N + (N - n0)) * 2u : (uint32_t)(cols * rk) * 2u;
  const auto rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(E + (T ? (int64_t)n0 : (int64_t)n0 * rk)), 0,
                                                    (int)bytes, kRawBuffer);
#pragma unroll
  for (int j = 0; j < LOADS; ++j) {
    const int L = (wave * LOADS + j) % (C / 16);
    uint32_t off;
    if constexpr (T) {
      constexpr int G = C / 8;
      const int k = L * (64 / G) + lane / G;
      const int r = R <= 16 ? k & (R - 1) : k0 + k;
      off = r < rk && (R > 16 || k < 2 * R) ? (uint32_t)(r * N + ((lane % G) ^ swizzle_k<C>(k)) * 8) * 2u : kOutOfRange;
    } else {
      const int k = ((lane & 3) ^ swizzle_r(lane >> 2)) * 8;
      const int r = R <= 16 ? k & (R - 1) : k0 + k;
      off = r < rk && (R > 16 || k < 2 * R) ? (uint32_t)((L * 16 + (lane >> 2)) * rk + r) * 2u : kOutOfRange;
    }
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(lds + L * 512), 16, (int)off, 0, 0, 0);
  }
}

// Adds the LoRA term t to the accumulators' columns J0 .. J0+TNP of the workgroup's tile, run by
// run of rows that share a LoRA.  V's halves of the tile's rows and E_k of up to four
// runs go through the ring's slots (the product is done with them), behind one barrier.
template <class T, int MODE, class S, int J0>
__device__ inline void add_term(const DenseParams& p, const LowRankTerm& t, f32x4 (&acc)[S::TM][S::TN], uint16_t* ring,
                                int m0, int n0, int wave, int lane) {
  constexpr int TM = S::TM, TNP = S::TNP, C = S::C, B0 = S::BM * kDenseK, SLOTS = 4;
  constexpr int LE = C / 16 < S::NW ? 1 : C / 16 / S::NW;
  static_assert(S::STAGES >= SLOTS, "ring slots");
  const SegMeta& sm = p.meta;
  const int ml = lane & 15;
  const int wm = wave / S::WN, wn = wave % S::WN;
  const int R = p.rank;
  const int chunks = R > 32 ? 2 : 1;              // of 32 ranks: B slots of a run
  const int steps = R <= 16 ? 1 : 2 * chunks;     // hi then lo (together at ranks up to 16): A slots
  const int depth = SLOTS / chunks;               // runs at once
  const int mend = m0 + S::BM < p.M ? m0 + S::BM : p.M;
  bool first = true;
  for (int s0 = first_segment_past(sm, m0); s0 < sm.num_segs; s0 += 64) {
    // Metadata of 64 segments at a time, one per lane.
    const int sl = s0 + lane < sm.num_segs ? s0 + lane : sm.num_segs - 1;
    const int lo_l = sm.seg_indptr[sl], end_l = sm.seg_indptr[sl + 1];
    const int hi_l = end_l < sm.n_rows ? end_l : sm.n_rows;
    int k_l = sm.lora_idx[sl];
    if (k_l < 0 || k_l >= sm.num_loras) k_l = -1;
    // (All loads of one LoRA at once: none under a condition of its own.)
    const int k_in = k_l < 0 ? 0 : k_l;
    const uint64_t e_l = t.ptrs[k_in], pair_l = t.pair[k_in];
    const int r_in = rank_of(t.ranks, R, k_in);
    const int r_l = k_l >= 0 && e_l != 0ull && pair_l != 0ull ? r_in : 0;
    const int ns = sm.num_segs - s0 < 64 ? sm.num_segs - s0 : 64;
    int u = 0;
    while (u < ns) {
      // The next `depth` runs with rows in this tile: E_k into their B slots.
      int r0[SLOTS], r1[SLOTS], found = 0;
      __builtin_amdgcn_s_barrier();  // the slots are free
#pragma unroll
      for (int d = 0; d < SLOTS; ++d) {
        r0[d] = r1[d] = 0;
        if (d >= depth) continue;
        for (; u < ns && r1[d] <= r0[d]; ++u) {
          const int lo = __builtin_amdgcn_readlane(lo_l, u), hi = __builtin_amdgcn_readlane(hi_l, u);
          const int rk = __builtin_amdgcn_readlane(r_l, u);
          if (lo >= mend) {
            u = ns;  // no later segment has rows here
            break;
          }
          if (rk <= 0) continue;
          r0[d] = lo > m0 ? lo : m0;
          r1[d] = hi < mend ? hi : mend;
          if (r1[d] <= r0[d]) continue;
          const uint32_t e_lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)e_l, u);
          const uint32_t e_hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(e_l >> 32), u);
          const uint16_t* E = reinterpret_cast<const uint16_t*>(((uint64_t)e_hi << 32) | e_lo);
          for (int c = 0; c < chunks; ++c)
            issue_e<C, LE, S::B_T>(E, rk, R, c * 32, p.N, n0, ring + (d * chunks + c) * S::SLOT + B0, wave, lane);
          found = d + 1;
        }
      }
      if (found == 0) break;
      if (first) {
        TileLoader<S::BM, S::LA, false> lv;
        lv.init(wave, lane, 2 * R);
        for (int a = 0; a < steps; ++a) {
          const int col = a / chunks * R + a % chunks * 32;
          lv.start(t.V16, 2 * R, m0, sm.n_rows, col, col + (2 * R < 32 ? 2 * R : 32));
          lv.issue(ring + a * S::SLOT);
        }
        first = false;
      }
      wait_loads_and_lds<0>();
      __builtin_amdgcn_s_barrier();
#pragma unroll
      for (int d = 0; d < SLOTS; ++d) {
        if (d >= found || r1[d] <= r0[d]) continue;
        constexpr int JN = TNP < 2 ? TNP : 2;  // column tiles at a time (registers)
#pragma unroll
        for (int j0 = 0; j0 < TNP; j0 += JN) {
          u32x4 ef[2][JN];
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < JN; ++j)
              ef[c][j] = read_operand<C, S::B_T>(ring + (d * chunks + (c < chunks ? c : 0)) * S::SLOT + B0,
                                                 (wn * TNP + j0 + j) * 16, lane);
#pragma unroll
          for (int i = 0; i < TM; ++i) {
            const int mb = m0 + (wm * TM + i) * 16;
            if (mb + 16 <= r0[d] || mb >= r1[d]) continue;
            f32x4 sum[JN];
#pragma unroll
            for (int j = 0; j < JN; ++j) sum[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int a = 3; a >= 0; --a) {  // lo halves first
              if (a >= steps) continue;
              const u32x4 vf = read_operand<S::BM, false>(ring + a * S::SLOT, (wm * TM + i) * 16, lane);
              if (chunks > 1 && (a & 1)) {
#pragma unroll
                for (int j = 0; j < JN; ++j) sum[j] = mfma<T>(ef[1][j], vf, sum[j]);
              } else {
#pragma unroll
                for (int j = 0; j < JN; ++j) sum[j] = mfma<T>(ef[0][j], vf, sum[j]);
              }
            }
            // The rows of the run take their sum: what another LoRA's matrices hold must not
            // reach them (fp16: scaled back up).
            const int row = mb + ml;
            const bool in = row >= r0[d] && row < r1[d];
            const float up = T::kMaxFinite < 1e6f ? t.row_scale[in ? row : r0[d]] : 1.f;
#pragma unroll
            for (int j = 0; j < JN; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                acc[i][J0 + j0 + j][e] =
                    in ? __builtin_fmaf(sum[j][e], up, acc[i][J0 + j0 + j][e]) : acc[i][J0 + j0 + j][e];
          }
        }
      }
      wait_loads_and_lds<0>();
    }
    if (__builtin_amdgcn_readlane(lo_l, ns - 1) >= mend) return;
  }
}

// The largest and the smallest of the powers of rows 0 .. n-1 but for rows of zeros (kZeroRow and its opposite: all are).
template <int WAVES>
__device__ inline void power_range(const int8_t* power, int n, int* lds, int& top, int& low) {
  const int t = threadIdx.x;
  top = kZeroRow;
  low = -kZeroRow;
  for (int i = t * 4; i < n; i += WAVES * 64 * 4) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(power + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int b = (int8_t)(w >> (8 * e));
      const bool row = i + e < n && b != kZeroRow;
      top = row && b > top ? b : top;
      low = row && b < low ? b : low;
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int a = __shfl_xor(top, d, 64), b = __shfl_xor(low, d, 64);
    top = a > top ? a : top;
    low = b < low ? b : low;
  }
  if ((t & 63) == 0) {
    lds[t >> 6] = top;
    lds[WAVES + (t >> 6)] = low;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    top = lds[w] > top ? lds[w] : top;
    low = lds[WAVES + w] < low ? lds[WAVES + w] : low;
  }
  __syncthreads();  // lds may be filled
  top = __builtin_amdgcn_readfirstlane(top);
  low = __builtin_amdgcn_readfirstlane(low);
}

// The fp16 factor 2^(8 (b - top)) of a row with power b <= top, in the low half (0 below the smallest denormal).
__device__ inline uint32_t power_factor(int b, int top) {
  const uint32_t d = (uint32_t)(top - b);
  const uint32_t f = (uint32_t)(0x000101001c003c00ull >> (16 * (d & 3))) & 0xffffu;
  return d < 4 ? f : 0u;
}
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x8 __attribute__((ext_vector_type(8)));
typedef const __attribute__((address_space(4))) u32x8* const_u32x8_ptr;  // read by scalar loads: no vector load to wait for
// Brings operands of contraction rows row .. row + 31 (lane q: rows 8 q .. 8 q + 7, two to a word) to the power top.
template <int TN>
__device__ inline void bring_to_power(const int8_t* power, int row, int top, int q, u32x4 (&v)[TN]) {
  const u32x8 words = *(const_u32x8_ptr)(power + row);
  const auto word = [&](int e) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)words[e]); };  // (keeps the load scalar)
  const uint32_t odd = 0u - (uint32_t)(q & 1), upper = 0u - (uint32_t)(q >> 1);
  uint32_t f[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = (word(h) & ~odd) | (word(2 + h) & odd), hi = (word(4 + h) & ~odd) | (word(6 + h) & odd);
    const uint32_t w = (lo & ~upper) | (hi & upper);
#pragma unroll
    for (int e = 0; e < 2; ++e)
      f[2 * h + e] = power_factor((int8_t)(w >> (16 * e)), top) | (power_factor((int8_t)(w >> (16 * e + 8)), top) << 16);
  }
#pragma unroll
  for (int j = 0; j < TN; ++j)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t x = v[j][w];  // (a bit cast of the vector's element itself would take element 0)
      v[j][w] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, x) * __builtin_bit_cast(f16x2, f[w]));
    }
}

template <class T>
__device__ inline u32x2 round4(const f32x4& v) {
  return u32x2{(uint32_t)T::round(v[0]) | ((uint32_t)T::round(v[1]) << 16),
               (uint32_t)T::round(v[2]) | ((uint32_t)T::round(v[3]) << 16)};
}

// TERM: compiled with the LoRA term in the tiles.
template <class T, int MODE, class S, bool TERM>
__device__ inline void dense_body(const DenseParams& p, int block, uint16_t* ring) {
  constexpr int STAGES = S::STAGES, TM = S::TM, TN = S::TN, TNP = S::TNP;
  constexpr int B0 = S::BM * kDenseK;  // a slot: A, then B
  uint16_t* lds[STAGES];
#pragma unroll
  for (int s = 0; s < STAGES; ++s) lds[s] = ring + s * S::SLOT;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
  const int q = lane >> 4, ml = lane & 15;

  // Tile of this workgroup: workgroup b runs on XCD b % 8; each XCD takes a
  // contiguous run of the tile order, in which kGroupRows row tiles walk the
  // columns together.
  const int tiles = p.tiles_m * p.tiles_n;
  const int total = tiles * p.ksplit;
  const int per_xcd = (total + kXcds - 1) / kXcds;
  const int idx = (block % kXcds) * per_xcd + block / kXcds;
  if (idx >= total || block / kXcds >= per_xcd) return;
  const int g = idx / tiles;
  const int t = idx - g * tiles;
  const int group = t / (kGroupRows * p.tiles_n);
  const int gr = p.tiles_m - group * kGroupRows < kGroupRows ? p.tiles_m - group * kGroupRows : kGroupRows;
  const int in_group = t - group * kGroupRows * p.tiles_n;
  const int m0 = (group * kGroupRows + in_group % gr) * S::BM;
  const int n0 = (in_group / gr) * S::C;
  const int proj = MODE == kDenseDw ? (int)blockIdx.y : 0;

  // Steps of the contraction: all of pair 0, then all of pair 1.
  const int kt = (p.K + kDenseK - 1) / kDenseK;
  constexpr bool PAIRS = MODE == kDenseDx || MODE == kDenseDw;
  const int steps_all = kt * (PAIRS ? p.pairs : 1);
  const int first = g * p.ktiles_per_split;
  const int last = first + p.ktiles_per_split < steps_all ? first + p.ktiles_per_split : steps_all;

  TileLoader<S::BM, S::LA, S::A_T> la;
  // A gated tile's columns are two sub-tiles; each wave loads pieces of one of them.
  TileLoader<S::C, S::LB, S::B_T> lb;
  constexpr int WB = S::NW / S::NB;  // waves that load one sub-tile
  const int sub = wave / WB;
  la.init(wave, lane, p.lda);
  lb.init(wave - sub * WB, lane, p.ldb);

  // Steps first .. last - 1 of the contraction, in order; dX and dW may go on from pair 0 to pair 1.
  auto start = [&](int s) {
    const int pair = PAIRS && s >= kt ? 1 : 0;
    const int k0 = (s - pair * kt) * kDenseK;
    const int in_pair = (last - pair * kt < kt ? last - pair * kt : kt) * kDenseK;
    const int K = in_pair < p.K ? in_pair : p.K;
    const int bi = MODE == kDenseDw ? proj : S::GATED ? sub : pair;
    la.start(MODE == kDenseDx && pair ? p.A[1] : p.A[0], p.lda, m0, p.M, k0, K);
    const int64_t behind = MODE == kDenseDw && pair ? (int64_t)p.K * p.ldb : 0;
    lb.start((bi ? p.B[1] : p.B[0]) + behind, p.ldb, n0, p.N, k0, K);
  };
  int left_in_pair = kt - first;  // steps before the second pair starts
  auto issue = [&](int slot) {
    la.issue(lds[slot]);
    lb.issue(lds[slot] + B0 + sub * S::C * kDenseK);
    if constexpr (PAIRS) {
      if (--left_in_pair == 0 && last > kt) start(kt);
    }
  };

  // fp16 dG and dU come with a power of two per row.  dX puts it back row by row.  In dW rows meet: where
  // their powers differ, all are brought to the largest on their way from LDS to the matrix cores (a row's values keep
  // their bits down to 2^-21 .. 2^-28 of the largest row's largest value, and count down to 2^-32 .. 2^-40 of it).
  constexpr bool POWERS = T::kMaxFinite < 1e6f && PAIRS;
  int top = 0, low = 0;
  // (In the ring's memory, before it is filled: a second array in LDS made the compiler wait for every load in flight.)
  if constexpr (POWERS && MODE == kDenseDw) {
    if (p.row_power != nullptr) power_range<S::NW>(p.row_power, p.K, reinterpret_cast<int*>(ring), top, low);
  }
  float row_w[TM];  // dX, asked for ahead of the contraction
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    row_w[i] = 1.f;
    if constexpr (POWERS && MODE == kDenseDx) {
      const int m = m0 + (wm * TM + i) * 16 + ml;
      if (p.row_power != nullptr && m < p.M) row_w[i] = power_of(p.row_power[m < p.meta.n_rows ? m : m - p.meta.n_rows]);
    }
  }

  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  u32x4 a[TM], b[2][TN];
  auto read_a = [&](int slot, int i) { a[i] = read_operand<S::BM, S::A_T>(lds[slot], (wm * TM + i) * 16, lane); };
  auto read_b = [&](int slot, u32x4 (&v)[TN]) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
      v[j] = read_operand<S::C, S::B_T>(lds[slot] + B0 + (j / TNP) * S::C * kDenseK, (wn * TNP + j % TNP) * 16, lane);
  };
  auto multiply = [&](int i, const u32x4 (&v)[TN]) {
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = mfma<T>(v[j], a[i], acc[i][j]);
  };

  if (last > first) {
    // A step's operands are read while the step before it multiplies, row tile
    // by row tile into the registers that its products leave.  After the first
    // HB row tiles of a step every wave holds all of the step's operands and the
    // next step's tile has landed: behind that one barrier the slot is refilled, a whole
    // ring ahead, and the reads of the next step begin.  (Steps past the end
    // are zeros, so the ring may turn whole.)
    constexpr int kPerStep = S::LA + S::LB;  // loads of one wave per step
    constexpr int HB = TM / 2;
    constexpr int TURN = STAGES % 2 ? 2 * STAGES : STAGES;  // steps per loop: slots and b[] at fixed places
    start(first);
#pragma unroll
    for (int s = 0; s < STAGES; ++s) issue(s);
    wait_loads_and_lds<kPerStep*(STAGES - 1)>();
    __builtin_amdgcn_s_barrier();
    read_b(0, b[0]);
#pragma unroll
    for (int i = 0; i < TM; ++i) read_a(0, i);
    for (int step = first; step < last; step += TURN) {
#pragma unroll
      for (int s = 0; s < TURN; ++s) {
        constexpr int kAhead = kPerStep * (STAGES - 2);
        const int slot = s % STAGES, next = (s + 1) % STAGES;
        if constexpr (POWERS && MODE == kDenseDw) {
          if (low < top) {
            const int in_pair = step + s < kt ? step + s : step + s - kt;  // (steps past the end hold zeros)
            bring_to_power(p.row_power, (in_pair < kt ? in_pair : kt - 1) * kDenseK, top, q, b[s % 2]);
          }
        }
#pragma unroll
        for (int i = 0; i < HB; ++i) multiply(i, b[s % 2]);
        wait_loads_and_lds<kAhead>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        read_b(next, b[(s + 1) % 2]);
        issue(slot);
#pragma unroll
        for (int i = HB; i < TM; ++i) {
          read_a(next, i - HB);
          multiply(i, b[s % 2]);
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = TM - HB; i < TM; ++i) read_a(next, i);
      }
    }
    wait_loads_and_lds<0>();  // no load may be in flight when the workgroup ends
  }

  // Epilogue.  acc[i][j][e]: row m0 + (wm TM + i) 16 + ml, column 16-tile j, 4 q + e.
  const int mw = m0 + wm * TM * 16;
  const int cw = n0 + wn * TNP * 16;
  if constexpr (POWERS) {
    if (p.row_power != nullptr) {
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const float w = MODE == kDenseDx ? row_w[i] : power_of(top);
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] *= w;
      }
    }
  }
  if constexpr (TERM) {
    if (p.term_in_tile && g == 0) {
      if constexpr (S::GATED) {
        if (p.term[0].V16 != nullptr) add_term<T, MODE, S, 0>(p, p.term[0], acc, ring, m0, n0, wave, lane);
        if (p.term[1].V16 != nullptr) add_term<T, MODE, S, TNP>(p, p.term[1], acc, ring, m0, n0, wave, lane);
      } else {
        for (int t = 0; t < (MODE == kDenseDx ? p.pairs : 1); ++t) {
          const LowRankTerm term{nullptr, t ? p.term[1].V16 : p.term[0].V16,
                                 t ? p.term[1].row_scale : p.term[0].row_scale,
                                 t ? p.term[1].ptrs : p.term[0].ptrs, t ? p.term[1].pair : p.term[0].pair,
                                 t ? p.term[1].ranks : p.term[0].ranks};
          if (term.V16 != nullptr) add_term<T, MODE, S, 0>(p, term, acc, ring, m0, n0, wave, lane);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int m = mw + i * 16 + ml;
#pragma unroll
    for (int j = 0; j < TNP; ++j) {
      const int c = cw + j * 16 + q * 4;
      if (m >= p.M || c >= p.N) continue;
      const int64_t o = (int64_t)m * p.N + c;
      if (p.to_planes) {
        const int64_t pl = (int64_t)(proj * p.ksplit + g) * p.plane_stride + o;
        *reinterpret_cast<f32x4*>(p.planes + pl) = acc[i][j];
        if constexpr (S::GATED)
          *reinterpret_cast<f32x4*>(p.planes + pl + (int64_t)p.ksplit * p.plane_stride) = acc[i][TNP + j];
      } else if constexpr (S::GATED) {
        const f32x4 gv = acc[i][j], uv = acc[i][TNP + j];
        f32x4 h;
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = act_value(p.act, gv[e]) * uv[e];
        if (p.out[0]) *reinterpret_cast<u32x2*>(p.out[0] + o) = round4<T>(gv);
        if (p.out[1]) *reinterpret_cast<u32x2*>(p.out[1] + o) = round4<T>(uv);
        *reinterpret_cast<u32x2*>(p.out[2] + o) = round4<T>(h);
      } else {
        f32x4 v = acc[i][j];
        uint16_t* dst = (MODE == kDenseDw && proj ? p.out[1] : p.out[0]);
        if (MODE == kDenseDw && p.accumulate) {
          const u32x2 old = *reinterpret_cast<const u32x2*>(dst + o);
          v[0] += T::lo(old[0]);
          v[1] += T::hi(old[0]);
          v[2] += T::lo(old[1]);
          v[3] += T::hi(old[1]);
        }
        *reinterpret_cast<u32x2*>(dst + o) = round4<T>(v);
      }
    }
  }
}

template <class T, int MODE, class S>
__global__ __launch_bounds__(S::NW * 64, S::WAVES_PER_SIMD) void sgmv_dense_kernel(DenseParams p) {
  __shared__ __attribute__((aligned(1024))) uint16_t lds[S::STAGES * S::SLOT];
  dense_body<T, MODE, S, MODE != kDenseDw>(p, (int)blockIdx.x, lds);
}

// One of two parameter blocks, field by field: a conditional copy of the struct
// would go through the stack.
__device__ inline ThinParams pick(const ThinParams& a, const ThinParams& b, bool first) {
  ThinParams t;
  t.Z = first ? a.Z : b.Z;
  t.ptrs = first ? a.ptrs : b.ptrs;
  t.ranks = first ? a.ranks : b.ranks;
  t.scales = first ? a.scales : b.scales;
  t.V = first ? a.V : b.V;
  t.V16 = nullptr;  // V stays in planes, or is the one plane
  t.row_scale = nullptr;
  t.planes = first ? a.planes : b.planes;
  t.to_planes = a.to_planes;
  t.sum_planes = 0;
  t.row_k = first ? a.row_k : b.row_k;
  t.z_power = nullptr;
  t.q_power = nullptr;
  t.K = a.K;
  t.rank = a.rank;
  t.transposed = 0;
  t.units = a.units;
  t.direct = a.direct;
  t.ksplit = a.ksplit;
  t.kc = a.kc;
  t.meta = a.meta;
  return t;
}

// The first dense_grid workgroups are the dense product's, the others thin
// products' (nothing waits for anything): while the dense ones stream W, the thin
// ones fill the slots that are left.
template <class T, int MODE, class S>
__global__ __launch_bounds__(kThreads, S::WAVES_PER_SIMD) void sgmv_dense_thin_kernel(DenseParams p, ThinParams t0,
                                                                                       ThinParams t1, int dense_grid,
                                                                                       int thin_grid) {
  constexpr int RING = S::STAGES * S::SLOT;
  static_assert(S::NW == kWaves && RING >= ThinShape<4>::LDS, "one workgroup size, one LDS ring");
  __shared__ __attribute__((aligned(1024))) uint16_t lds[RING];
  const int b = (int)blockIdx.x;
  if (b < dense_grid) {
    dense_body<T, MODE, S, false>(p, b, lds);  // the epilogue adds the term
    return;
  }
  const int x = b - dense_grid;
  const ThinParams t = pick(t0, t1, x < thin_grid);
  const int item = x < thin_grid ? x : x - thin_grid;
  if (p.rank <= 16)
    thin_body<T, 1, false>(t, item, lds);
  else if (p.rank == 32)
    thin_body<T, 2, false>(t, item, lds);
  else
    thin_body<T, 4, false>(t, item, lds);
}

// ---------------------------------------------------------------- epilogue of the partial planes
// One wave per (row i, 256 columns): lane l owns columns c .. c+3.  Sums the
// planes in plane order; when the tiles did not add the LoRA term, adds
// V[i] @ E_k with vector FMA in fp32 (decode, short segments: a row brings its own E_k).
// Bound by the latency of its dependent loads: the first kPlanes planes, V's planes and
// the row's LoRA are all asked for before any of them is waited for, then 16 ranks of E_k of both terms:
// 5.0 us for a dense row of 4096, 9.4 us for a gated row of 11008, 12.0 us for 32 gated rows of as many
// LoRAs (22 MB of E_k).  Eight columns per lane and four planes at a time took 11.2 us for the gated row.
constexpr int kPlanes = 8;
constexpr int kEpilogueCols = 256;
typedef const __attribute__((address_space(1))) u32x2* global_u32x2_ptr;
struct PlaneBatch {
  f32x4 a[kPlanes];
};
__device__ inline void load_planes(const DenseParams& p, int proj, int64_t o, int g0, PlaneBatch& x) {
  const float* src = p.planes + (int64_t)proj * p.ksplit * p.plane_stride + o;
#pragma unroll
  for (int u = 0; u < kPlanes; ++u)
    x.a[u] = *reinterpret_cast<const f32x4*>(src + (int64_t)(g0 + u < p.ksplit ? g0 + u : p.ksplit - 1) *
                                                       p.plane_stride);
}
// y = the sum of all planes; x holds the first kPlanes of them.
__device__ inline void plane_sum(const DenseParams& p, int proj, int64_t o, PlaneBatch& x, f32x4& y) {
  y = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int g0 = 0; g0 < p.ksplit; g0 += kPlanes) {
    if (g0 > 0) load_planes(p, proj, o, g0, x);
#pragma unroll
    for (int u = 0; u < kPlanes; ++u) {
      const bool live = g0 + u < p.ksplit;
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = live ? y[e] + x.a[u][e] : y[e];
    }
  }
}

// Ranks j0 .. j0+15 of E_k over the lane's four columns.  Forward, B_k [r_k, N]: m[w] is rank
// j0 + w (half a vector each).  dX, A_k [N, r_k]: m[2 w], m[2 w + 1] are the ranks of column c + w.
template <int MODE>
__device__ inline void load_rows(const DenseParams& p, const uint16_t* E, int rk, int c, int j0, u32x2 (&m)[16]) {
#pragma unroll
  for (int w = 0; w < 16; ++w) {
    const int r = MODE == kDenseDx ? j0 + (w & 3) * 4 : j0 + w;
    const int64_t at = MODE == kDenseDx ? (int64_t)(c + w / 4) * rk + r : (int64_t)r * p.N + c;
    m[w] = __builtin_nontemporal_load((global_u32x2_ptr)(E + (r < rk ? at : 0)));
  }
}
// y += V[i] @ E_k; v: V[i] (LDS); m: ranks 0 .. 15 of E_k.
template <class T, int MODE>
__device__ inline void row_term(const DenseParams& p, const float* v, const uint16_t* E, int rk, int c, u32x2 (&m)[16],
                                f32x4& y) {
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < rk; j0 += 16) {
    if (j0 > 0) load_rows<MODE>(p, E, rk, c, j0, m);
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      const int r = MODE == kDenseDx ? j0 + (w & 3) * 4 : j0 + w;
      if (r >= rk) continue;  // uniform
      const float f[4] = {T::lo(m[w][0]), T::hi(m[w][0]), T::lo(m[w][1]), T::hi(m[w][1])};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (MODE == kDenseDx)
          s[w / 4] = __builtin_fmaf(v[r + e], f[e], s[w / 4]);
        else
          s[e] = __builtin_fmaf(v[r], f[e], s[e]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] += s[e];
}

template <class T, int MODE>
__global__ __launch_bounds__(64) void sgmv_dense_epilogue_kernel(DenseParams p) {
  constexpr int NT = MODE == kDenseForward ? 1 : 2;  // LoRA terms
  constexpr int NP = MODE == kDenseGated ? 2 : 1;    // projections' planes
  constexpr int kBatch = 16;
  __shared__ __attribute__((aligned(16))) float lds_v[NT][64];
  const int lane = threadIdx.x;
  const int i = blockIdx.x;
  const int c = blockIdx.y * kEpilogueCols + lane * 4;
  if (i >= p.M) return;
  const bool terms = !p.term_in_tile && p.meta.num_segs > 0 && p.term[0].V != nullptr;
  int k[NT], end = 0;
#pragma unroll
  for (int t = 0; t < NT; ++t) k[t] = -1;
  if (terms && p.row_k != nullptr) {
    // Covered rows are those before the last segment's end.
    end = p.meta.seg_indptr[p.meta.num_segs];
#pragma unroll
    for (int t = 0; t < NT; ++t) k[t] = p.row_k[(int64_t)t * p.meta.n_rows + i];
  }
  const int64_t vs = (int64_t)p.meta.n_rows * p.rank;
  float vx[NT][kBatch];
  const float* vp[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const bool on = terms && !(t > 0 && MODE == kDenseDx && p.pairs < 2);
    vp[t] = on ? p.term[t].V + (int64_t)i * p.rank + (lane < p.rank ? lane : 0) : nullptr;
    if (on) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) vx[t][u] = vp[t][(u < p.v_planes ? u : p.v_planes - 1) * vs];
    }
  }
  const bool col = c < p.N;
  const int64_t o = (int64_t)i * p.N + (col ? c : 0);
  PlaneBatch x[NP];
#pragma unroll
  for (int n = 0; n < NP; ++n) load_planes(p, n, o, 0, x[n]);

  if (terms) {
    if (p.row_k == nullptr) {
      const int s = first_segment_past(p.meta, i);
      if (s < p.meta.num_segs && p.meta.seg_indptr[s] <= i) k[0] = p.meta.lora_idx[s];
#pragma unroll
      for (int t = 1; t < NT; ++t) k[t] = k[0];
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if (k[t] >= p.meta.num_loras || (p.row_k != nullptr && i >= end)) k[t] = -1;
  }
  const uint16_t* E[NT];
  bool whole[NT];  // both matrices are there (row_k has looked already)
  int rk[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    k[t] = __builtin_amdgcn_readfirstlane(k[t]);
    const bool on = k[t] >= 0 && vp[t] != nullptr;
    E[t] = on ? reinterpret_cast<const uint16_t*>(p.term[t].ptrs[k[t]]) : nullptr;
    whole[t] = p.row_k != nullptr || (on && p.term[t].pair[k[t]] != 0ull);
    rk[t] = on ? rank_of(p.term[t].ranks, p.rank, k[t]) : 0;
  }
  u32x2 m[NT][16];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (E[t] == nullptr) rk[t] = 0;
    if (rk[t] > 0) load_rows<MODE>(p, E[t], rk[t], col ? c : 0, 0, m[t]);
  }
  // V[i] = the sum of its planes, in plane order; lane j holds rank j.
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (vp[t] == nullptr) continue;
    float v = 0.f;
    for (int g0 = 0; g0 < p.v_planes; g0 += kBatch) {
      if (g0 > 0) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) vx[t][u] = vp[t][(g0 + u < p.v_planes ? g0 + u : p.v_planes - 1) * vs];
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) v = g0 + u < p.v_planes ? v + vx[t][u] : v;
    }
    lds_v[t][lane] = v;
    if (!whole[t]) rk[t] = 0;
  }
  __syncthreads();
  if (!col) return;
  f32x4 y;
  plane_sum(p, 0, o, x[0], y);
  row_term<T, MODE>(p, lds_v[0], E[0], rk[0], c, m[0], y);
  if constexpr (MODE == kDenseGated) {
    f32x4 u, h;
    plane_sum(p, 1, o, x[1], u);
    row_term<T, MODE>(p, lds_v[1], E[1], rk[1], c, m[1], u);
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = act_value(p.act, y[e]) * u[e];
    if (p.out[0]) *reinterpret_cast<u32x2*>(p.out[0] + o) = round4<T>(y);
    if (p.out[1]) *reinterpret_cast<u32x2*>(p.out[1] + o) = round4<T>(u);
    *reinterpret_cast<u32x2*>(p.out[2] + o) = round4<T>(h);
  } else {
    if constexpr (MODE == kDenseDx) row_term<T, MODE>(p, lds_v[1], E[1], rk[1], c, m[1], y);
    *reinterpret_cast<u32x2*>(p.out[0] + o) = round4<T>(y);
  }
}

// The epilogue where no LoRA term is left to add: eight values per thread.
template <class T, int MODE>
__global__ __launch_bounds__(kThreads) void sgmv_dense_sum_kernel(DenseParams p) {
  constexpr int NP = MODE == kDenseGated ? 2 : 1;
  const int64_t o = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 8;
  if (o >= (int64_t)p.M * p.N) return;
  float y[NP][8];
#pragma unroll
  for (int n = 0; n < NP; ++n) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      PlaneBatch x;
      f32x4 v;
      load_planes(p, n, o + 4 * h, 0, x);
      plane_sum(p, n, o + 4 * h, x, v);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[n][4 * h + e] = v[e];
    }
  }
  if constexpr (MODE == kDenseGated) {
    float h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = act_value(p.act, y[0][e]) * y[1][e];
    if (p.out[0]) store_vec(p.out[0] + o, pack8<T>(y[0]));
    if (p.out[1]) store_vec(p.out[1] + o, pack8<T>(y[1]));
    store_vec(p.out[2] + o, pack8<T>(h));
  } else {
    store_vec(p.out[0] + o, pack8<T>(y[0]));
  }
}

template <class T, int MODE, int BM, int BN, int WM, int WN, int STAGES, int WPS>
hipError_t launch_tile(const DenseParams& p, hipStream_t s) {
  using S = DenseShape<MODE, BM, BN, WM, WN, STAGES, WPS>;
  const int64_t total = (int64_t)p.tiles_m * p.tiles_n * p.ksplit;
  const int64_t grid = (total + kXcds - 1) / kXcds * kXcds;
  if (grid <= 0 || grid > 0x7fffffff || p.ktiles_per_split < 0) return hipErrorInvalidValue;
  const unsigned gy = MODE == kDenseDw ? (unsigned)p.projections : 1u;
  hipLaunchKernelGGL((sgmv_dense_kernel<T, MODE, S>), dim3((unsigned)grid, gy), dim3(S::NW * 64), 0, s, p);
  return hipGetLastError();
}

template <class T, int MODE, int BM, int BN, int WM, int WN, int STAGES, int WPS>
hipError_t launch_tile_thin(const DenseParams& p, const ThinParams* t, int count, hipStream_t s) {
  using S = DenseShape<MODE, BM, BN, WM, WN, STAGES, WPS>;
  const int64_t total = (int64_t)p.tiles_m * p.tiles_n * p.ksplit;
  const int64_t dense = (total + kXcds - 1) / kXcds * kXcds, thin = (int64_t)t[0].units * t[0].ksplit;
  if (dense <= 0 || thin <= 0 || dense + thin * count > 0x7fffffff || p.term_in_tile) return hipErrorInvalidValue;
  hipLaunchKernelGGL((sgmv_dense_thin_kernel<T, MODE, S>), dim3((unsigned)(dense + thin * count)), dim3(kThreads), 0, s,
                     p, t[0], t[count - 1], (int)dense, (int)thin);
  return hipGetLastError();
}

template <class T, int MODE>
hipError_t launch_mode_thin(int cfg, const DenseParams& p, const ThinParams* t, int count, hipStream_t s) {
  switch (cfg) {
    case kTile128: return launch_tile_thin<T, MODE, 128, 128, 2, 2, 4, 2>(p, t, count, s);
    case kTile64: return launch_tile_thin<T, MODE, 64, 256, 1, 4, 4, 2>(p, t, count, s);
    case kTile32: return launch_tile_thin<T, MODE, 32, 256, 1, 4, 4, 2>(p, t, count, s);
  }
  return hipErrorInvalidValue;
}

template <class T, int MODE>
hipError_t launch_mode(int cfg, const DenseParams& p, hipStream_t s) {
  switch (cfg) {
    case kTile256: return launch_tile<T, MODE, 256, 256, 2, 4, 4, 2>(p, s);
    case kTile192: return launch_tile<T, MODE, 192, 256, 2, 4, 4, 2>(p, s);
    case kTile128: return launch_tile<T, MODE, 128, 128, 2, 2, 4, 2>(p, s);
    case kTile64: return launch_tile<T, MODE, 64, 256, 1, 4, 4, 2>(p, s);
    case kTile32: return launch_tile<T, MODE, 32, 256, 1, 4, 4, 2>(p, s);
  }
  return hipErrorInvalidValue;
}

template <class T>
hipError_t launch_t(int mode, int cfg, const DenseParams& p, hipStream_t s) {
  switch (mode) {
    case kDenseForward: return launch_mode<T, kDenseForward>(cfg, p, s);
    case kDenseGated: return launch_mode<T, kDenseGated>(cfg, p, s);
    case kDenseDx: return launch_mode<T, kDenseDx>(cfg, p, s);
    case kDenseDw:
      return cfg == kTile256 ? launch_tile<T, kDenseDw, 256, 256, 2, 4, 4, 2>(p, s)
                             : launch_tile<T, kDenseDw, 128, 128, 2, 2, 4, 2>(p, s);
  }
  return hipErrorInvalidValue;
}

template <class T, int MODE>
hipError_t launch_epilogue_mode(const DenseParams& p, hipStream_t s) {
  if (p.term_in_tile || p.meta.num_segs <= 0 || p.term[0].V == nullptr) {
    const int64_t blocks = ((int64_t)p.M * p.N / 8 + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffff) return hipErrorInvalidValue;
    hipLaunchKernelGGL((sgmv_dense_sum_kernel<T, MODE>), dim3((unsigned)blocks), dim3(kThreads), 0, s, p);
  } else {
    const dim3 grid((unsigned)p.M, (unsigned)((p.N + kEpilogueCols - 1) / kEpilogueCols));
    hipLaunchKernelGGL((sgmv_dense_epilogue_kernel<T, MODE>), grid, dim3(64), 0, s, p);
  }
  return hipGetLastError();
}

template <class T>
hipError_t launch_epilogue_t(int mode, const DenseParams& p, hipStream_t s) {
  switch (mode) {
    case kDenseForward: return launch_epilogue_mode<T, kDenseForward>(p, s);
    case kDenseGated: return launch_epilogue_mode<T, kDenseGated>(p, s);
    case kDenseDx: return launch_epilogue_mode<T, kDenseDx>(p, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_dense(int dtype, int mode, int cfg, const DenseParams& p, hipStream_t stream) {
  if (p.M <= 0 || p.N <= 0) return hipSuccess;
  return dtype == 1 ? launch_t<BF16>(mode, cfg, p, stream) : launch_t<F16>(mode, cfg, p, stream);
}

hipError_t launch_dense_thin(int dtype, int mode, int cfg, const DenseParams& p, const ThinParams* t, int count,
                             hipStream_t stream) {
  if (p.M <= 0 || p.N <= 0) return hipSuccess;
  if (mode == kDenseGated)
    return dtype == 1 ? launch_mode_thin<BF16, kDenseGated>(cfg, p, t, count, stream)
                      : launch_mode_thin<F16, kDenseGated>(cfg, p, t, count, stream);
  if (mode == kDenseForward)
    return dtype == 1 ? launch_mode_thin<BF16, kDenseForward>(cfg, p, t, count, stream)
                      : launch_mode_thin<F16, kDenseForward>(cfg, p, t, count, stream);
  return hipErrorInvalidValue;
}

hipError_t launch_dense_epilogue(int dtype, int mode, const DenseParams& p, hipStream_t stream) {
  if (p.M <= 0 || p.N <= 0) return hipSuccess;
  return dtype == 1 ? launch_epilogue_t<BF16>(mode, p, stream) : launch_epilogue_t<F16>(mode, p, stream);
}

}  // namespace sgmv
