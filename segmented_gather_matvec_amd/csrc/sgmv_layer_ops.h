// sgmv_layer_ops.h - device helpers shared by the layer kernels (gfx950).
#pragma once

#include "sgmv_device.h"
#include "sgmv_layer.h"
#include "sgmv_mfma_ops.h"
#include "sgmv_units.h"

namespace sgmv {

typedef __attribute__((address_space(3))) void lds_void;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4_ptr;
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// 32 bits of format flags of a raw (untyped) buffer descriptor.
constexpr int kRawBuffer = 0x00020000;
// Byte offset beyond every descriptor made here: such a lane's load returns 0.
constexpr uint32_t kOutOfRange = 0x80000000u;

// Transposing LDS read: of the 4 rows x 16 columns that a group of 16 lanes
// addresses (lane i: 4 values of row i / 4 from column 4 (i % 4)), lane i gets
// column i.  __restrict: without it the compiler takes the read for one that may
// see any load to LDS in flight, and waits for all of them; callers wait for
// the tile that they read.
__device__ inline u32x2 read_transposed(const uint16_t* __restrict p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)p));
}

// v as hi + lo, two 16-bit values: about 16 (bf16) or 22 (fp16) significant
// bits.  A hi that is not finite stands alone (its lo would be NaN).
template <class T>
__device__ inline void split_hi_lo(float v, uint16_t& hi, uint16_t& lo) {
  hi = T::round(v);
  const float h = T::one(hi);
  lo = T::round(__builtin_isfinite(h) ? v - h : 0.f);
}

// Eight fp32 values as hi and lo operand vectors.
template <class T>
__device__ inline void split8(const float (&v)[8], u32x4& hi, u32x4& lo) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    uint16_t h0, l0, h1, l1;
    split_hi_lo<T>(v[2 * w], h0, l0);
    split_hi_lo<T>(v[2 * w + 1], h1, l1);
    hi[w] = (uint32_t)h0 | ((uint32_t)h1 << 16);
    lo[w] = (uint32_t)l0 | ((uint32_t)l1 << 16);
  }
}

// What fp16 dG and dU of a row are divided by: 2^(8 b), b = row_power[i], or kZeroRow (as 0) for a row of zeros.
__device__ inline float power_of(int b) {
  return b == kZeroRow ? 0.f : __uint_as_float((uint32_t)(127 + 8 * b) << 23);
}

// First segment whose end lies beyond row i (num_segs: none), by a 64-ary
// search over the non-decreasing seg_indptr; uniform over the wave.
__device__ inline int first_segment_past(const SegMeta& m, int i) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = m.num_segs;  // the answer is in [lo, lo + n]
  while (n > 0) {
    const int step = (n + 63) / 64;
    const int first = lane * step;
    const int last = (first + step < n ? first + step : n) - 1;
    const bool past = first < n && m.seg_indptr[lo + last + 1] > i;
    const unsigned long long hit = __ballot(past);
    if (hit == 0) return __builtin_amdgcn_readfirstlane(lo + n);
    // The first piece whose last segment ends past i: that one, or one before it there.
    const int f = __builtin_ctzll(hit) * step;
    n = (f + step < n ? f + step : n) - 1 - f;
    lo += f;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// Rank of LoRA k: the table's, or the problem's.
__device__ inline int rank_of(const int32_t* ranks, int rank, int k) {
  return ranks == nullptr ? rank : clamp_rank(ranks[k], rank);
}

// Activations of the gated block (sgmv_act_t): value and derivative in fp32.
// silu: g * sig, sig = 1 / (1 + e^-g);  sig * (1 + g * (1 - sig)).
// Both sigmoids of one exponential that cannot overflow: sig(x) = 1 / (1 + e^-x), sig(-x) = e^-x / (1 + e^-x) for x >= 0.
// tanh gelu: 0.5 g (1 + t) = g * sig(2z), z = sqrt(2/pi) (g + 0.044715 g^3).
__device__ inline float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }
__device__ inline float gelu_arg2(float g) {
  // 2 z = 2 sqrt(2/pi) g (1 + 0.044715 g^2)
  return 1.5957691216057308f * g * __builtin_fmaf(0.044715f * g, g, 1.f);
}
__device__ inline float act_value(int act, float g) { return g * sigmoid(act == 0 ? g : gelu_arg2(g)); }
__device__ inline void act_both(int act, float g, float& value, float& slope) {
  const float z2 = act == 0 ? g : gelu_arg2(g);
  const float x = expf(-fabsf(z2)), r = 1.f / (1.f + x);
  const float s = z2 >= 0.f ? r : x * r;
  const float c = z2 >= 0.f ? x * r : r;  // 1 - s without cancellation
  // d(2z)/dg = 1, or 2 sqrt(2/pi) (1 + 3 * 0.044715 g^2)
  const float d = act == 0 ? 1.f : 1.5957691216057308f * __builtin_fmaf(0.134145f * g, g, 1.f);
  const float t = s * c;  // 0 far out, where d may have overflowed
  value = g * s;
  slope = t == 0.f ? s : __builtin_fmaf(g * d, t, s);
}

}  // namespace sgmv
