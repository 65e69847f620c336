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

// Activations of the dense call with an epilogue (sgmv_act_t), and their slopes, by the hardware's exponential and reciprocal:
// good to some units in the last place (and |x| 2^-23 of the argument's own rounding), far below a 16-bit output's rounding, at
// a third of the instructions of expf and a division, which show in a tile's epilogue and bound an elementwise pass
// (dZ of 8192 x 11008: 133 us by expf and a division where reading and writing alone take 104).
constexpr int kActSilu = 0, kActGeluTanh = 1, kActNone = 2, kActRelu = 3, kActGelu = 4;
__device__ inline float exp_of(float x) { return __builtin_amdgcn_exp2f(1.4426950408889634f * x); }
__device__ inline float fast_sigmoid(float x) { return __builtin_amdgcn_rcpf(1.f + exp_of(-x)); }
// Phi(-a) for a >= 0, the normal distribution's tail, and E = e^(-a^2 / 2): E t q(t), t = 1 / (1 + 0.35 a), where
// q is smooth, positive and bounded, so that its polynomial (least squares of the relative error on 0 <= a <= 15, reweighted
// until the extremes level; 5.0e-8 with its numbers rounded to fp32) gives the tail a relative error below (a^2 + 10) 2^-24, the
// rounding of a^2 and a unit in the last place each of the hardware's reciprocal and exponential included.
// (erfcf in its place cost gelu of 8192 x 11008 92 us of the tiles, now 40.)
__device__ inline float normal_tail(float a, float& E) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(a, 0.35f, 1.f));
  E = __builtin_amdgcn_exp2f(-0.7213475204444817f * (a * a));
  float q = -0.02916393242776394f;
  q = __builtin_fmaf(q, t, 0.14406083524227142f);
  q = __builtin_fmaf(q, t, -0.25590193271636963f);
  q = __builtin_fmaf(q, t, 0.15939298272132874f);
  q = __builtin_fmaf(q, t, -0.02326388657093048f);
  q = __builtin_fmaf(q, t, 0.1055748239159584f);
  q = __builtin_fmaf(q, t, 0.11981549113988876f);
  q = __builtin_fmaf(q, t, 0.13986434042453766f);
  q = __builtin_fmaf(q, t, 0.13962125778198242f);
  return E * t * q;
}
template <int N, class V>
__device__ inline void act_apply(int act, V& z) {
  if (act == kActRelu) {
#pragma unroll
    for (int e = 0; e < N; ++e) z[e] = z[e] < 0.f ? 0.f : z[e];  // (NaN stays)
  } else if (act == kActSilu) {
#pragma unroll
    for (int e = 0; e < N; ++e) z[e] *= fast_sigmoid(z[e]);
  } else if (act == kActGeluTanh) {
#pragma unroll
    for (int e = 0; e < N; ++e) z[e] *= fast_sigmoid(gelu_arg2(z[e]));
  } else if (act == kActGelu) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      float E;
      const float tail = normal_tail(fabsf(z[e]), E);
      z[e] *= z[e] > 0.f ? 1.f - tail : tail;
    }
  }
}
// z *= the derivative at z's place in x.
template <int N>
__device__ inline void act_slopes(int act, const float (&x)[N], float (&z)[N]) {
  if (act == kActRelu) {
#pragma unroll
    for (int e = 0; e < N; ++e) z[e] = x[e] > 0.f ? z[e] : x[e] != x[e] ? x[e] : 0.f * z[e];
  } else if (act == kActGelu) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      // (The slope is 0 or 1 long before 20; an infinite x would make NaN of it.)
      const float v = x[e] < -20.f ? -20.f : x[e] > 20.f ? 20.f : x[e];
      float E;
      const float tail = normal_tail(fabsf(v), E);
      z[e] *= __builtin_fmaf(v * 0.3989422804014327f, E, v > 0.f ? 1.f - tail : tail);
    }
  } else {
    // s + x s (1 - s) d, with 1 - s = e^-x s, free of cancellation.  silu: d = 1, and 0 or 1 to within 1e-33 beyond 80;
    // tanh gelu: the slope is 0 or 1 to within 1e-19 beyond 8.
    const float far = act == kActSilu ? 80.f : 8.f;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float v = x[e] < -far ? -far : x[e] > far ? far : x[e];
      const float a = act == kActSilu ? v : gelu_arg2(v);
      const float d = act == kActSilu ? v : v * 1.5957691216057308f * __builtin_fmaf(0.134145f * v, v, 1.f);
      const float p = exp_of(-a), s = __builtin_amdgcn_rcpf(1.f + p);
      z[e] *= __builtin_fmaf(d * s, p * s, s);
    }
  }
}

}  // namespace sgmv
