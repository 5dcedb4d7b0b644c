// act.cuh -- the activations of the product epilogues and their slopes, on
// pairs of values (packed fp32 arithmetic).
//
// Every one is built on 2^x and 1 / x from the special-function unit (within
// 2 ulp and 1 ulp): the exact library forms cost several times the
// instructions, and an epilogue of 60 instructions a value outlasts the tensor
// core's work on the tile.  Errors stay below 1e-6 of the magnitudes involved
// (2^-23 * |x| relative for exp(x)), far below the bf16 rounding of the
// results.
//
//   silu       z s, s = 1 / (1 + exp(-z))                slope s + z s (1 - s)
//   gelu       z Phi(z)                                  slope Phi(z) + z phi(z)
//   gelu_tanh  z s(w), w = 2 sqrt(2/pi) (z + 0.044715 z^3)  (1 + tanh(w/2) = 2 s(w))
//
// Phi from its tail: Phi(-a) = exp(-a^2 / 2) t Q(t), t = 1 / (1 + 0.305 a),
// a >= 0, with Q of degree 7 fitted here (weighted least squares with
// re-weighting towards the largest relative error, a in [0, 14]).  The relative
// error of t Q(t) in fp32 is below 4.2e-7 for every a; that of the tail grows
// with the rounded exponent, by about 2^-23 * a^2 / 2 (1.4e-6 up to a = 5,
// 7.7e-6 up to 13).  exp(-a^2 / 2) is shared with phi.
#pragma once

#include <cuda_runtime.h>

#include "gmm_fp8.h"

namespace gmm {

__device__ __forceinline__ float fast_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float fast_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTanhC0 = 1.5957691216057308f;              // 2 sqrt(2 / pi)
constexpr float kTanhC1 = 1.5957691216057308f * 0.044715f;

// 1 / (1 + exp(-x)): 0 and 1 far out (2^x overflows to inf, 1 / inf is 0; what
// would be below 2^-126 is 0 too)
__device__ __forceinline__ float2 sigmoid2(float2 x) {
  const float2 e = __fmul2_rn(x, splat(-kLog2e));
  const float2 d = __fadd2_rn(make_float2(fast_exp2(e.x), fast_exp2(e.y)), splat(1.0f));
  return make_float2(fast_rcp(d.x), fast_rcp(d.y));
}

// Phi(z) and exp(-z^2 / 2)
__device__ __forceinline__ float2 normal_cdf2(float2 z, float2 &e) {
  const float2 a = make_float2(fabsf(z.x), fabsf(z.y));
  const float2 q = __fmul2_rn(__fmul2_rn(a, a), splat(-0.5f * kLog2e));
  e = make_float2(fast_exp2(q.x), fast_exp2(q.y));
  const float2 d = __ffma2_rn(a, splat(0.305f), splat(1.0f));
  const float2 t = make_float2(fast_rcp(d.x), fast_rcp(d.y));
  float2 h = splat(0.03669919818639755f);
  h = __ffma2_rn(h, t, splat(-0.15298834443092346f));
  h = __ffma2_rn(h, t, splat(0.18571697175502777f));
  h = __ffma2_rn(h, t, splat(-0.037976883351802826f));
  h = __ffma2_rn(h, t, splat(0.12102170288562775f));
  h = __ffma2_rn(h, t, splat(0.10342086106538773f));
  h = __ffma2_rn(h, t, splat(0.12246681749820709f));
  h = __ffma2_rn(h, t, splat(0.12163973599672318f));
  const float2 tail = __fmul2_rn(e, __fmul2_rn(t, h));
  return make_float2(z.x > 0.0f ? 1.0f - tail.x : tail.x, z.y > 0.0f ? 1.0f - tail.y : tail.y);
}

// act(z) of the one-input activations
template <int kAct>
__device__ __forceinline__ float2 act2(float2 z) {
  if constexpr (kAct == GMM_ACT_RELU) {
    return make_float2(z.x < 0.0f ? 0.0f : z.x, z.y < 0.0f ? 0.0f : z.y);  // NaN stays
  } else if constexpr (kAct == GMM_ACT_SILU) {
    return __fmul2_rn(z, sigmoid2(z));
  } else if constexpr (kAct == GMM_ACT_GELU) {
    float2 e;
    return __fmul2_rn(z, normal_cdf2(z, e));
  } else if constexpr (kAct == GMM_ACT_GELU_TANH) {
    return __fmul2_rn(z, sigmoid2(__fmul2_rn(z, __ffma2_rn(__fmul2_rn(z, z), splat(kTanhC1), splat(kTanhC0)))));
  } else {
    return z;
  }
}

// d act(z) / dz (ReLU's gradient chooses and has no slope here)
template <int kAct>
__device__ __forceinline__ float2 slope2(float2 z) {
  static_assert(kAct != GMM_ACT_RELU && kAct != GMM_ACT_SWIGLU);
  if constexpr (kAct == GMM_ACT_SILU) {
    const float2 s = sigmoid2(z);
    return __ffma2_rn(__fmul2_rn(z, s), __ffma2_rn(s, splat(-1.0f), splat(1.0f)), s);
  } else if constexpr (kAct == GMM_ACT_GELU) {
    float2 e;
    const float2 c = normal_cdf2(z, e);
    return __ffma2_rn(z, __fmul2_rn(e, splat(0.3989422804014327f)), c);
  } else if constexpr (kAct == GMM_ACT_GELU_TANH) {
    // beyond |z| = 16 the slope is 0 or 1 in fp32; z^2 below stays finite
    const float2 c = make_float2(fminf(fmaxf(z.x, -16.0f), 16.0f), fminf(fmaxf(z.y, -16.0f), 16.0f));
    const float2 c2 = __fmul2_rn(c, c);
    const float2 s = sigmoid2(__fmul2_rn(c, __ffma2_rn(c2, splat(kTanhC1), splat(kTanhC0))));
    const float2 dw = __ffma2_rn(c2, splat(3.0f * kTanhC1), splat(kTanhC0));
    const float2 r = __ffma2_rn(__fmul2_rn(__fmul2_rn(c, s), __ffma2_rn(s, splat(-1.0f), splat(1.0f))), dw, s);
    return make_float2(isnan(z.x) ? z.x : r.x, isnan(z.y) ? z.y : r.y);
  } else {
    return splat(1.0f);
  }
}

}  // namespace gmm
