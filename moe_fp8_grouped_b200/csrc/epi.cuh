// epi.cuh -- what the row-pass epilogues share: output stores, and for the
// products with a fused epilogue the bias, the kept pre-activations, the
// activation and the residual of 32 consecutive columns of one row.
#pragma once

#include <cuda_bf16.h>

#include "act.cuh"
#include "internal.h"

namespace gmm {

// x * sigmoid(x); -0 for large negative x, where exp(-x) overflows
__device__ __forceinline__ float silu(float x) { return x / (1.0f + expf(-x)); }

__device__ __forceinline__ void st_v8(void *dst, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t a4,
                                      uint32_t a5, uint32_t a6, uint32_t a7) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(a0), "r"(a1), "r"(a2),
               "r"(a3), "r"(a4), "r"(a5), "r"(a6), "r"(a7)
               : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&b);
}

// Stores 32 consecutive outputs of one row.  v8: the destination is 32-byte
// aligned, so each instruction writes one full 32-byte sector.
__device__ __forceinline__ void store_row32(void *out, int64_t off_elems, const float (&v)[32], int out_f32,
                                            bool v8) {
  if (out_f32) {
    float *dst = static_cast<float *>(out) + off_elems;
    if (v8) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        st_v8(dst + 8 * i, __float_as_uint(v[8 * i]), __float_as_uint(v[8 * i + 1]), __float_as_uint(v[8 * i + 2]),
              __float_as_uint(v[8 * i + 3]), __float_as_uint(v[8 * i + 4]), __float_as_uint(v[8 * i + 5]),
              __float_as_uint(v[8 * i + 6]), __float_as_uint(v[8 * i + 7]));
    } else {
      float4 *d4 = reinterpret_cast<float4 *>(dst);
#pragma unroll
      for (int i = 0; i < 8; ++i) d4[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
  } else {
    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(out) + off_elems;
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    if (v8) {
      st_v8(dst, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
      st_v8(dst + 16, w[8], w[9], w[10], w[11], w[12], w[13], w[14], w[15]);
    } else {
      uint4 *d4 = reinterpret_cast<uint4 *>(dst);
#pragma unroll
      for (int i = 0; i < 4; ++i) d4[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
  }
}

__device__ __forceinline__ bool aligned32(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

// o += bias[g, col ..]; the 32 lanes of a warp read the same addresses
__device__ __forceinline__ void epi_bias(const GemmParams &p, int g, int col, float (&o)[32]) {
  if (!p.bias) return;
  const float4 *b = reinterpret_cast<const float4 *>(p.bias + static_cast<int64_t>(g) * p.ncols + col);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 v = __ldg(b + i);
    o[4 * i] += v.x;
    o[4 * i + 1] += v.y;
    o[4 * i + 2] += v.z;
    o[4 * i + 3] += v.w;
  }
}

// o += residual[row, col ..] (row pitch ld_out).  The residual may be the
// output itself: each value is read by the thread that then writes it.
__device__ __forceinline__ void epi_residual(const GemmParams &p, int64_t row, int col, float (&o)[32]) {
  if (!p.residual) return;
  const int64_t off = row * p.ld_out + col;
  if (p.res_f32) {
    const float4 *r = reinterpret_cast<const float4 *>(static_cast<const float *>(p.residual) + off);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 v = r[i];
      o[4 * i] += v.x;
      o[4 * i + 1] += v.y;
      o[4 * i + 2] += v.z;
      o[4 * i + 3] += v.w;
    }
  } else {
    const uint4 *r = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.residual) + off);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = r[i];
      const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&v);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = __bfloat1622float2(h[e]);
        o[8 * i + 2 * e] += f.x;
        o[8 * i + 2 * e + 1] += f.y;
      }
    }
  }
}

__device__ __forceinline__ void epi_keep(const GemmParams &p, int64_t row, int col, const float (&o)[32]) {
  if (p.preact) store_row32(p.preact, row * p.ncols + col, o, 0, aligned32(p.preact));
}

// o: 32 products z of row `row`, columns col ..; on return the outputs
__device__ __forceinline__ void epi_apply(const GemmParams &p, int g, int64_t row, int col, float (&o)[32]) {
  epi_bias(p, g, col, o);
  epi_keep(p, row, col, o);
#define GMM_EPI_ACT(A)                                   \
  case A:                                                \
    _Pragma("unroll") for (int i = 0; i < 32; ++i) o[i] = act_value(A, o[i]); \
    break;
  switch (p.act) {
    GMM_EPI_ACT(GMM_ACT_RELU)
    GMM_EPI_ACT(GMM_ACT_SILU)
    GMM_EPI_ACT(GMM_ACT_GELU)
    GMM_EPI_ACT(GMM_ACT_GELU_TANH)
    default: break;
  }
#undef GMM_EPI_ACT
  epi_residual(p, row, col, o);
}

// o: 32 gate products of row `row` (gate columns col ..), u: the matching up
// products; on return o holds the outputs, columns col ..
__device__ __forceinline__ void epi_swiglu(const GemmParams &p, int g, int64_t row, int col, float (&o)[32],
                                           float (&u)[32]) {
  epi_bias(p, g, col, o);
  epi_bias(p, g, p.swiglu_f + col, u);
  epi_keep(p, row, col, o);
  epi_keep(p, row, p.swiglu_f + col, u);
#pragma unroll
  for (int i = 0; i < 32; ++i) o[i] = silu(o[i]) * u[i];
  epi_residual(p, row, col, o);
}

}  // namespace gmm
