// epi.cuh -- what the row-pass epilogues share: output stores, and for the
// products with a fused epilogue the bias, the kept pre-activations, the
// activation and the residual.
//
// The E4M3 passes hold a thread's 128 accumulators in registers and finish them
// 32 columns at a time, in one instantiation per activation.  16 columns at a
// time, with narrower stores, ran 5 % slower; a rolled loop over shifted
// accumulators 40 % (it spills them); a chunk's residual loaded while the chunk
// before it is finished 5 to 10 %.  The bf16 family reads its chunks from TMEM
// in one rolled loop.  The activations' instructions are what an epilogue is
// made of: with the exact library forms of act.cuh's functions the Mixtral-like
// up projection (16384 x 4096 x 28672, short runs at full clocks) took 2.4 ms with
// SiLU and 5.1 ms with GELU, with these 1.55 and 1.57 ms (1.48 ms without an
// epilogue).  32 accumulator columns a TMEM load and 232 registers a thread
// instead of 216 or 224 brought them there from 1.64 and 1.66 ms, and SwiGLU with
// a bias and kept z from 1.71 to 1.58 ms.  Pass after pass, under the power cap,
// that product takes 1.90 to 1.95 ms and the plain one 1.68.
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

// Asks L2 for `n` columns of the residual's row, ahead of the product.
__device__ __forceinline__ void epi_prefetch(const GemmParams &p, int64_t row, int col, int n) {
  if (!p.residual) return;
  const int esz = p.res_f32 ? 4 : 2;
  const char *r = static_cast<const char *>(p.residual) + (row * p.ld_out + col) * esz;
  const int cols = static_cast<int>(p.ld_out) - col;  // columns left in the row
  for (int b = 0; b < min(n, cols) * esz; b += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(r + b));
}

__device__ __forceinline__ float2 bf16x2_f32(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// o += bias[g, col ..]; the lanes of a warp read the same addresses
template <int kPairs>
__device__ __forceinline__ void epi_bias(const GemmParams &p, int g, int col, float2 (&o)[kPairs]) {
  if (!p.bias) return;
  const float4 *b = reinterpret_cast<const float4 *>(p.bias + static_cast<int64_t>(g) * p.ncols + col);
#pragma unroll
  for (int i = 0; i < kPairs / 2; ++i) {
    const float4 v = __ldg(b + i);
    o[2 * i] = __fadd2_rn(o[2 * i], make_float2(v.x, v.y));
    o[2 * i + 1] = __fadd2_rn(o[2 * i + 1], make_float2(v.z, v.w));
  }
}

// 2 kPairs (16 or 32) values of one row as bf16
template <int kPairs>
__device__ __forceinline__ void epi_store_bf16(__nv_bfloat16 *dst, const float2 (&o)[kPairs], bool v8) {
  uint32_t w[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) w[i] = pack_bf16x2(o[i].x, o[i].y);
#pragma unroll
  for (int i = 0; i < kPairs; i += 8) {
    if (v8) {
      st_v8(dst + 2 * i, w[i], w[i + 1], w[i + 2], w[i + 3], w[i + 4], w[i + 5], w[i + 6], w[i + 7]);
    } else {
      uint4 *d4 = reinterpret_cast<uint4 *>(dst + 2 * i);
      d4[0] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
      d4[1] = make_uint4(w[i + 4], w[i + 5], w[i + 6], w[i + 7]);
    }
  }
}

template <int kPairs>
__device__ __forceinline__ void epi_keep(const GemmParams &p, int64_t row, int col, const float2 (&o)[kPairs]) {
  if (p.preact)
    epi_store_bf16(static_cast<__nv_bfloat16 *>(p.preact) + row * p.ncols + col, o, aligned32(p.preact));
}

// The residual (bf16: asked for before the activation, added after it).  It
// may be the output itself: each value is read by the thread that then writes
// it.
template <int kPairs>
__device__ __forceinline__ void epi_load_residual(const GemmParams &p, int64_t off, uint4 (&r)[kPairs / 4]) {
  if (!p.residual || p.res_f32) return;
  const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.residual) + off);
#pragma unroll
  for (int i = 0; i < kPairs / 4; ++i) r[i] = src[i];
}

template <int kPairs>
__device__ __forceinline__ void epi_add_residual(const GemmParams &p, int64_t off, const uint4 (&r)[kPairs / 4],
                                                 float2 (&o)[kPairs]) {
  if (!p.residual) return;
  if (p.res_f32) {
    const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(p.residual) + off);
#pragma unroll
    for (int i = 0; i < kPairs / 2; ++i) {
      const float4 v = src[i];
      o[2 * i] = __fadd2_rn(o[2 * i], make_float2(v.x, v.y));
      o[2 * i + 1] = __fadd2_rn(o[2 * i + 1], make_float2(v.z, v.w));
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPairs / 4; ++i) {
      o[4 * i] = __fadd2_rn(o[4 * i], bf16x2_f32(r[i].x));
      o[4 * i + 1] = __fadd2_rn(o[4 * i + 1], bf16x2_f32(r[i].y));
      o[4 * i + 2] = __fadd2_rn(o[4 * i + 2], bf16x2_f32(r[i].z));
      o[4 * i + 3] = __fadd2_rn(o[4 * i + 3], bf16x2_f32(r[i].w));
    }
  }
}

template <int kAct, int kPairs>
__device__ __forceinline__ void epi_act(float2 (&o)[kPairs]) {
#pragma unroll
  for (int i = 0; i < kPairs; ++i) o[i] = act2<kAct>(o[i]);
}

// One chunk: o holds the products of row `row`, columns col .. (for SwiGLU the
// gate columns, u the matching up columns); writes the outputs.
template <int kEpi, int kPairs>
__device__ __forceinline__ void epi_finish(const GemmParams &p, int g, int64_t row, bool sw, int col,
                                           float2 (&o)[kPairs], float2 (&u)[kPairs], bool out_v8) {
  const int64_t off = row * p.ld_out + col;
  uint4 res[kPairs / 4];
  epi_load_residual<kPairs>(p, off, res);
  epi_bias(p, g, col, o);
  epi_keep(p, row, col, o);
  if (sw) {
    epi_bias(p, g, p.swiglu_f + col, u);
    epi_keep(p, row, p.swiglu_f + col, u);
    epi_act<GMM_ACT_SILU>(o);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) o[i] = __fmul2_rn(o[i], u[i]);
  } else if constexpr (kEpi >= 0) {
    epi_act<kEpi>(o);
  } else {
    switch (p.act) {
      case GMM_ACT_RELU: epi_act<GMM_ACT_RELU>(o); break;
      case GMM_ACT_SILU: epi_act<GMM_ACT_SILU>(o); break;
      case GMM_ACT_GELU: epi_act<GMM_ACT_GELU>(o); break;
      case GMM_ACT_GELU_TANH: epi_act<GMM_ACT_GELU_TANH>(o); break;
      default: break;
    }
  }
  epi_add_residual<kPairs>(p, off, res, o);
  if (p.out_f32) {
    float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + off);
#pragma unroll
    for (int i = 0; i < kPairs / 2; ++i) dst[i] = make_float4(o[2 * i].x, o[2 * i].y, o[2 * i + 1].x, o[2 * i + 1].y);
  } else {
    epi_store_bf16(static_cast<__nv_bfloat16 *>(p.out) + off, o, out_v8);
  }
}

// products of 32 tile columns: acc (* before) * cf[column] (* after)
template <bool kBefore, bool kAfter>
__device__ __forceinline__ void epi_products(const float2 *acc, const float *cf, bool scaled, float before,
                                             float after, float2 (&o)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = kBefore ? __fmul2_rn(acc[i], splat(before)) : acc[i];
  if (scaled) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 s = *reinterpret_cast<const float4 *>(cf + 4 * i);
      o[2 * i] = __fmul2_rn(o[2 * i], make_float2(s.x, s.y));
      o[2 * i + 1] = __fmul2_rn(o[2 * i + 1], make_float2(s.z, s.w));
    }
  }
  if constexpr (kAfter) {
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = __fmul2_rn(o[i], splat(after));
  }
}

// A thread's 128 tile columns (column half h of the 256-column tile ct; for
// SwiGLU 64 gate columns, then the matching 64 up columns); cf: the tile's
// column scales in shared memory (scaled: there are any).
template <int kEpi, bool kBefore, bool kAfter>
__device__ __forceinline__ void epi_tile(const GemmParams &p, int g, int64_t row, int ct, int h,
                                         const float2 (&acc)[64], const float *cf, bool scaled, float before,
                                         float after, bool out_v8) {
  float2 o[16], u[16];
  if constexpr (kEpi == GMM_ACT_SWIGLU) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int in_tile = h * 64 + c * 32;
      epi_products<kBefore, kAfter>(acc + c * 16, cf + in_tile, scaled, before, after, o);
      epi_products<kBefore, kAfter>(acc + 32 + c * 16, cf + 128 + in_tile, scaled, before, after, u);
      epi_finish<kEpi>(p, g, row, true, ct * 128 + in_tile, o, u, out_v8);
    }
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int in_tile = h * 128 + c * 32, col = ct * 256 + in_tile;
      if (col >= p.ncols) continue;
      epi_products<kBefore, kAfter>(acc + c * 16, cf + in_tile, scaled, before, after, o);
      epi_finish<kEpi>(p, g, row, false, col, o, u, out_v8);
    }
  }
}

// One chunk straight from tensor memory (bf16 family: no scales); vb: the up
// columns of SwiGLU.
__device__ __forceinline__ void epi_chunk(const GemmParams &p, int g, int64_t row, bool sw, int col,
                                          const uint32_t (&va)[32], const uint32_t (&vb)[32], bool out_v8) {
  if (!sw && col >= p.ncols) return;
  float2 o[16], u[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    o[i] = make_float2(__uint_as_float(va[2 * i]), __uint_as_float(va[2 * i + 1]));
    if (sw) u[i] = make_float2(__uint_as_float(vb[2 * i]), __uint_as_float(vb[2 * i + 1]));
  }
  epi_finish<kAnyEpi>(p, g, row, sw, col, o, u, out_v8);
}

}  // namespace gmm
