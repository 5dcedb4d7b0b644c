// epilogue.cu -- gradient of the product epilogue out = act(z) + residual,
// z = product + bias[g]:
//   dz[m, n]    = dout[m, n] * act'(z[m, n])         (SwiGLU: gate and up parts)
//   dbias[g, n] = sum over the rows m of group g of dz[m, n]
// (the residual's gradient is dout itself).  One pass: dout and z are read
// once, dz is written once, and the column sums are taken from the registers
// that hold dz before its rounding to bf16.  A CTA sums one tile of at most
// 128 rows of one group; the tiles of a group are then added in row order by
// a second small kernel (1/64 of the bytes), so the result does not depend
// on timing.  Bound by HBM.
#include <cuda_bf16.h>

#include "act.cuh"
#include "epilogue.h"
#include "internal.h"

namespace gmm {
namespace {

constexpr int kActThreads = 256;
constexpr int kActCols = 256;  // columns of a CTA: 32 threads of 8
constexpr int kActRowThreads = kActThreads / 32;
constexpr int kActUnroll = 1;

__device__ __forceinline__ float2 bf16x2_f32(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

__device__ __forceinline__ uint4 pack8(const float2 (&v)[4]) {
  uint4 u;
  __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __float22bfloat162_rn(v[i]);
  return u;
}

template <int kAct>
__global__ void __launch_bounds__(kActThreads, 4) act_bwd_kernel(const ActBwdParams p) {
  constexpr bool kGated = kAct == GMM_ACT_SWIGLU;
  constexpr int kParts = kGated ? 2 : 1;
  __shared__ float s_sum[kActRowThreads][kParts][kActCols];
  // rows of this CTA: tile `ti` of the groups, or a 128-row slice of the rows
  // behind the last group
  const int ti = blockIdx.y, ntiles = p.tpre[p.G];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * kActCols + cx * 8;
  const bool col_ok = col < p.F;
  int64_t r0, r1;
  bool tail = false;
  if (ti < ntiles) {
    int lo = 0, hi = p.G;  // group g with tpre[g] <= ti < tpre[g + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.tpre[mid] <= ti) lo = mid;
      else hi = mid;
    }
    r0 = p.offs[lo] + static_cast<int64_t>(ti - p.tpre[lo]) * kBlk;
    r1 = min(r0 + kBlk, static_cast<int64_t>(p.offs[lo + 1]));
  } else {
    tail = true;
    r0 = p.offs[p.G] + static_cast<int64_t>(ti - ntiles) * kBlk;
    r1 = min(r0 + kBlk, p.M);
  }
  if (r0 >= r1) return;
  float2 sum[kParts][4];
#pragma unroll
  for (int s = 0; s < kParts; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[s][i] = make_float2(0.0f, 0.0f);
  const __nv_bfloat16 *dout = p.dout + col, *z = p.z + col;
  __nv_bfloat16 *dz = p.dz + col;
  if (col_ok && tail) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int64_t r = r0 + ry; r < r1; r += kActRowThreads)
#pragma unroll
      for (int s = 0; s < kParts; ++s) *reinterpret_cast<uint4 *>(dz + r * p.N + s * p.F) = zero;
  } else if (col_ok) {
    for (int64_t rb = r0 + ry; rb < r1; rb += kActRowThreads * kActUnroll) {
      uint4 vd[kActUnroll], vz[kActUnroll][kParts];
#pragma unroll
      for (int u = 0; u < kActUnroll; ++u) {
        const int64_t r = rb + u * kActRowThreads;
        if (r < r1) {
          vd[u] = __ldcs(reinterpret_cast<const uint4 *>(dout + r * p.F));
#pragma unroll
          for (int s = 0; s < kParts; ++s) vz[u][s] = __ldcs(reinterpret_cast<const uint4 *>(z + r * p.N + s * p.F));
        }
      }
#pragma unroll
      for (int u = 0; u < kActUnroll; ++u) {
        const int64_t r = rb + u * kActRowThreads;
        if (r >= r1) continue;
        float2 o[kParts][4];
        const uint32_t *dw = reinterpret_cast<const uint32_t *>(&vd[u]);
        const uint32_t *aw = reinterpret_cast<const uint32_t *>(&vz[u][0]);
        const uint32_t *bw = reinterpret_cast<const uint32_t *>(&vz[u][kParts - 1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 d = bf16x2_f32(dw[i]), a = bf16x2_f32(aw[i]);
          if constexpr (kGated) {
            const float2 b = bf16x2_f32(bw[i]), s = sigmoid2(a), as = __fmul2_rn(a, s);
            // d silu = s + a s (1 - s)
            const float2 ds = __ffma2_rn(as, __ffma2_rn(s, splat(-1.0f), splat(1.0f)), s);
            o[0][i] = __fmul2_rn(__fmul2_rn(d, b), ds);
            o[kParts - 1][i] = __fmul2_rn(d, as);
          } else {
            o[0][i] = __fmul2_rn(d, slope2<kAct>(a));
          }
        }
#pragma unroll
        for (int s = 0; s < kParts; ++s) {
          __stcs(reinterpret_cast<uint4 *>(dz + r * p.N + s * p.F), pack8(o[s]));
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[s][i] = __fadd2_rn(sum[s][i], o[s][i]);
        }
      }
    }
  }
  if (!p.partial || tail) return;
#pragma unroll
  for (int s = 0; s < kParts; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<float2 *>(&s_sum[ry][s][cx * 8 + 2 * i]) = sum[s][i];
  __syncthreads();
  for (int i = threadIdx.x; i < kParts * kActCols; i += kActThreads) {
    const int s = i / kActCols, c = i % kActCols;
    const int64_t gc = static_cast<int64_t>(blockIdx.x) * kActCols + c;
    if (gc >= p.F) continue;
    float a = 0.0f;
#pragma unroll
    for (int r = 0; r < kActRowThreads; ++r) a += s_sum[r][s][c];
    p.partial[static_cast<int64_t>(ti) * p.N + s * p.F + gc] = a;
  }
}

// dbias[g, n] = the group's tile sums, in row order (0 for an empty group)
__global__ void __launch_bounds__(128) dbias_kernel(const float *__restrict__ partial, const int *__restrict__ tpre,
                                                    int64_t N, float *__restrict__ dbias) {
  const int g = blockIdx.y;
  const int64_t n = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x);
  if (n >= N) return;
  float a = 0.0f;
#pragma unroll 8
  for (int t = tpre[g]; t < tpre[g + 1]; ++t) a += partial[t * N + n];
  dbias[g * N + n] = a;
}

}  // namespace

cudaError_t launch_act_bwd(int act, const ActBwdParams &p, cudaStream_t st) {
  // every tile of a group, then the slices of the rows behind the last group:
  // n lengths of sum M have at most floor((M + 127 n) / 128) tiles of 128, which
  // for n = G + 1 <= 1025 is at most ceil(M / 128) + G (and so below 2^16)
  const dim3 grid(static_cast<unsigned>((p.F + kActCols - 1) / kActCols),
                  static_cast<unsigned>((p.M + kBlk - 1) / kBlk + p.G));
  switch (act) {
    case GMM_ACT_NONE: act_bwd_kernel<GMM_ACT_NONE><<<grid, kActThreads, 0, st>>>(p); break;
    case GMM_ACT_RELU: act_bwd_kernel<GMM_ACT_RELU><<<grid, kActThreads, 0, st>>>(p); break;
    case GMM_ACT_SILU: act_bwd_kernel<GMM_ACT_SILU><<<grid, kActThreads, 0, st>>>(p); break;
    case GMM_ACT_GELU: act_bwd_kernel<GMM_ACT_GELU><<<grid, kActThreads, 0, st>>>(p); break;
    case GMM_ACT_GELU_TANH: act_bwd_kernel<GMM_ACT_GELU_TANH><<<grid, kActThreads, 0, st>>>(p); break;
    case GMM_ACT_SWIGLU: act_bwd_kernel<GMM_ACT_SWIGLU><<<grid, kActThreads, 0, st>>>(p); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

cudaError_t launch_dbias(const float *partial, const int *tpre, int G, int64_t N, float *dbias, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((N + 127) / 128), static_cast<unsigned>(G));
  dbias_kernel<<<grid, 128, 0, st>>>(partial, tpre, N, dbias);
  return cudaGetLastError();
}

}  // namespace gmm
