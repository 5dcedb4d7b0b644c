// epilogue.cu -- gradient of the product epilogue out = act(z) + residual,
// z = product + bias[g]:
//   dz[m, n]    = dout[m, n] * act'(z[m, n])         (SwiGLU: gate and up parts)
//   dbias[g, n] = sum over the rows m of group g of dz[m, n]
// (the residual's gradient is dout itself).  One pass: dout and z are read
// once, dz is written once, and the column sums are taken from the registers
// that hold dz before its rounding to bf16.  A CTA sums one tile of at most
// 128 rows of one group.  Whichever of a group's CTAs finishes last adds the
// tiles (1/64 of the bytes, from L2), in an order that depends on their number
// only; a group of one tile needs none of that.  Bound by HBM.
#include <cuda_bf16.h>

#include "act.cuh"
#include "epilogue.h"
#include "internal.h"

namespace gmm {
namespace {

constexpr int kActThreads = 256;
// columns of a CTA: 32 threads of 8 (Mixtral-like SwiGLU, 16384 x 28672, and
// GELU of 256 groups in 8195 rows of 2048 columns, us: 128 columns 396 / 25.7,
// 256 387 / 20.2, 512 391 / 23.1, 1024 405 / 26.3)
constexpr int kActCols = 256;
constexpr int kActRowThreads = kActThreads / 32;
constexpr int kActUnroll = 1;  // rows of a thread step (2: 442 / 21.8)

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
  __shared__ __align__(16) float s_sum[kActRowThreads][kParts][kActCols];
  __shared__ bool s_last;
  // rows of this CTA: tile `ti` of the groups, or a 128-row slice of the rows
  // behind the last group
  cudaGridDependencySynchronize();  // the launch may overlap the plan's; all reads come after it
  const int ti = blockIdx.y, ntiles = p.tpre[p.G];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * kActCols + cx * 8;
  const bool col_ok = col < p.F;
  int64_t r0, r1;
  bool tail = false;
  // group lo with tpre[lo] <= ti < tpre[lo + 1], by counting: one round of
  // loads (a binary search's eight dependent ones took as long as a tile of 40
  // rows)
  int lo = 0;
  for (int g = 0; g < p.G; g += kActThreads)
    lo += __syncthreads_count(g + static_cast<int>(threadIdx.x) < p.G && p.tpre[g + threadIdx.x + 1] <= ti);
  if (ti < ntiles) {
    r0 = p.offs[lo] + static_cast<int64_t>(ti - p.tpre[lo]) * kBlk;
    r1 = min(r0 + kBlk, static_cast<int64_t>(p.offs[lo + 1]));
  } else {
    tail = true;
    r0 = p.offs[p.G] + static_cast<int64_t>(ti - ntiles) * kBlk;
    r1 = min(r0 + kBlk, p.M);
  }
  if (r0 >= r1) {
    // CTAs without rows (there are at least as many as empty groups, see the
    // grid): the empty groups' sums
    if (!p.dbias) return;
    const int first = ntiles + static_cast<int>((p.M - p.offs[p.G] + kBlk - 1) / kBlk);
    for (int g = ti - first; g < p.G; g += gridDim.y - first) {
      if (p.offs[g] != p.offs[g + 1]) continue;
      for (int i = threadIdx.x; i < kParts * kActCols; i += kActThreads) {
        const int64_t gc = static_cast<int64_t>(blockIdx.x) * kActCols + i % kActCols;
        if (gc < p.F) p.dbias[g * p.N + i / kActCols * p.F + gc] = 0.0f;
      }
    }
    return;
  }
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
          } else if constexpr (kAct == GMM_ACT_RELU) {
            // a choice, not a product: an infinite or NaN d times 0 is NaN
            o[0][i] = make_float2(a.x > 0.0f ? d.x : 0.0f, a.y > 0.0f ? d.y : 0.0f);
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
  if (!p.dbias || tail) return;
  const int t0 = p.tpre[lo], nt = p.tpre[lo + 1] - t0;
  float *dst = nt == 1 ? p.dbias + lo * p.N : p.partial + ti * p.N;
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
    dst[s * p.F + gc] = a;
  }
  if (nt == 1) return;
  // the last of the group's CTAs in this column block adds its tiles: row
  // thread ry the tiles ry, ry + 8, .., then the eight sums in order
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0)
    s_last = atomicAdd(p.done + static_cast<int64_t>(lo) * gridDim.x + blockIdx.x, 1u) == static_cast<uint32_t>(nt - 1);
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  if (col_ok) {
#pragma unroll
    for (int s = 0; s < kParts; ++s) {
      float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b = a;
      const float4 *src = reinterpret_cast<const float4 *>(p.partial + static_cast<int64_t>(t0 + ry) * p.N + s * p.F + col);
#pragma unroll 4
      for (int t = ry; t < nt; t += kActRowThreads, src += kActRowThreads * p.N / 4) {
        const float4 u = __ldcg(src), v = __ldcg(src + 1);
        a = make_float4(a.x + u.x, a.y + u.y, a.z + u.z, a.w + u.w);
        b = make_float4(b.x + v.x, b.y + v.y, b.z + v.z, b.w + v.w);
      }
      *reinterpret_cast<float4 *>(&s_sum[ry][s][cx * 8]) = a;
      *reinterpret_cast<float4 *>(&s_sum[ry][s][cx * 8 + 4]) = b;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kParts * kActCols; i += kActThreads) {
    const int s = i / kActCols, c = i % kActCols;
    const int64_t gc = static_cast<int64_t>(blockIdx.x) * kActCols + c;
    if (gc >= p.F) continue;
    float a = 0.0f;
#pragma unroll
    for (int r = 0; r < kActRowThreads; ++r) a += s_sum[r][s][c];
    p.dbias[lo * p.N + s * p.F + gc] = a;
  }
}

}  // namespace

int64_t act_bwd_counters(int64_t N, int G) { return (N + kActCols - 1) / kActCols * G; }

cudaError_t launch_act_bwd(int act, const ActBwdParams &p, cudaStream_t st) {
  // every tile of a group, then the slices of the rows behind the last group:
  // n lengths of sum M have at most floor((M + 127 n) / 128) tiles of 128, which
  // for n = G + 1 <= 1025 is at most ceil(M / 128) + G (and so below 2^16); an
  // empty group lowers n, and so leaves one CTA of each column block without rows
  const dim3 grid(static_cast<unsigned>((p.F + kActCols - 1) / kActCols),
                  static_cast<unsigned>((p.M + kBlk - 1) / kBlk + p.G));
  cudaLaunchAttribute overlap;  // CTAs start while the plan's kernel ends
  overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  overlap.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kActThreads);
  cfg.stream = st;
  cfg.attrs = &overlap;
  cfg.numAttrs = 1;
  cudaError_t e = cudaErrorInvalidValue;
  switch (act) {
    case GMM_ACT_NONE: e = cudaLaunchKernelEx(&cfg, act_bwd_kernel<GMM_ACT_NONE>, p); break;
    case GMM_ACT_RELU: e = cudaLaunchKernelEx(&cfg, act_bwd_kernel<GMM_ACT_RELU>, p); break;
    case GMM_ACT_SILU: e = cudaLaunchKernelEx(&cfg, act_bwd_kernel<GMM_ACT_SILU>, p); break;
    case GMM_ACT_GELU: e = cudaLaunchKernelEx(&cfg, act_bwd_kernel<GMM_ACT_GELU>, p); break;
    case GMM_ACT_GELU_TANH: e = cudaLaunchKernelEx(&cfg, act_bwd_kernel<GMM_ACT_GELU_TANH>, p); break;
    case GMM_ACT_SWIGLU: e = cudaLaunchKernelEx(&cfg, act_bwd_kernel<GMM_ACT_SWIGLU>, p); break;
  }
  if (e != cudaSuccess) cudaGetLastError();  // reported by the return value
  return e;
}


}  // namespace gmm
