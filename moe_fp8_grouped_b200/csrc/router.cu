// router.cu -- the router of a mixture-of-experts layer and its gradient:
//
//   p = softmax(x) or sigmoid(x);  k experts of largest key (p + bias, or x);
//   w_j = scale * p_j, or scale * p_j / sum of the chosen p
//
// and, for the backward, the gradient of the combine's weights,
//   dw[t, j] = sum_n dy[t, n] * rows[slot[t, j], n],
// which then flows through the formulas above to the logits.
//
// The choice reads T x E logits once and keeps a token's row in one warp's
// registers (E / 32 values a lane): k rounds of a warp maximum pick the
// experts, ties going to the lowest index.  Without a bias the logits
// themselves are compared (both scores are increasing in them), so the choice
// is exact.  With a bias the keys are scores that fp32 rounds: when two of
// the k + 1 largest lie closer than that rounding, the token's keys are
// worked out again in fp64 and the choice is made by those.
#include <cuda_bf16.h>
#include <cfloat>
#include <cmath>

#include "act.cuh"
#include "internal.h"
#include "router.h"

namespace gmm {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kRouterWarps = 4;  // tokens of a CTA

__device__ __forceinline__ float load_logit(const void *x, int64_t i, bool bf16) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(x)[i]) : static_cast<const float *>(x)[i];
}

// Unsigned order of a key: larger key, larger number; NaN above everything
// (it wins, so that it shows in the weights), -inf is 0 (never chosen).
__device__ __forceinline__ uint32_t order32(float v) {
  if (isnan(v)) return 0xffffffffu;
  if (v == -INFINITY) return 0u;
  const uint32_t u = __float_as_uint(v + 0.0f);  // -0 counts as 0
  return (u >> 31) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ unsigned long long order64(double v) {
  if (isnan(v)) return ~0ull;
  if (v == -INFINITY) return 0ull;
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(v + 0.0));
  return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}

__device__ __forceinline__ float key_of_order32(uint32_t o) {
  return __uint_as_float((o >> 31) ? o & 0x7fffffffu : ~o);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, d));
  return v;
}

// exp(x): |x| 2^-23 relative from the product, 2 ulp from the unit
__device__ __forceinline__ float fast_exp(float x) { return fast_exp2(x * kLog2e); }

// log(sigmoid(x)) without overflow
__device__ __forceinline__ float log_sigmoid(float x) { return fminf(x, 0.0f) - log1pf(fast_exp(-fabsf(x))); }

__device__ __forceinline__ float sigmoid(float x) { return fast_rcp(1.0f + fast_exp(-x)); }

// One round of the choice: the lane's largest order with its lowest index,
// then the warp's; the winner is removed.  Returns its index, -1 when nothing
// is left, its order in `best` and its logit in `logit`.
template <int kV, class T>
__device__ __forceinline__ int take_largest(T (&ord)[kV], const float (&x)[kV], int lane, T &best, float &logit) {
  T m = ord[0];
  int v = 0;
  float xv = x[0];
#pragma unroll
  for (int i = 1; i < kV; ++i)
    if (ord[i] > m) {
      m = ord[i];
      v = i;
      xv = x[i];
    }
  if constexpr (sizeof(T) == 4) {
    best = __reduce_max_sync(kFull, m);
  } else {
    best = m;
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      const T o = __shfl_xor_sync(kFull, best, d);
      best = o > best ? o : best;
    }
  }
  if (best == 0) return -1;
  const int e = __reduce_min_sync(kFull, m == best ? v * 32 + lane : 0x7fffffff);
  logit = __shfl_sync(kFull, xv, e & 31);
#pragma unroll
  for (int i = 0; i < kV; ++i)
    if (i * 32 + lane == e) ord[i] = 0;
  return e;
}

// Weights of the chosen experts: lane j < k holds logit xs of choice j
// (valid: an expert was chosen).
__device__ __forceinline__ float chosen_weight(float xs, bool valid, float mx, float sum, bool sig, bool norm,
                                               float scale) {
  if (norm) {
    // p_j / sum p: a softmax of the chosen log scores (the full softmax's
    // denominator cancels), safe where every p underflows
    const float l = sig ? log_sigmoid(xs) : xs;
    const float m = warp_max(valid ? l : -INFINITY);
    const bool nan = __any_sync(kFull, valid && (isnan(l) || l == INFINITY));
    const float e = valid ? fast_exp(l - m) : 0.0f;
    const float s = warp_sum(e);
    return nan ? __int_as_float(0x7fffffff) : scale * (e / s);
  }
  return sig ? scale * sigmoid(xs) : scale * (fast_exp(xs - mx) / sum);
}

template <int kV>
__global__ void __launch_bounds__(kRouterWarps * 32) router_topk_kernel(const RouterParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouterWarps + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const int E = p.E, k = p.k;
  float x[kV], b[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int e = i * 32 + lane;
    x[i] = e < E ? load_logit(p.logits, t * E + e, p.bf16) : -INFINITY;
    b[i] = p.bias && e < E ? p.bias[e] : 0.0f;
  }
  // softmax statistics of the row (not needed for sigmoid, nor when the
  // chosen weights are normalised and no bias is added to the scores)
  float mx = 0.0f, sum = 1.0f;
  const bool sig = p.sigmoid;
  if (!sig && (!p.normalize || p.bias)) {
    float m = x[0];
#pragma unroll
    for (int i = 1; i < kV; ++i) m = fmaxf(m, x[i]);
    mx = warp_max(m);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kV; ++i) s += x[i] == -INFINITY ? 0.0f : fast_exp(x[i] - mx);
    sum = warp_sum(s);
  }
  const float inv_sum = 1.0f / sum;
  uint32_t ord[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    float key = x[i];
    if (p.bias && x[i] != -INFINITY) key = (sig ? sigmoid(x[i]) : fast_exp(x[i] - mx) * inv_sum) + b[i];
    ord[i] = order32(key);
  }
  int mine = -1;  // lane j: expert of choice j, and its logit
  float xs = 0.0f;
  bool near = false;
  uint32_t prev = 0;
  // A key is within `off` + 2^-24 |key| of the true one: a sigmoid's error is
  // s (1 - s) (|x| + 4) 2^-23 from the exponential, below 2e-7, and 1.5 ulp; a
  // softmax score's, relative, (|x - m| + 8) 2^-23 and the sum's E / 32 + 5
  // roundings, below 3e-6 of a score where that score is near the largest and
  // absolutely below 3e-6 everywhere
  const float off = sig ? 8e-7f : 6e-6f;  // of two keys
  for (int j = 0; j < k + (p.bias ? 1 : 0); ++j) {
    uint32_t o;
    float xv;
    const int e = take_largest(ord, x, lane, o, xv);
    if (e < 0) break;
    if (p.bias && j > 0) {
      const float a = key_of_order32(prev), c = key_of_order32(o);
      near |= !(a - c > off + 2e-7f * (fabsf(a) + fabsf(c)));
    }
    prev = o;
    if (lane == j && j < k) {
      mine = e;
      xs = xv;
    }
  }
  if (near) {
    double s64 = 1.0, m64 = mx;
    if (!sig) {
      double s = 0.0;
#pragma unroll
      for (int i = 0; i < kV; ++i) s += x[i] == -INFINITY ? 0.0 : exp(static_cast<double>(x[i]) - m64);
#pragma unroll
      for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
      s64 = s;
    }
    unsigned long long o64[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int e = i * 32 + lane;
      double key = x[i];
      if (e < E && x[i] != -INFINITY)
        key = (sig ? 1.0 / (1.0 + exp(-key)) : exp(key - m64) / s64) + static_cast<double>(b[i]);
      o64[i] = order64(key);
    }
    mine = -1;
    for (int j = 0; j < k; ++j) {
      unsigned long long o;
      float xv;
      const int e = take_largest(o64, x, lane, o, xv);
      if (e < 0) break;
      if (lane == j) {
        mine = e;
        xs = xv;
      }
    }
  }
  const bool valid = lane < k && mine >= 0;
  const float w = chosen_weight(xs, valid, mx, sum, sig, p.normalize, p.scale);
  if (lane < k) {
    p.ids[t * k + lane] = mine;
    p.weights[t * k + lane] = valid ? w : 0.0f;
  }
}

// dlogits of one token per warp, put together in shared memory: the softmax's
// common term first, then the chosen experts' terms in the order of choice
// (an expert named twice gets both).
__global__ void __launch_bounds__(kRouterWarps * 32) router_topk_bwd_kernel(const RouterParams p) {
  extern __shared__ float s_rows[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouterWarps + warp;
  if (t >= p.T) return;
  const int E = p.E, k = p.k;
  float *row = s_rows + warp * E;
  const bool sig = p.sigmoid;
  const int id = lane < k ? p.ids[t * k + lane] : -1;
  bool valid = id >= 0 && id < E;
  const float xs = valid ? load_logit(p.logits, t * E + id, p.bf16) : 0.0f;
  valid = valid && xs != -INFINITY;  // a masked expert has score 0 and no slope
  const float dw = valid ? p.dweights[t * k + lane] : 0.0f;
  float c;  // what choice j adds to its logit's gradient
  if (p.normalize) {
    const float l = sig ? log_sigmoid(xs) : xs;
    const float m = warp_max(valid ? l : -INFINITY);
    const float e = valid ? fast_exp(l - m) : 0.0f;
    const float w = e / warp_sum(e);
    const float dot = warp_sum(valid ? w * dw : 0.0f);
    c = w * (dw - dot);
    if (sig) c *= sigmoid(-xs);  // d log sigmoid = 1 - sigmoid
    for (int e2 = lane; e2 < E; e2 += 32) row[e2] = 0.0f;
  } else if (sig) {
    c = dw * sigmoid(xs) * sigmoid(-xs);
    for (int e2 = lane; e2 < E; e2 += 32) row[e2] = 0.0f;
  } else {
    float m = -INFINITY;
    for (int e2 = lane; e2 < E; e2 += 32) {
      const float v = load_logit(p.logits, t * E + e2, p.bf16);
      row[e2] = v;
      m = fmaxf(m, v);
    }
    m = warp_max(m);
    float s = 0.0f;
    for (int e2 = lane; e2 < E; e2 += 32) {
      const float e = row[e2] == -INFINITY ? 0.0f : fast_exp(row[e2] - m);
      row[e2] = e;
      s += e;
    }
    s = warp_sum(s);
    const float pr = valid ? fast_exp(xs - m) / s : 0.0f;
    c = pr * dw;
    const float dot = warp_sum(valid ? c : 0.0f);
    const float f = s == 0.0f ? 0.0f : dot / s;  // s = 0: every expert is masked; a NaN in the row stays
    for (int e2 = lane; e2 < E; e2 += 32) row[e2] = -row[e2] * f;
  }
  __syncwarp();
  for (int j = 0; j < k; ++j) {
    if (lane == j && valid) row[id] += c;
    __syncwarp();
  }
  for (int e2 = lane; e2 < E; e2 += 32) {
    const float v = row[e2] * p.scale;
    if (p.bf16) static_cast<__nv_bfloat16 *>(p.dlogits)[t * E + e2] = __float2bfloat16_rn(v);
    else static_cast<float *>(p.dlogits)[t * E + e2] = v;
  }
}

// dw[t, j] for kJ choices at a time: one CTA per token, 8 columns per thread
// step, so that kJ + 1 16-byte loads are in flight per thread.  Sums in fp32,
// in an order fixed by the sizes.
template <int kJ>
__global__ void __launch_bounds__(128) combine_dweight_kernel(const uint4 *__restrict__ dy,
                                                              const uint4 *__restrict__ rows,
                                                              const int32_t *__restrict__ slot, int k, int64_t nrows,
                                                              int64_t n8, float *__restrict__ dw) {
  __shared__ float s_part[4][kJ];
  const int64_t t = blockIdx.x;
  for (int j0 = 0; j0 < k; j0 += kJ) {
    const uint4 *src[kJ];
    bool ok[kJ];
    float acc[kJ];
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const int64_t r = j0 + j < k ? slot[t * k + j0 + j] : -1;
      ok[j] = r >= 0 && r < nrows;
      src[j] = rows + (ok[j] ? r : 0) * n8;
      acc[j] = 0.0f;
    }
    for (int64_t c = threadIdx.x; c < n8; c += 128) {
      const uint4 d = dy[t * n8 + c];
      uint4 v[kJ];
#pragma unroll
      for (int j = 0; j < kJ; ++j)
        if (ok[j]) v[j] = __ldcs(src[j] + c);
      const __nv_bfloat162 *dh = reinterpret_cast<const __nv_bfloat162 *>(&d);
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        if (!ok[j]) continue;
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&v[j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 a = __bfloat1622float2(dh[e]), b = __bfloat1622float2(h[e]);
          acc[j] = fmaf(a.x, b.x, acc[j]);
          acc[j] = fmaf(a.y, b.y, acc[j]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kJ; ++j) acc[j] = warp_sum(acc[j]);
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int j = 0; j < kJ; ++j) s_part[threadIdx.x >> 5][j] = acc[j];
    __syncthreads();
    const int j = threadIdx.x;
    if (j < kJ && j0 + j < k) dw[t * k + j0 + j] = (s_part[0][j] + s_part[1][j]) + (s_part[2][j] + s_part[3][j]);
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_router_topk(const RouterParams &p, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>((p.T + kRouterWarps - 1) / kRouterWarps);
  const int nt = kRouterWarps * 32;
  if (p.E <= 32) router_topk_kernel<1><<<grid, nt, 0, st>>>(p);
  else if (p.E <= 64) router_topk_kernel<2><<<grid, nt, 0, st>>>(p);
  else if (p.E <= 128) router_topk_kernel<4><<<grid, nt, 0, st>>>(p);
  else if (p.E <= 256) router_topk_kernel<8><<<grid, nt, 0, st>>>(p);
  else if (p.E <= 512) router_topk_kernel<16><<<grid, nt, 0, st>>>(p);
  else router_topk_kernel<32><<<grid, nt, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_router_topk_bwd(const RouterParams &p, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>((p.T + kRouterWarps - 1) / kRouterWarps);
  router_topk_bwd_kernel<<<grid, kRouterWarps * 32, kRouterWarps * p.E * sizeof(float), st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_combine_dweight(const void *dy, const void *rows, const int32_t *slot, int64_t T, int k,
                                   int64_t nrows, int64_t N, float *dw, cudaStream_t st) {
  const uint4 *d = static_cast<const uint4 *>(dy), *r = static_cast<const uint4 *>(rows);
  const unsigned grid = static_cast<unsigned>(T);
  if (k <= 1) combine_dweight_kernel<1><<<grid, 128, 0, st>>>(d, r, slot, k, nrows, N / 8, dw);
  else if (k <= 2) combine_dweight_kernel<2><<<grid, 128, 0, st>>>(d, r, slot, k, nrows, N / 8, dw);
  else if (k <= 4) combine_dweight_kernel<4><<<grid, 128, 0, st>>>(d, r, slot, k, nrows, N / 8, dw);
  else combine_dweight_kernel<8><<<grid, 128, 0, st>>>(d, r, slot, k, nrows, N / 8, dw);
  return cudaGetLastError();
}

}  // namespace gmm
