// router.h -- interface between api.cu and the router kernels (router.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace gmm {

struct RouterParams {
  const void *logits;  // [T, E] f32 or bf16
  int bf16;
  const float *bias;   // [E] added to the scores for the choice only, or NULL
  int64_t T;
  int E, k;
  int sigmoid, normalize;
  float scale;
  int32_t *ids;           // [T, k]
  float *weights;         // [T, k] (forward)
  const float *dweights;  // [T, k] (backward)
  void *dlogits;          // [T, E] of the logits' type (backward)
};

cudaError_t launch_router_topk(const RouterParams &p, cudaStream_t st);
cudaError_t launch_router_topk_bwd(const RouterParams &p, cudaStream_t st);
cudaError_t launch_combine_dweight(const void *dy, const void *rows, const int32_t *slot, int64_t T, int k,
                                   int64_t nrows, int64_t N, float *dw, cudaStream_t st);

}  // namespace gmm
