// epilogue.h -- interface between api.cu and the epilogue gradient (epilogue.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace gmm {

struct ActBwdParams {
  const __nv_bfloat16 *dout;  // [M, F]
  const __nv_bfloat16 *z;     // [M, N]
  __nv_bfloat16 *dz;          // [M, N]
  float *partial;             // [tiles, N] column sums of each 128-row tile
  uint32_t *done;             // [G, column blocks] tiles summed so far (0 before the launch)
  float *dbias;               // [G, N], or NULL (partial and done are then unused)
  const int *offs, *tpre;     // group plan
  int G;
  int64_t M, N, F;            // N = F, or 2 F for SwiGLU
};

// Counters of ActBwdParams::done for N columns (the same for either F).
int64_t act_bwd_counters(int64_t N, int G);
cudaError_t launch_act_bwd(int act, const ActBwdParams &p, cudaStream_t st);

}  // namespace gmm
