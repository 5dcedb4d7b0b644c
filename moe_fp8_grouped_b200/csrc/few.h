// few.h -- interface between api.cu and the few-token layer kernel (few.cu).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace gmm {

constexpr int kFewMaxPairs = 1024;  // tokens x choices of one call

struct FewParams {
  const __nv_bfloat16 *x;  // [T, K]
  const int32_t *ids;      // [T, k]
  const float *weights;    // [T, k]
  const float *s1, *s2;    // [G, 2F], [G, N] (E4M3 weights)
  __nv_bfloat16 *h;        // [pairs, F] silu(gate) * up
  uint32_t *largest;       // [T] and [pairs]: largest magnitudes of the rows of x and h (bf16 bits)
  float *partial;          // [pairs][columns] sums of a product (its tiles' first slice)
  float *extra;            // few_extra_floats: the other slices of tiles left over
  void *y;                 // [T, N]
  int T, k, pairs, G, F, N;
  int tiles1, kb1, tiles2, kb2;  // 128-column tiles and contraction blocks of the two products
  int y_f32;
  uint32_t *status;
  uint64_t wait_limit_ns;
};

// Floats of FewParams::extra.
size_t few_extra_floats();

cudaError_t launch_moe_few(int elem, bool mn_major, const CUtensorMap &tm1, const CUtensorMap &tm2,
                           const FewParams &p, cudaStream_t st);

}  // namespace gmm
