// gemm_act_none.cu -- the E4M3 row passes of gmm_fwd_act with this activation in
// their epilogue (instantiations of gemm_tc.cu and gemm_pair.cu; one file per
// activation so that they compile side by side).
#define GMM_EPI_ACT 0  // GMM_ACT_NONE
#include "gemm_tc.cu"
#include "gemm_pair.cu"

namespace gmm {

template <>
cudaError_t launch_gemm_act_of<GMM_EPI_ACT>(const GemmConfig &cfg, const CUtensorMap &tmA, const CUtensorMap &tmB,
                                            const CUtensorMap &tmOut, const GemmParams &p, int grid,
                                            cudaStream_t st) {
  if (cfg.cta_pairs) return pair::launch_static_act<GMM_EPI_ACT>(cfg, tmA, tmB, tmOut, p, grid, st);
  return launch_rows_e4m3<GMM_EPI_ACT>(cfg, tmA, tmB, tmOut, p, grid, st);
}

}  // namespace gmm
