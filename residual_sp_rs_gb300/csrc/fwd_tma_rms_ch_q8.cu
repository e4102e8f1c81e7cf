// TMA-fed forward instances with y in 8 bits: bf16, norm rms, column-chunk stages.
#include "fwd_tma_inst.cuh"

namespace spf {
cudaError_t launch_fwd_tma_rms_ch_q8(const FwdArgs& a, int T, const FwdTmaPlan& p, dim3 grid,
                                      cudaStream_t st) {
  return launch_fwd_tma_impl<false, true, true>(a, T, p, grid, st);
}
}  // namespace spf
