// eqlin_attn_tc_dq.cu -- dq (and delta) of the document attention; see eqlin_attn_tc_bwd.cuh.
#include "eqlin_attn_tc_bwd.cuh"

namespace eqlin {
cudaError_t launch_attn_tc_dq(const attn::Params& p, eqlin_dtype_t dt, cudaStream_t st) {
  return attn_tc::backward_pick<false>(p, dt, st);
}
}  // namespace eqlin
