// Capped-score fused backward kernel instantiations.
#include "bwd_fused_kernel.cuh"

namespace sdpa {

cudaError_t launch_bwd_fused_cap(bool bf16, int d_qk, int d_v, const CUtensorMap& q, const CUtensorMap& k,
                                 const CUtensorMap& v, const CUtensorMap& dout, const CUtensorMap& dk,
                                 const CUtensorMap& dv, const BwdParams& p, cudaStream_t st) {
  if (bf16 && d_qk == 64 && d_v == 64) return launch_bwd_fused_cap_t<64, 64, true>(q, k, v, dout, dk, dv, p, st);
  if (!bf16 && d_qk == 64 && d_v == 64) return launch_bwd_fused_cap_t<64, 64, false>(q, k, v, dout, dk, dv, p, st);
  if (bf16 && d_qk == 128 && d_v == 128) return launch_bwd_fused_cap_t<128, 128, true>(q, k, v, dout, dk, dv, p, st);
  if (!bf16 && d_qk == 128 && d_v == 128) return launch_bwd_fused_cap_t<128, 128, false>(q, k, v, dout, dk, dv, p, st);
  return cudaErrorInvalidValue;
}

}  // namespace sdpa
