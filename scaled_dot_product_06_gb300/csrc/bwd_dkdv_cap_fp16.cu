// Capped-score dK/dV kernel instantiations for fp16 inputs.
#include "bwd_dkdv_kernel.cuh"

namespace sdpa {

cudaError_t launch_bwd_dkdv_cap_fp16(int d_qk, int d_v, const CUtensorMap& q, const CUtensorMap& k,
                                     const CUtensorMap& v, const CUtensorMap& dout, const CUtensorMap& dk,
                                     const CUtensorMap& dv, const BwdParams& p, cudaStream_t st) {
  if (d_qk == 64 && d_v == 64) return launch_bwd_dkdv_cap_t<64, 64, false>(q, k, v, dout, dk, dv, p, st);
  if (d_qk == 128 && d_v == 128) return launch_bwd_dkdv_cap_t<128, 128, false>(q, k, v, dout, dk, dv, p, st);
  if (d_qk == 192 && d_v == 128) return launch_bwd_dkdv_cap_t<192, 128, false>(q, k, v, dout, dk, dv, p, st);
  return cudaErrorInvalidValue;
}

}  // namespace sdpa
