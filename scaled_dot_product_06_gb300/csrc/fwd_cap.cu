// Capped-score forward kernel instantiations.
#include "fwd_kernel.cuh"

namespace sdpa {

cudaError_t launch_fwd_cap(bool bf16, int d_qk, int d_v, const CUtensorMap& q, const CUtensorMap& k,
                           const CUtensorMap& v, const FwdParams& p, cudaStream_t st) {
  if (bf16 && d_qk == 64 && d_v == 64) return launch_fwd_cap_t<64, 64, true>(q, k, v, p, st);
  if (!bf16 && d_qk == 64 && d_v == 64) return launch_fwd_cap_t<64, 64, false>(q, k, v, p, st);
  if (bf16 && d_qk == 128 && d_v == 128) return launch_fwd_cap_t<128, 128, true>(q, k, v, p, st);
  if (!bf16 && d_qk == 128 && d_v == 128) return launch_fwd_cap_t<128, 128, false>(q, k, v, p, st);
  if (bf16 && d_qk == 192 && d_v == 128) return launch_fwd_cap_t<192, 128, true>(q, k, v, p, st);
  if (!bf16 && d_qk == 192 && d_v == 128) return launch_fwd_cap_t<192, 128, false>(q, k, v, p, st);
  return cudaErrorInvalidValue;
}

}  // namespace sdpa
