// Paged attention kernel instantiations for fp16 inputs.
#include "paged_kernel.cuh"

namespace sdpa {

cudaError_t launch_paged_fp16(int d_qk, int d_v, const CUtensorMap (&m)[3], const PagedParams& p, cudaStream_t st) {
  if (d_qk == 64 && d_v == 64) return launch_paged_d<64, 64, false>(m, p, st);
  if (d_qk == 128 && d_v == 128) return launch_paged_d<128, 128, false>(m, p, st);
  if (d_qk == 192 && d_v == 128) return launch_paged_d<192, 128, false>(m, p, st);
  return cudaErrorInvalidValue;
}

}  // namespace sdpa
