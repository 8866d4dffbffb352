// Shared-prefix attention kernel instantiations for bf16 inputs.
#include "prefix_kernel.cuh"

namespace sdpa {

cudaError_t launch_prefix_bf16(int d_qk, int d_v, const CUtensorMap (&m)[6], const PrefixParams& p, cudaStream_t st) {
  if (d_qk == 64 && d_v == 64) return launch_prefix_t<64, 64, true>(m, p, st);
  if (d_qk == 128 && d_v == 128) return launch_prefix_t<128, 128, true>(m, p, st);
  if (d_qk == 192 && d_v == 128) return launch_prefix_t<192, 128, true>(m, p, st);
  return cudaErrorInvalidValue;
}

}  // namespace sdpa
