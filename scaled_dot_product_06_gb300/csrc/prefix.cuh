// Parameters and launchers of the shared-prefix attention (prefix_kernel.cuh,
// prefix_join.cu).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace sdpa {

struct PrefixParams {
  int B, H_kv, R, s_q;         // R = (h / h_kv) * s_q rows a sequence and K/V head
  int s_prefix, s_max;
  const int* seqlen;           // [B] own keys, the new tokens' among them
  float scale_log2;            // factor of the raw score in the exponent
  float cap_in, lse_shift;     // capped scores: see cap_r8; lse_shift = softcap log2(e)
  // work items: the prefix's first, then the own keys'
  int items_prefix, items_own;
  int row_tiles_p, row_blocks_p, splits_p, chunk_p, dual_p;
  int row_tiles_o, row_blocks_o, splits_o, chunk_o, dual_o;
  int seqs_tile;               // sequences a row tile of the prefix holds (R <= 128)
  uint32_t q_box_p, q_box_o;   // bytes of Q's boxes
  int slots_p, slots_o;        // partial slots of the two key sets
  int64_t rows;                // B * H_kv * R
  float* part;                 // [slots][rows][d_v]
  float* part_lse;             // [slots][rows]
  void* o;
  float* lse;
  uint32_t* err;
};

cudaError_t launch_prefix_bf16(int d_qk, int d_v, const CUtensorMap (&m)[6], const PrefixParams& p, cudaStream_t st);
cudaError_t launch_prefix_fp16(int d_qk, int d_v, const CUtensorMap (&m)[6], const PrefixParams& p, cudaStream_t st);
cudaError_t launch_prefix_join(bool bf16, int d_v, const PrefixParams& p, cudaStream_t st);

}  // namespace sdpa
