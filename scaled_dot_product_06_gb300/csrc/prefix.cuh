// Parameters and launchers of the shared-prefix attention (prefix_kernel.cuh,
// prefix_join.cu).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace sdpa {

constexpr int kPrefixDualMax = 128;  // widest d_qk with row blocks of two tiles

struct PrefixParams {
  int B, H_kv, R, s_q;         // R = (h / h_kv) * s_q rows a sequence and K/V head
  int s_prefix, s_max;
  const int* seqlen;           // [B] own keys, the new tokens' among them
  float scale_log2;            // factor of the raw score in the exponent
  float cap_in, lse_shift;     // capped scores: see cap_r8; lse_shift = softcap log2(e)
  // work items: the prefix's first, then the own keys'
  int items_prefix, items_own;
  int grid;                    // CTAs
  int* next;                   // items taken beyond the first of each CTA (null: there are none)
  int row_tiles_p, row_blocks_p, splits_p, chunk_p, dual_p;
  int row_tiles_o, row_blocks_o, splits_o, chunk_o, dual_o, quart_o;
  int seqs_tile;               // sequences a row tile of the prefix holds (R <= 128)
  uint32_t q_box_p, q_box_o;   // bytes of Q's boxes
  int slots_p, slots_o;        // partial slots of the two key sets
  int64_t rows;                // B * H_kv * R
  float* part;                 // see prefix_part_index
  float* part_lse;             // [slots][rows]
  void* o;
  float* lse;
  uint32_t* err;
};

// Where slot `slot` of partial row `row` starts, in float4: rows in slabs of 8,
// their columns in groups of 4 side by side (group c at 8 c): threads of
// neighbouring rows write whole lines, and so does the join read them.
__host__ __device__ inline int64_t prefix_part_index(int64_t slot, int64_t rows, int64_t row, int d_v) {
  return (slot * ((rows + 7) / 8) + row / 8) * (d_v * 2) + row % 8;
}

cudaError_t launch_prefix_bf16(int d_qk, int d_v, const CUtensorMap (&m)[6], const PrefixParams& p, cudaStream_t st);
cudaError_t launch_prefix_fp16(int d_qk, int d_v, const CUtensorMap (&m)[6], const PrefixParams& p, cudaStream_t st);
cudaError_t launch_prefix_zero(const PrefixParams& p, cudaStream_t st);  // *p.next = 0
cudaError_t launch_prefix_join(bool bf16, int d_v, const PrefixParams& p, cudaStream_t st);

}  // namespace sdpa
