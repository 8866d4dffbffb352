// Parameters and launchers of the query/key norm with the position rotation
// (norm_rope.cu), shared with the C entry points.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace sdpa {

// Rows of a [batch][token][head][width] tensor: element strides (the width's
// is 1), base pointer.
struct RowSet {
  void* ptr;
  int64_t sb, st, sh;
};

// One kind of row (queries, keys or values) of a call. The `token` side is the
// projection's layout, the `head` side the attention's (its sb / st / sh are
// the strides of batch, row and head there).
struct RowKind {
  RowSet token, head;
  const void* weight;  // [d] norm weight or null: no norm
  int heads, width;    // heads; elements a row (the values' may be fewer than d)
  int rotate;          // whether the rows are rotated
  int cached;          // head-side row = kv_rows[batch] + token instead of token
  int block0;          // first block of this kind
  uint32_t units;      // its work units, one a warp at a time
};

struct NormRopeParams {
  RowKind kind[3];
  int n_kinds;
  int64_t tokens;  // b * s
  int s;
  int d, rot, interleaved;
  int seg;         // heads a work unit walks (norm_rope_plan)
  float eps;
  int weight_fp32;       // weights are fp32 (else the io type)
  const float* cos;      // [n_pos][rot / 2]
  const float* sin;
  int64_t n_pos;
  const int* positions;  // [tokens] or null: the token's number in its sequence
  const int* kv_rows;    // [b] or null
  int64_t cache_rows;    // rows of the caches
  // backward: head = dy, token = dx, x = the forward's input; fp32 partial weight
  // gradients, one row of d per block of kinds 0 and 1
  RowSet x[3];
  float* dw_part;
};

// Blocks of the whole call (-1: too many), and each kind's share (fills block0, units, seg).
int norm_rope_plan(NormRopeParams* p, bool backward);
cudaError_t launch_norm_rope_fwd(bool bf16, const NormRopeParams& p, int blocks, cudaStream_t st);
// dw_q / dw_k: [d] in the weights' type (null where the kind has no weight)
cudaError_t launch_norm_rope_bwd(bool bf16, const NormRopeParams& p, int blocks, void* dw_q, void* dw_k,
                                 cudaStream_t st);

}  // namespace sdpa
