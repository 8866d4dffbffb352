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

// Division of numbers below 2^31 by one that the host knows, by a multiplication
// (Granlund and Montgomery, 1994): with 2^s >= d > 2^(s - 1) and m = floor(2^32 (2^s - d) / d)
// + 1, n / d = (floor(m n / 2^32) + n) / 2^s.
struct Divider {
  uint32_t d, m, s;
};
inline Divider divider(int64_t d) {
  uint32_t s = 0;
  while ((int64_t{1} << s) < d) ++s;
  const uint64_t rest = (uint64_t{1} << s) - static_cast<uint64_t>(d);
  return Divider{static_cast<uint32_t>(d), static_cast<uint32_t>((rest << 32) / static_cast<uint64_t>(d) + 1), s};
}

// One kind of row (queries, keys or values) of a call. The `token` side is the
// projection's layout, the `head` side the attention's (its sb / st / sh are
// the strides of batch, row and head there).
struct RowKind {
  RowSet token, head;
  const void* weight;  // [d] norm weight or null: no norm
  int heads, width;    // heads; elements a row (the values' may be fewer than d)
  int rotate;          // whether the rows are rotated
  int cached;          // head-side row = kv_rows[batch] + token, or from kv_slots, instead of token
  int block0;          // first block of this kind
  uint32_t units;      // its work units, one a warp at a time
};

struct NormRopeParams {
  RowKind kind[3];
  int n_kinds;
  int64_t tokens;  // b * s
  Divider s;
  Divider n_tb;    // blocks of tokens (norm_rope_plan)
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
  // pages instead of caches: token t's row is row slot % page_size of page
  // slot / page_size (head.sb is then the stride of the pages)
  const int* kv_slots;   // [tokens] or null
  Divider page_size;
  uint32_t n_slots;      // rows of all pages
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
