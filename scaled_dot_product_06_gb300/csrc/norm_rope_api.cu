// C entry points of the query/key norm with the position rotation: argument
// checks and launch parameters.
#include <cmath>
#include <cstdio>

#include "../../include/sdpa.h"
#include "common.cuh"
#include "norm_rope.cuh"

namespace {

using namespace sdpa;

sdpa_status_t fail(sdpa_status_t s, const char* what) {
  set_last_error(what);
  return s;
}

// Rows moved 16 bytes at a time: the base and, where a dimension has more than
// one element, its stride are multiples of 16 bytes.
sdpa_status_t check_rows(const sdpa_rows_t* r, int64_t n_batch, int64_t n_row, int64_t n_head, const char* what) {
  char msg[96];
  if (r == nullptr || r->ptr == nullptr) {
    snprintf(msg, sizeof(msg), "%s is null", what);
    return fail(SDPA_ERR_INVALID_ARG, msg);
  }
  const bool odd = (n_batch > 1 && (r->batch_stride & 7) != 0) || (n_row > 1 && (r->row_stride & 7) != 0) ||
                   (n_head > 1 && (r->head_stride & 7) != 0);
  if ((reinterpret_cast<uintptr_t>(r->ptr) & 15u) != 0 || odd) {
    snprintf(msg, sizeof(msg), "%s: base and strides must be multiples of 16 bytes", what);
    return fail(SDPA_ERR_MISALIGNED, msg);
  }
  return SDPA_OK;
}

RowSet row_set(const sdpa_rows_t* r, int64_t n_batch, int64_t n_row, int64_t n_head) {
  return RowSet{r->ptr, n_batch > 1 ? r->batch_stride : 0, n_row > 1 ? r->row_stride : 0,
                n_head > 1 ? r->head_stride : 0};
}

constexpr int64_t kMaxTokens = (int64_t{1} << 30);

// Checks shared by both directions that need no row pointer; *empty: no tokens.
sdpa_status_t check_common(int64_t b, int64_t s, int64_t h, int64_t h_kv, int64_t d, int64_t d_v, int dtype,
                           int64_t rot, const float* cos, const float* sin, int64_t n_pos, const int32_t* positions,
                           const void* q_weight, const void* k_weight, float eps, bool* empty) {
  if (b < 0 || s < 0 || h < 1 || h_kv < 1) return fail(SDPA_ERR_INVALID_ARG, "sizes");
  if (dtype != SDPA_BF16 && dtype != SDPA_FP16) return fail(SDPA_ERR_UNSUPPORTED, "dtype");
  if ((d != 64 && d != 128 && d != 192) || (d_v != 64 && d_v != 128 && d_v != 192) || d_v > d)
    return fail(SDPA_ERR_UNSUPPORTED, "head sizes must be 64, 128 or 192, d_v at most d");
  if (h > (int64_t{1} << 20) || h_kv > (int64_t{1} << 20) || s > kMaxTokens || b > kMaxTokens ||
      b * s > kMaxTokens)
    return fail(SDPA_ERR_UNSUPPORTED, "too many tokens or heads");
  if (rot < 0 || rot > d || rot % 16 != 0)
    return fail(SDPA_ERR_UNSUPPORTED, "the rotated width must be a multiple of 16, at most d");
  if (!(eps > 0.f) || !std::isfinite(eps)) return fail(SDPA_ERR_INVALID_ARG, "eps must be positive and finite");
  *empty = b == 0 || s == 0;
  if (*empty) return SDPA_OK;
  if (rot > 0) {
    if (cos == nullptr || sin == nullptr || n_pos < 1) return fail(SDPA_ERR_INVALID_ARG, "cos, sin");
    if (((reinterpret_cast<uintptr_t>(cos) | reinterpret_cast<uintptr_t>(sin)) & 15u) != 0)
      return fail(SDPA_ERR_MISALIGNED, "cos, sin");
    if (positions == nullptr && n_pos < s) return fail(SDPA_ERR_INVALID_ARG, "fewer angles than tokens");
  }
  if ((reinterpret_cast<uintptr_t>(positions) & 3u) != 0) return fail(SDPA_ERR_MISALIGNED, "positions");
  if (((reinterpret_cast<uintptr_t>(q_weight) | reinterpret_cast<uintptr_t>(k_weight)) & 15u) != 0)
    return fail(SDPA_ERR_MISALIGNED, "weights");
  return SDPA_OK;
}

void fill_common(NormRopeParams* p, int64_t b, int64_t s, int64_t d, int64_t rot, int interleaved,
                 const float* cos, const float* sin, int64_t n_pos, const int32_t* positions, int weight_fp32,
                 float eps) {
  p->tokens = b * s;
  p->s = static_cast<int>(s);
  p->d = static_cast<int>(d);
  p->rot = static_cast<int>(rot);
  p->interleaved = interleaved ? 1 : 0;
  p->eps = eps;
  p->weight_fp32 = weight_fp32 ? 1 : 0;
  p->cos = cos;
  p->sin = sin;
  p->n_pos = n_pos;
  p->positions = positions;
}

}  // namespace

extern "C" {

sdpa_status_t sdpa_qk_norm_rope(int64_t b, int64_t s, int64_t h, int64_t h_kv, int64_t d, int64_t d_v,
                                sdpa_dtype_t dtype, const sdpa_rows_t* q, const sdpa_rows_t* k,
                                const sdpa_rows_t* v, const sdpa_rows_t* q_out, const sdpa_rows_t* k_out,
                                const sdpa_rows_t* v_out, int64_t rot, int interleaved, const float* cos,
                                const float* sin, int64_t n_pos, const int32_t* positions, const void* q_weight,
                                const void* k_weight, int weight_fp32, float eps, const int32_t* kv_rows,
                                int64_t cache_rows, void* stream) {
  bool empty = false;
  if (sdpa_status_t st = check_common(b, s, h, h_kv, d, d_v, dtype, rot, cos, sin, n_pos, positions, q_weight,
                                      k_weight, eps, &empty))
    return st;
  if ((v == nullptr) != (v_out == nullptr)) return fail(SDPA_ERR_INVALID_ARG, "v and v_out go together");
  if (cache_rows < 0 || cache_rows > kMaxTokens) return fail(SDPA_ERR_INVALID_ARG, "cache_rows");
  if (empty) return SDPA_OK;
  if ((reinterpret_cast<uintptr_t>(kv_rows) & 3u) != 0) return fail(SDPA_ERR_MISALIGNED, "kv_rows");
  const int64_t kv_out_rows = kv_rows != nullptr ? cache_rows : s;
  sdpa_status_t st = check_rows(q, b, s, h, "q");
  if (!st) st = check_rows(k, b, s, h_kv, "k");
  if (!st && v != nullptr) st = check_rows(v, b, s, h_kv, "v");
  if (!st) st = check_rows(q_out, b, s, h, "q_out");
  if (!st) st = check_rows(k_out, b, kv_out_rows, h_kv, "k_out");
  if (!st && v != nullptr) st = check_rows(v_out, b, kv_out_rows, h_kv, "v_out");
  if (st) return st;

  NormRopeParams p{};
  fill_common(&p, b, s, d, rot, interleaved, cos, sin, n_pos, positions, weight_fp32, eps);
  p.kv_rows = kv_rows;
  p.cache_rows = cache_rows;
  const int hi = static_cast<int>(h), hk = static_cast<int>(h_kv), di = static_cast<int>(d);
  const int cached = kv_rows != nullptr ? 1 : 0;
  p.n_kinds = v != nullptr ? 3 : 2;
  p.kind[0] = RowKind{row_set(q, b, s, h), row_set(q_out, b, s, h), q_weight, hi, di, rot > 0, 0, 0, 0};
  p.kind[1] = RowKind{row_set(k, b, s, h_kv), row_set(k_out, b, kv_out_rows, h_kv), k_weight, hk, di, rot > 0,
                      cached, 0, 0};
  if (v != nullptr)
    p.kind[2] = RowKind{row_set(v, b, s, h_kv), row_set(v_out, b, kv_out_rows, h_kv), nullptr, hk,
                        static_cast<int>(d_v), 0, cached, 0, 0};
  const int blocks = norm_rope_plan(&p, false);
  if (blocks < 0) return fail(SDPA_ERR_UNSUPPORTED, "too many rows");
  const cudaError_t e = launch_norm_rope_fwd(dtype == SDPA_BF16, p, blocks, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, cudaGetErrorString(e));
  return SDPA_OK;
}

size_t sdpa_qk_norm_rope_bwd_workspace_size(int64_t b, int64_t s, int64_t h, int64_t h_kv, int64_t d, int64_t d_v) {
  bool empty = false;
  if (check_common(b, s, h, h_kv, d, d_v, SDPA_BF16, 0, nullptr, nullptr, 0, nullptr, nullptr, nullptr, 1.f,
                   &empty) != SDPA_OK)
    return 0;
  // blocks with the values' rows (block numbers of the others do not depend on them past this bound)
  NormRopeParams p{};
  fill_common(&p, b, s, d, 0, 0, nullptr, nullptr, 0, nullptr, 0, 1.f);
  size_t most = 0;
  for (int call = 0; call < 6; ++call) {  // with and without values, either weight or both
    const int kinds = 2 + call / 3, weights = call % 3 + 1;
    p.n_kinds = kinds;
    for (int i = 0; i < kinds; ++i) {
      p.kind[i].heads = static_cast<int>(i == 0 ? h : h_kv);
      p.kind[i].weight = (weights >> i) & 1 ? &p : nullptr;  // (whether there is one)
    }
    const int blocks = empty ? 0 : norm_rope_plan(&p, true);
    if (blocks < 0) return 0;
    const size_t bytes = static_cast<size_t>(blocks) * static_cast<size_t>(d) * sizeof(float);
    if (bytes > most) most = bytes;
  }
  return (most + 255) & ~size_t(255);
}

sdpa_status_t sdpa_qk_norm_rope_bwd(int64_t b, int64_t s, int64_t h, int64_t h_kv, int64_t d, int64_t d_v,
                                    sdpa_dtype_t dtype, const sdpa_rows_t* dq_out, const sdpa_rows_t* dk_out,
                                    const sdpa_rows_t* dv_out, const sdpa_rows_t* q, const sdpa_rows_t* k,
                                    const sdpa_rows_t* dq, const sdpa_rows_t* dk, const sdpa_rows_t* dv,
                                    int64_t rot, int interleaved, const float* cos, const float* sin,
                                    int64_t n_pos, const int32_t* positions, const void* q_weight,
                                    const void* k_weight, int weight_fp32, float eps, void* dq_weight,
                                    void* dk_weight, void* workspace, size_t workspace_bytes, void* stream) {
  bool empty = false;
  if (sdpa_status_t st = check_common(b, s, h, h_kv, d, d_v, dtype, rot, cos, sin, n_pos, positions, q_weight,
                                      k_weight, eps, &empty))
    return st;
  if ((dv_out == nullptr) != (dv == nullptr)) return fail(SDPA_ERR_INVALID_ARG, "dv_out and dv go together");
  if ((q_weight == nullptr) != (dq_weight == nullptr) || (k_weight == nullptr) != (dk_weight == nullptr))
    return fail(SDPA_ERR_INVALID_ARG, "a weight and its gradient go together");
  if (((reinterpret_cast<uintptr_t>(dq_weight) | reinterpret_cast<uintptr_t>(dk_weight)) & 15u) != 0)
    return fail(SDPA_ERR_MISALIGNED, "dq_weight, dk_weight");
  const bool normed = q_weight != nullptr || k_weight != nullptr;
  if (empty && !normed) return SDPA_OK;

  NormRopeParams p{};
  fill_common(&p, b, s, d, rot, interleaved, cos, sin, n_pos, positions, weight_fp32, eps);
  p.n_kinds = dv != nullptr ? 3 : 2;
  if (!empty) {
    sdpa_status_t st = check_rows(dq_out, b, s, h, "dq_out");
    if (!st) st = check_rows(dk_out, b, s, h_kv, "dk_out");
    if (!st && dv != nullptr) st = check_rows(dv_out, b, s, h_kv, "dv_out");
    if (!st && q_weight != nullptr) st = check_rows(q, b, s, h, "q");
    if (!st && k_weight != nullptr) st = check_rows(k, b, s, h_kv, "k");
    if (!st) st = check_rows(dq, b, s, h, "dq");
    if (!st) st = check_rows(dk, b, s, h_kv, "dk");
    if (!st && dv != nullptr) st = check_rows(dv, b, s, h_kv, "dv");
    if (st) return st;
    const int hi = static_cast<int>(h), hk = static_cast<int>(h_kv), di = static_cast<int>(d);
    p.kind[0] = RowKind{row_set(dq, b, s, h), row_set(dq_out, b, s, h), q_weight, hi, di, rot > 0, 0, 0, 0};
    p.kind[1] = RowKind{row_set(dk, b, s, h_kv), row_set(dk_out, b, s, h_kv), k_weight, hk, di, rot > 0, 0, 0, 0};
    if (dv != nullptr)
      p.kind[2] = RowKind{row_set(dv, b, s, h_kv), row_set(dv_out, b, s, h_kv), nullptr, hk,
                          static_cast<int>(d_v), 0, 0, 0, 0};
    if (q_weight != nullptr) p.x[0] = row_set(q, b, s, h);
    if (k_weight != nullptr) p.x[1] = row_set(k, b, s, h_kv);
  }
  const int blocks = empty ? 0 : norm_rope_plan(&p, true);
  if (blocks < 0) return fail(SDPA_ERR_UNSUPPORTED, "too many rows");
  if (normed && blocks > 0) {
    if (workspace == nullptr || workspace_bytes < static_cast<size_t>(blocks) * d * sizeof(float))
      return fail(SDPA_ERR_WORKSPACE, "workspace");
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return fail(SDPA_ERR_MISALIGNED, "workspace");
  }
  p.dw_part = static_cast<float*>(workspace);
  const cudaError_t e = launch_norm_rope_bwd(dtype == SDPA_BF16, p, blocks, dq_weight, dk_weight,
                                             static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, cudaGetErrorString(e));
  return SDPA_OK;
}

}  // extern "C"
