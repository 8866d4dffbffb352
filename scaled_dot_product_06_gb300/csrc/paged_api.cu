// C entry points of the paged cache: block tables and slot maps, and the attention
// over the pages. Argument checks, tensor maps and launch parameters.
#include <algorithm>
#include <atomic>
#include <chrono>
#include <cmath>
#include <cstdio>

#include <cudaTypedefs.h>

#include "../../include/sdpa.h"
#include "common.cuh"
#include "host.cuh"
#include "page_slots.cuh"
#include "paged.cuh"

namespace {

using namespace sdpa;

constexpr int64_t kMaxInt = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxKeys = (int64_t{1} << 29) - 256;  // keys of a sequence, as elsewhere

sdpa_status_t fail(sdpa_status_t s, const char* what) {
  set_last_error(what);
  return s;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Pages as rows of [n_pages][h_kv][page_size][d], any strides that TMA takes: positive
// multiples of 16 bytes below 2^40, where a dimension has more than one element.
sdpa_status_t check_pages(const sdpa_rows_t* r, int64_t n_pages, int64_t page_size, int64_t h_kv, const char* what) {
  char msg[96];
  if (r == nullptr || r->ptr == nullptr) {
    snprintf(msg, sizeof(msg), "%s is null", what);
    return fail(SDPA_ERR_INVALID_ARG, msg);
  }
  const int64_t n[3] = {n_pages, page_size, h_kv}, stride[3] = {r->batch_stride, r->row_stride, r->head_stride};
  bool odd = !aligned(r->ptr, 16);
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;
    if (stride[i] <= 0 || stride[i] >= (int64_t{1} << 38)) {
      snprintf(msg, sizeof(msg), "%s: strides must be positive and below 2^38 elements", what);
      return fail(SDPA_ERR_INVALID_ARG, msg);
    }
    odd |= (stride[i] & 7) != 0;
  }
  if (odd) {
    snprintf(msg, sizeof(msg), "%s: base and strides must be multiples of 16 bytes", what);
    return fail(SDPA_ERR_MISALIGNED, msg);
  }
  return SDPA_OK;
}

// 4-D map of 16-bit elements, boxes of 64 columns and box_rows rows; strides in elements.
sdpa_status_t make_map4(CUtensorMap* m, int dtype, const void* ptr, const int64_t (&n)[4], const int64_t (&stride)[3],
                        uint32_t box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc;
  if (sdpa_status_t s = tensor_map_encoder(&enc)) return s;
  cuuint64_t dims[4], strides[3];
  for (int i = 0; i < 4; ++i) dims[i] = static_cast<cuuint64_t>(n[i]);
  for (int i = 0; i < 3; ++i) strides[i] = static_cast<cuuint64_t>((n[i + 1] > 1 ? stride[i] : n[0]) * 2);
  cuuint32_t box[4] = {64, box_rows, 1, 1}, es[4] = {1, 1, 1, 1};
  const CUresult r = enc(m, dtype == SDPA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                         const_cast<void*>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r == CUDA_SUCCESS) return SDPA_OK;
  char msg[96];
  snprintf(msg, sizeof(msg), "cuTensorMapEncodeTiled (pages) failed (CUresult %d)", static_cast<int>(r));
  return fail(SDPA_ERR_CUDA, msg);
}

int log2_of(int64_t n) {
  int s = 0;
  while ((int64_t{1} << s) < n) ++s;
  return s;
}

// Workspace: partial rows, their log-sums, and the words that parts are counted in at
// or the runs' records.
size_t paged_bytes(int64_t R, int64_t d_v) {
  const size_t rows = static_cast<size_t>(2 * kPagedGrid) * static_cast<size_t>(paged_rows(static_cast<int>(R)));
  return rows * (static_cast<size_t>(d_v) + 1) * sizeof(float) + 6 * kPagedGrid * sizeof(unsigned long long);
}

// A number of 48 bits that no workspace holds by chance: from a random place on (the
// clock and an address, mixed by the finaliser of splitmix64), another for each call.
unsigned long long next_nonce() {
  static std::atomic<unsigned long long> next{[] {
    unsigned long long x = static_cast<unsigned long long>(std::chrono::steady_clock::now().time_since_epoch().count());
    x ^= reinterpret_cast<uintptr_t>(&x) * 0x9E3779B97F4A7C15ull;
    x = (x ^ (x >> 30)) * 0xBF58476D1CE4E5B9ull;
    x = (x ^ (x >> 27)) * 0x94D049BB133111EBull;
    return x ^ (x >> 31);
  }()};
  return (next.fetch_add(1, std::memory_order_relaxed) & ((1ull << 48) - 1)) | (1ull << 47);
}

// Whether units of sequences of up to `capacity` keys are left whole, of which s_q
// tokens see no more than left + s_q (left < 0: all), in up to a tile more.
bool whole_units(int64_t capacity, int64_t units = 0, int64_t left = -1, int64_t s_q = 0) {
  const int64_t most = (units >= kPagedGrid / 4 ? kPagedWholeMany : kPagedWhole) * kPagedTile;
  return capacity <= most || (left >= 0 && left <= most && left + s_q + kPagedTile - 1 <= most);
}

// Heads and rows that both the size and the call check; *R: rows of a K/V head.
sdpa_status_t check_rows_of(int64_t b, int64_t h, int64_t h_kv, int64_t s_q, int64_t d_qk, int64_t d_v, int64_t* R) {
  if (b < 0 || h < 0 || s_q < 0) return fail(SDPA_ERR_INVALID_ARG, "sizes");
  if (!((d_qk == 64 && d_v == 64) || (d_qk == 128 && d_v == 128) || (d_qk == 192 && d_v == 128)))
    return fail(SDPA_ERR_UNSUPPORTED, "head sizes must be (64, 64), (128, 128) or (192, 128)");
  constexpr int64_t kMost = int64_t{1} << 24;
  if (b > kMost || h > kMost || s_q > kMost || b * h > kMost || h * s_q > kMost || b * h * s_q > (int64_t{1} << 30))
    return fail(SDPA_ERR_UNSUPPORTED, "too many query rows");
  if (h_kv < 1 || h_kv > kMost || (h > 0 && (h_kv > h || h % h_kv != 0)))
    return fail(SDPA_ERR_INVALID_ARG, "h_kv must divide h");
  *R = h / h_kv * s_q;
  return SDPA_OK;
}

}  // namespace

extern "C" {

sdpa_status_t sdpa_page_slots(int64_t b, int64_t page_size, int64_t table_width, int64_t table_stride,
                              int64_t n_pages, int64_t rows, int64_t width, const int32_t* seqlens,
                              const int32_t* new_tokens, int32_t* block_table, int32_t* free_pages,
                              const int64_t* free_range, int32_t* slots, int32_t* positions, int32_t* starts,
                              int32_t* seqlens_out, int64_t* free_range_out, void* stream) {
  if (b < 0 || page_size < 1 || table_width < 0 || n_pages < 0 || rows < 0 || width < 0)
    return fail(SDPA_ERR_INVALID_ARG, "sizes");
  if (rows > 0 && width > 0) return fail(SDPA_ERR_INVALID_ARG, "either packed rows or a width of a padded batch");
  constexpr int64_t kMost = int64_t{1} << 30;
  if (b > kMost || page_size > kMost || table_width > kMost || n_pages > kMost || rows > kMost || width > kMost ||
      b * width > kMost || b * table_width > kMost || n_pages * page_size > kMaxInt ||
      table_width * page_size > kMaxInt)
    return fail(SDPA_ERR_UNSUPPORTED, "too many tokens or pages");
  if (b > 1 && table_stride < table_width) return fail(SDPA_ERR_INVALID_ARG, "table_stride");
  if (b > 1 && table_stride > (int64_t{1} << 40)) return fail(SDPA_ERR_UNSUPPORTED, "table_stride");
  const bool packed = rows > 0 || starts != nullptr;
  if (packed && width > 0) return fail(SDPA_ERR_INVALID_ARG, "starts are of packed rows");
  const int64_t entries = packed ? rows : b * width;
  if ((b > 0 && (!seqlens || !new_tokens || !seqlens_out || (table_width > 0 && !block_table))) ||
      (n_pages > 0 && !free_pages) || !free_range || !free_range_out ||
      (entries > 0 && (!slots || !positions)) || (packed && !starts))
    return fail(SDPA_ERR_INVALID_ARG, "null pointer");
  if (!aligned(slots, 16) || !aligned(positions, 16) || !aligned(seqlens, 4) || !aligned(new_tokens, 4) ||
      !aligned(block_table, 4) || !aligned(free_pages, 4) || !aligned(starts, 4) || !aligned(seqlens_out, 4) ||
      !aligned(free_range, 8) || !aligned(free_range_out, 8))
    return fail(SDPA_ERR_MISALIGNED, "slots and positions on 16 bytes, the others on an element's");
  PageSlotsParams p{};
  p.b = static_cast<int>(b);
  p.page = static_cast<int>(page_size);
  p.shift = (page_size & (page_size - 1)) == 0 ? log2_of(page_size) : -1;
  p.in_place = seqlens_out == seqlens || free_range_out == free_range;
  p.width = static_cast<int>(table_width);
  p.table_stride = b > 1 ? table_stride : 0;
  p.pool = static_cast<uint32_t>(n_pages);
  p.packed = packed ? 1 : 0;
  p.rows = static_cast<int>(rows);
  p.per = static_cast<int>(width);
  p.seqlens = seqlens;
  p.new_tokens = new_tokens;
  p.table = block_table;
  p.ring = free_pages;
  p.range = free_range;
  p.slots = slots;
  p.positions = positions;
  p.starts = starts;
  p.seqlens_out = seqlens_out;
  p.range_out = free_range_out;
  const cudaError_t e = launch_page_slots(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, cudaGetErrorString(e));
  return SDPA_OK;
}

size_t sdpa_fwd_paged_workspace_size(int64_t h, int64_t h_kv, int64_t s_q, int64_t d_qk, int64_t d_v,
                                     int64_t page_size, int64_t table_width) {
  int64_t R = 0;
  if (check_rows_of(1, h, h_kv, s_q, d_qk, d_v, &R) != SDPA_OK || R == 0) return 0;
  if (page_size < 1 || table_width < 0 || page_size > kMaxKeys || table_width > kMaxKeys) return 0;
  if (whole_units(page_size * table_width)) return 0;
  return (paged_bytes(R, d_v) + 255) & ~size_t(255);
}

sdpa_status_t sdpa_fwd_paged(int64_t b, int64_t h, int64_t h_kv, int64_t s_q, int64_t d_qk, int64_t d_v, float scale,
                             float softcap, int64_t window_left, sdpa_dtype_t dtype, const void* q,
                             const sdpa_rows_t* k_pages, const sdpa_rows_t* v_pages, int64_t n_pages,
                             int64_t page_size, const int32_t* block_table, int64_t table_width,
                             int64_t table_stride, const int32_t* seqlen_k, void* o, float* lse, void* workspace,
                             size_t workspace_bytes, void* stream) {
  if (dtype != SDPA_BF16 && dtype != SDPA_FP16) return fail(SDPA_ERR_UNSUPPORTED, "dtype");
  int64_t R = 0;
  if (sdpa_status_t s = check_rows_of(b, h, h_kv, s_q, d_qk, d_v, &R)) return s;
  if (n_pages < 0 || table_width < 0) return fail(SDPA_ERR_INVALID_ARG, "n_pages, table_width");
  if (page_size < 8 || page_size > (int64_t{1} << 20) || (page_size & (page_size - 1)) != 0)
    return fail(SDPA_ERR_UNSUPPORTED, "page_size must be a power of two from 8 to 2^20");
  if (n_pages > kMaxInt || n_pages * page_size > kMaxInt || table_width > kMaxKeys ||
      table_width * page_size > kMaxKeys)
    return fail(SDPA_ERR_UNSUPPORTED, "too many keys");
  if (b > 1 && table_stride < table_width) return fail(SDPA_ERR_INVALID_ARG, "table_stride");
  if (b > 1 && table_stride > (int64_t{1} << 40)) return fail(SDPA_ERR_UNSUPPORTED, "table_stride");
  if (!std::isfinite(scale) || !std::isfinite(scale * kLog2e)) return fail(SDPA_ERR_INVALID_ARG, "scale must be finite");
  if (softcap != 0.f) {
    if (!(softcap > 0.f && softcap <= kSoftcapMost)) return fail(SDPA_ERR_INVALID_ARG, "softcap must lie in (0, 4096]");
    if (!std::isfinite(2.f * kLog2e * scale / softcap))
      return fail(SDPA_ERR_INVALID_ARG, "scale / softcap must be finite");
  }
  if (b == 0 || R == 0) return SDPA_OK;
  const int64_t capacity = n_pages > 0 ? table_width * page_size : 0;
  const int rows = paged_rows(static_cast<int>(R));
  const int64_t blocks = (R + rows - 1) / rows;
  const int64_t units = b * h_kv * blocks;
  const bool whole = whole_units(table_width * page_size, units, window_left, s_q);
  const int64_t line =
      units * ((whole ? kPagedWholeMany : (capacity + kPagedTile - 1) / kPagedTile) + kPagedCost);
  if (blocks * h_kv > kMaxInt / b || line > kMaxInt) return fail(SDPA_ERR_UNSUPPORTED, "too many key tiles");
  if (!q || !o || !lse || !seqlen_k || (capacity > 0 && !block_table)) return fail(SDPA_ERR_INVALID_ARG, "null pointer");
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 16) || !aligned(seqlen_k, 4) || !aligned(block_table, 4))
    return fail(SDPA_ERR_MISALIGNED, "q, o and lse on 16 bytes, seqlen_k and block_table on 4");
  if (capacity > 0) {
    if (sdpa_status_t s = check_pages(k_pages, n_pages, page_size, h_kv, "k_pages")) return s;
    if (sdpa_status_t s = check_pages(v_pages, n_pages, page_size, h_kv, "v_pages")) return s;
  }
  if (!whole && (workspace == nullptr || workspace_bytes < paged_bytes(R, d_v)))
    return fail(SDPA_ERR_WORKSPACE, "workspace");
  if (!whole && !aligned(workspace, 256)) return fail(SDPA_ERR_MISALIGNED, "workspace");

  PagedParams p{};
  p.B = static_cast<int>(b);
  p.H_kv = static_cast<int>(h_kv);
  p.R = static_cast<int>(R);
  p.s_q = static_cast<int>(s_q);
  p.row_blocks = static_cast<int>(blocks);
  p.page_shift = log2_of(page_size);
  p.box = static_cast<int>(std::min<int64_t>(page_size, kPagedBox));
  p.box_shift = log2_of(p.box);
  p.n_pages = static_cast<int>(n_pages);
  p.table_stride = b > 1 ? table_stride : 0;
  p.capacity = static_cast<int>(capacity);
  p.left = window_left < 0 || window_left >= capacity ? -1 : static_cast<int>(window_left);
  p.table = block_table;
  p.seqlen = seqlen_k;
  if (softcap != 0.f) {
    p.capped = 1;
    p.cap_in = scale / softcap;
    p.scale_log2 = kLog2e * softcap;
  } else if (scale == 0.f) {
    // every score 0: the capped form with a cap of 1 (the plain one masks raw
    // scores with infinities, which a zero factor would turn into NaN)
    p.capped = 1;
    p.scale_log2 = kLog2e;
  } else {
    p.scale_log2 = scale * kLog2e;
  }
  const int box_q = static_cast<int>(std::min<int64_t>(R, rows));
  p.q_box = static_cast<uint32_t>(128 * box_q);
  p.grid = static_cast<int>(std::min<int64_t>(kPagedGrid, whole ? units : line));
  p.whole = !whole ? kUnitsCut : units <= kPagedGrid || capacity <= kPagedTile ? kUnitsAlike : kUnitsWhole;
  if (!whole) {
    p.part = static_cast<float*>(workspace);
    p.part_lse = p.part + static_cast<int64_t>(2 * kPagedGrid) * rows * d_v;
    void* rest = p.part_lse + static_cast<int64_t>(2 * kPagedGrid) * rows;
    if (2 * units < p.grid) {  // more than two parts a unit (paged_kernel.cuh)
      p.runs = static_cast<int4*>(rest);
    } else {
      p.words = static_cast<unsigned long long*>(rest);
      p.nonce = next_nonce();
    }
  }
  p.o = o;
  p.lse = lse;
  CUtensorMap m[3];
  if (sdpa_status_t s = make_map4(&m[0], dtype, q, {d_qk, R, b, h_kv}, {d_qk, h_kv * R * d_qk, R * d_qk},
                                  static_cast<uint32_t>(box_q)))
    return s;
  if (capacity > 0) {
    const uint32_t box = static_cast<uint32_t>(p.box);
    if (sdpa_status_t s = make_map4(&m[1], dtype, k_pages->ptr, {d_qk, page_size, h_kv, n_pages},
                                    {k_pages->row_stride, k_pages->head_stride, k_pages->batch_stride}, box))
      return s;
    if (sdpa_status_t s = make_map4(&m[2], dtype, v_pages->ptr, {d_v, page_size, h_kv, n_pages},
                                    {v_pages->row_stride, v_pages->head_stride, v_pages->batch_stride}, box))
      return s;
  } else {
    m[1] = m[2] = m[0];  // (no copy reads them)
  }
  if (sdpa_status_t s = device_error_word(&p.err)) return s;
  const bool bf16 = dtype == SDPA_BF16;
  const int di = static_cast<int>(d_qk), dvi = static_cast<int>(d_v);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = bf16 ? launch_paged_bf16(di, dvi, m, p, st) : launch_paged_fp16(di, dvi, m, p, st);
  if (e == cudaSuccess && p.runs != nullptr) e = launch_paged_join(bf16, dvi, p, st);
  if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, cudaGetErrorString(e));
  return SDPA_OK;
}

}  // extern "C"
