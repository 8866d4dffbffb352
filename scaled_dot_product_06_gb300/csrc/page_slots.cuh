// Parameters and launcher of the block tables and slot maps (page_slots.cu).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace sdpa {

struct PageSlotsParams {
  int b;                   // requests
  int page, shift;         // tokens a page; its log2, or -1
  int in_place;            // seqlens_out is seqlens or range_out is range
  int width;               // pages a row of the table holds
  int64_t table_stride;    // elements between its rows
  uint32_t pool;           // pages of the pool = entries of the ring
  int packed;              // tokens of all requests one after another, else `per` entries a request
  int rows;                // packed: entries of slots and positions
  int per;
  const int* seqlens;      // [b] tokens in the cache
  const int* new_tokens;   // [b] new ones; negative: the request has ended
  int* table;
  int* ring;               // [pool] free pages: entries [range[0], range[1]) modulo pool
  const int64_t* range;
  int* slots;              // [rows] or [b][per]
  int* positions;
  int* starts;             // [b + 1] (packed)
  int* seqlens_out;        // may be seqlens
  int64_t* range_out;      // may be range
};

cudaError_t launch_page_slots(const PageSlotsParams& p, cudaStream_t st);

}  // namespace sdpa
