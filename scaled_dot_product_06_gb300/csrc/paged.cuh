// Parameters and launchers of the attention over a paged cache (paged_kernel.cuh,
// paged_join.cu).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace sdpa {

constexpr int kPagedTile = 128;   // keys a tile
constexpr int kPagedBox = 64;     // most keys of one copy
constexpr int kPagedCost = 1;     // what a unit costs besides its key tiles, in tiles
constexpr int kPagedGrid = 152;   // CTAs at most: one an SM
// Key tiles up to which units are not cut, few units and many (a quarter of the CTAs). 80
// units of 8 tiles (10 sequences of 1000 keys, 8 K/V heads) took 14.1 us cut and take 11.2, 512
// ragged ones of up to 8 28.6 and 27.0, 4096 133.5 and 132.0; 8 units 8.2 cut and 9.1 whole.
// (Up to 16 tiles: 64 units 13.2 cut and 15.5 whole, 512 46.9 and 47.4.) Up to 4: three units
// 8.0 and 5.9, 600 units 28.4 and 25.1.
constexpr int kPagedWhole = 4, kPagedWholeMany = 8;
constexpr int kPagedGroup = 32;   // parts that are joined at once

// A unit of work is a sequence, a K/V head and a block of its query rows. The
// units of all sequences, each as long as its key tiles and kPagedCost, are one
// line that is cut into as many equal runs as there are CTAs. Where a sequence can have
// no more than kPagedWhole... key tiles (the host knows what a row of the table holds and the
// window, not the lengths), units are not cut: each is all of the run's in which it
// begins; then there is nothing to join and no workspace. Where there are no more of them
// than CTAs, or a sequence has one tile, each has a length of 1, so that no length is waited
// for (2048 units of up to 100 keys 19.6 us for 20.2); else they have the lengths they
// have cut (2048 of up to 512 keys 46.7 us, for 55.7 with a length of 1 each; 256 equal
// ones of 512 keys 14.5 for 14.0).
enum : int { kUnitsCut = 0, kUnitsAlike, kUnitsWhole };

struct PagedParams {
  int B, H_kv;
  int R, s_q;              // query rows of a K/V head: (h / h_kv) * s_q, row x of token x % s_q
  int row_blocks;          // blocks of the rows
  int page_shift;          // log2 of the tokens a page
  int box, box_shift;      // keys a copy: the page's, at most kPagedBox
  int n_pages;             // pages of the pool
  int64_t table_stride;
  int capacity;            // tokens a row of the table can hold
  int left;                // keys before a token that it sees, < 0: all
  const int* table;
  const int* seqlen;
  float scale_log2;        // factor of the raw score in the exponent
  float cap_in;            // capped scores: factor of the raw score in the tanh (scale_log2 = softcap log2(e))
  int capped;
  uint32_t q_box;          // bytes of a 64-column box of Q
  int grid;
  int whole;               // kUnits...
  // Partial rows of units cut by a run's end: run c leaves slot 2 c + 1 for the unit whose
  // first part it has, and slot 2 c for the unit it begins within.
  float* part;             // [2 grid][rows a block][d_v]
  float* part_lse;         // [2 grid][rows a block], base 2
  // [grid][first group, later group, unit][half of the rows]: parts left so far (paged_count_in),
  // at the first run of the group or unit
  unsigned long long* words;
  unsigned long long nonce;  // 48 bits, of this call
  // Not null: the parts are joined by the kernel for that, which finds here {unit + 1 of
  // slot 2 c or 0, 1 if the unit ends there, unit + 1 of slot 2 c + 1 or 0, 0}
  int4* runs;              // [grid]
  void* o;
  float* lse;
  uint32_t* err;
};

// Rows a block.
__host__ __device__ constexpr int paged_rows(int R) { return R <= 8 ? 8 : R <= 16 ? 16 : R <= 32 ? 32 : 64; }

cudaError_t launch_paged_bf16(int d_qk, int d_v, const CUtensorMap (&m)[3], const PagedParams& p, cudaStream_t st);
cudaError_t launch_paged_fp16(int d_qk, int d_v, const CUtensorMap (&m)[3], const PagedParams& p, cudaStream_t st);
cudaError_t launch_paged_join(bool bf16, int d_v, const PagedParams& p, cudaStream_t st);

}  // namespace sdpa
