// Block tables and slot maps of a paged cache, built from request lengths.
//
// Request i has n tokens cached and x new ones; with pages of P tokens
//   have = ceil(n / P),  need = ceil((n + x) / P),  k = need - have
// pages are asked for, and page have + j of the request is entry
//   head + sum_{i' < i} k_i' + j   (modulo the pool)
// of the ring of free pages. New token t lies at
//   slot = table[i][(n + t) / P] P + (n + t) mod P.
// Ended requests' pages go behind the ring's tail in the same way. So three
// sums over the requests (tokens, pages asked for, pages given back) are all
// that one entry needs of the others.
//
// Nothing here is worth more than a launch and three trips to memory (lengths,
// then pages, then the stores): a few CTAs, each of which scans all
// requests, 1024 at a time, and then takes its share of the tokens and table
// entries, found by bisection of the sums in shared memory. Where the lengths or
// the ring's counters are advanced in place, the CTAs are a cluster, and they are
// written after a barrier of all that read them. A token each of 256 requests takes 5.5
// us, 16384 tokens of 13 prompts 6.4, 131072 entries of 1000 requests 8.7 (1 MB: none of
// it is bandwidth), captured and in a row.
#include "common.cuh"
#include "page_slots.cuh"

namespace sdpa {

namespace {

constexpr int kReq = 1024;  // threads, and requests scanned at a time
constexpr int kWarps = kReq / 32;
// A CTA takes 4096 entries in one go; where there are more, more CTAs do, up to the
// eight of a cluster where something is advanced in place. (Eight always took 19 us
// of 131072 entries of 1000 requests.)
constexpr int kCluster = 8, kCtas = 64;
constexpr int64_t kShare = 4096;

__device__ __forceinline__ uint32_t ceil_div(uint32_t a, uint32_t b) { return a / b + (a % b != 0 ? 1u : 0u); }

// Page of a token; pages of a power of two (shift >= 0) without a division.
__device__ __forceinline__ uint32_t page_of(uint32_t token, const PageSlotsParams& p) {
  return p.shift >= 0 ? token >> p.shift : token / static_cast<uint32_t>(p.page);
}
__device__ __forceinline__ uint32_t pages_of(uint32_t tokens, const PageSlotsParams& p) {
  return tokens > 0 ? page_of(tokens - 1, p) + 1u : 0u;
}

// Sums of tokens (held at `cap`, so that they stay in 32 bits; they matter only up
// to the rows there are), pages asked for, pages given back.
struct Sums {
  uint32_t tok, take, back;
};
__device__ __forceinline__ Sums add(const Sums& a, const Sums& b, uint32_t cap) {
  return Sums{min(a.tok + b.tok, cap), a.take + b.take, a.back + b.back};
}
__device__ __forceinline__ Sums up(const Sums& s, int o) {
  return Sums{__shfl_up_sync(0xffffffffu, s.tok, o), __shfl_up_sync(0xffffffffu, s.take, o),
              __shfl_up_sync(0xffffffffu, s.back, o)};
}

struct Shared {
  uint32_t tok_end[kReq], take_end[kReq], back_end[kReq];  // inclusive sums
  uint32_t len[kReq], add[kReq], take[kReq];               // cached tokens, new ones, pages asked for
  uint8_t served[kReq];
  Sums warp[kWarps];
  Sums carry;
  uint32_t taken;  // pages taken by served requests
};

// x modulo n, n > 0: counters below 2^32 without a 64-bit division.
__device__ __forceinline__ uint32_t mod(uint64_t x, uint32_t n) {
  return (x >> 32) == 0 ? static_cast<uint32_t>(x) % n : static_cast<uint32_t>(x % n);
}

// The first of n entries above x (n: none).
__device__ __forceinline__ int above(const uint32_t* ends, int n, uint32_t x) {
  int lo = 0;
#pragma unroll 1
  for (int step = kReq / 2; step > 0; step >>= 1)
    if (lo + step <= n && ends[lo + step - 1] <= x) lo += step;
  return lo < n && ends[lo] <= x ? lo + 1 : lo;
}

__global__ void __launch_bounds__(kReq, 1) page_slots_kernel(const __grid_constant__ PageSlotsParams p) {
  __shared__ Shared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t ctas = gridDim.x, first = blockIdx.x * kReq + tid, step = ctas * kReq;
  const uint32_t page = static_cast<uint32_t>(p.page);
  const bool packed = p.packed != 0;
  const uint32_t rows = static_cast<uint32_t>(p.rows), cap = packed ? rows + 1u : 0u;
  // Launched while the kernel before runs out, as the one behind may be while this one
  // does (256 requests 5.5 us for 5.8): memory is looked at from here on.
  asm volatile("griddepcontrol.launch_dependents;\ngriddepcontrol.wait;" ::: "memory");
  const int64_t head = p.range[0], tail = p.range[1];
  int n_in = tid < p.b ? p.seqlens[tid] : 0, x_in = tid < p.b ? p.new_tokens[tid] : 0;  // of the chunk to come
  if (tid == 0) s.taken = 0u;
  __syncthreads();
  // (any contents of the counters stay inside the ring)
  const uint32_t avail =
      tail <= head ? 0u : static_cast<uint32_t>(min(static_cast<uint64_t>(tail) - static_cast<uint64_t>(head),
                                                    static_cast<uint64_t>(p.pool)));
  const uint32_t head0 = p.pool > 0 ? mod(static_cast<uint64_t>(head), p.pool) : 0u;
  const uint32_t tail0 = p.pool > 0 ? mod(static_cast<uint64_t>(tail), p.pool) : 0u;
  auto ring_at = [&](uint32_t from, uint32_t i) {  // i < pool
    const uint32_t at = from + i;
    return at >= p.pool ? at - p.pool : at;
  };

  Sums before{0u, 0u, 0u};  // of the requests before this chunk
  int len_out = 0;
  // Scans requests r0 .. r0 + kReq - 1 into s; returns this thread's new length.
  auto scan = [&](int r0) -> int {
    const bool live = r0 + tid < p.b;
    const int x = x_in;
    const uint32_t n = static_cast<uint32_t>(max(n_in, 0)), more = static_cast<uint32_t>(max(x, 0));
    const uint32_t have = pages_of(n, p), need = pages_of(n + more, p);
    const uint32_t wide = static_cast<uint32_t>(p.width);
    const bool room = live && x >= 0 && need <= wide;
    // (a padded request asks for pages when its tokens have entries; a packed one's
    // place is known after the sum, and where there is no room for it none of those
    // behind it has any, so that what it asks for changes nothing)
    const bool padded_fits = packed || more <= static_cast<uint32_t>(p.per);
    Sums mine{packed ? min(more, cap) : 0u, room && padded_fits ? need - have : 0u,
              live && x < 0 ? min(have, wide) : 0u};
    const uint32_t asked = mine.take;
    Sums sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Sums u = up(sum, o);
      if (lane >= o) sum = add(sum, u, cap);
    }
    if (lane == 31) s.warp[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      Sums w = s.warp[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const Sums u = up(w, o);
        if (lane >= o) w = add(w, u, cap);
      }
      s.warp[lane] = w;
    }
    __syncthreads();
    if (warp > 0) sum = add(sum, s.warp[warp - 1], cap);
    sum = add(sum, before, cap);
    const bool fits = room && (packed ? sum.tok <= rows : padded_fits);
    const bool served = fits && (asked == 0 || sum.take <= avail);
    s.tok_end[tid] = sum.tok;
    s.take_end[tid] = sum.take;
    s.back_end[tid] = sum.back;
    s.len[tid] = n;
    s.add[tid] = more;
    s.take[tid] = asked;
    s.served[tid] = served ? 1 : 0;
    // served requests are the first ones in the order of their pages: the most taken is
    // the last one's sum
    const uint32_t upto = __reduce_max_sync(0xffffffffu, served && asked > 0 ? sum.take : 0u);
    if (lane == 0 && upto > 0) atomicMax(&s.taken, upto);
    if (tid == kReq - 1) s.carry = sum;
    // the next chunk's
    const int next = r0 + kReq + tid;
    n_in = next < p.b ? p.seqlens[next] : 0;
    x_in = next < p.b ? p.new_tokens[next] : 0;
    __syncthreads();
    return x < 0 ? 0 : static_cast<int>(served ? n + more : n);
  };

#pragma unroll 1
  for (int r0 = 0; r0 < p.b; r0 += kReq) {
    len_out = scan(r0);
    const int n_req = min(kReq, p.b - r0);
    const Sums after = s.carry;
    // ---- tokens, four at a time
    const uint32_t lo = packed ? min(before.tok, rows)
                                   : static_cast<uint32_t>(r0) * static_cast<uint32_t>(p.per);
    const uint32_t hi = packed ? min(after.tok, rows)
                                   : static_cast<uint32_t>(r0 + n_req) * static_cast<uint32_t>(p.per);
#pragma unroll 1
    for (uint32_t g = lo / 4 + first; g < ceil_div(hi, 4); g += step) {
      // where the tokens' page numbers are, and their rows of the page; the four are
      // then fetched together
      const int* where[4] = {nullptr, nullptr, nullptr, nullptr};
      uint32_t off[4] = {0u, 0u, 0u, 0u};
      int4 pos = make_int4(0, 0, 0, 0);
      int i = -1;                       // request of the chunk
      uint32_t start = 0, end = 0;      // its entries
#pragma unroll 1
      for (uint32_t r = 4 * g; r < 4 * g + 4; ++r) {
        const int* own = nullptr;
        uint32_t own_off = 0;
        int own_pos = 0;
        if (r >= lo && r < hi) {
          if (r >= end) {  // another request's first token here
            if (packed) {
              if (i < 0) {
                i = above(s.tok_end, n_req, r);
              } else {  // the next one that has tokens
#pragma unroll 1
                while (s.tok_end[i] <= r) ++i;
              }
              start = i > 0 ? s.tok_end[i - 1] : before.tok;
              end = s.tok_end[i];
            } else {
              i = i < 0 ? static_cast<int>(r / static_cast<uint32_t>(p.per)) - r0 : i + 1;
              start = static_cast<uint32_t>(r0 + i) * static_cast<uint32_t>(p.per);
              end = start + static_cast<uint32_t>(p.per);
            }
          }
          const uint32_t t = r - start;
          if (t < s.add[i]) {
            const uint32_t place = s.len[i] + t, pg = page_of(place, p);
            own_pos = static_cast<int>(place);
            if (s.served[i]) {
              const uint32_t have = pages_of(s.len[i], p);
              own = pg < have ? p.table + (r0 + i) * p.table_stride + pg
                              : p.ring + ring_at(head0, s.take_end[i] - s.take[i] + pg - have);
              own_off = place - pg * page;
            }
          }
        }
        where[0] = where[1], where[1] = where[2], where[2] = where[3], where[3] = own;
        off[0] = off[1], off[1] = off[2], off[2] = off[3], off[3] = own_off;
        pos = make_int4(pos.y, pos.z, pos.w, own_pos);
      }
      int id[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) id[e] = where[e] != nullptr ? *where[e] : -1;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        id[e] = static_cast<uint32_t>(id[e]) < p.pool ? static_cast<int>(id[e] * page + off[e]) : -1;
      int4 slot = make_int4(id[0], id[1], id[2], id[3]);
      if (4 * g >= lo && 4 * g + 4 <= hi) {
        reinterpret_cast<int4*>(p.slots)[g] = slot;
        reinterpret_cast<int4*>(p.positions)[g] = pos;
      } else {  // shared with the chunk before or after, or the end
#pragma unroll 1
        for (uint32_t r = 4 * g; r < 4 * g + 4; ++r) {
          if (r >= lo && r < hi) {
            p.slots[r] = slot.x;
            p.positions[r] = pos.x;
          }
          slot = make_int4(slot.y, slot.z, slot.w, 0);
          pos = make_int4(pos.y, pos.z, pos.w, 0);
        }
      }
    }
    // ---- new entries of the table
    // (by other warps than the tokens', where there are few of both)
#pragma unroll 1
    for (uint32_t e = before.take + (first ^ 512u); e < min(after.take, avail); e += step) {
      const int i = above(s.take_end, n_req, e);
      if (!s.served[i]) continue;
      const uint32_t j = e - (s.take_end[i] - s.take[i]);
      p.table[(r0 + i) * p.table_stride + pages_of(s.len[i], p) + j] = p.ring[ring_at(head0, e)];
    }
    // ---- pages given back
#pragma unroll 1
    for (uint32_t e = before.back + (first ^ 256u); e < after.back; e += step) {
      const int i = above(s.back_end, n_req, e);
      const uint32_t j = e - (i > 0 ? s.back_end[i - 1] : before.back);
      if (p.pool > 0) p.ring[ring_at(tail0, e % p.pool)] = p.table[(r0 + i) * p.table_stride + j];
    }
    if (packed && blockIdx.x == 0) {
      if (r0 == 0 && tid == 0) p.starts[0] = 0;
      if (tid < n_req) p.starts[r0 + tid + 1] = static_cast<int>(min(s.tok_end[tid], rows));
    }
    before = after;
    __syncthreads();  // s is free again
  }
  if (packed) {  // behind the last token
    if (p.b == 0 && first == 0) p.starts[0] = 0;
    const uint32_t lo = min(before.tok, rows);
#pragma unroll 1
    for (uint32_t g = lo / 4 + first; g < ceil_div(rows, 4); g += step) {
      if (4 * g >= lo && 4 * g + 4 <= rows) {
        reinterpret_cast<int4*>(p.slots)[g] = make_int4(-1, -1, -1, -1);
        reinterpret_cast<int4*>(p.positions)[g] = make_int4(0, 0, 0, 0);
      } else {
#pragma unroll 1
        for (uint32_t r = max(4 * g, lo); r < min(4 * g + 4, rows); ++r) {
          p.slots[r] = -1;
          p.positions[r] = 0;
        }
      }
    }
  }
  // ---- what may be advanced in place, after all have read it
  if (p.in_place && ctas > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
  if (blockIdx.x != 0) return;
  if (p.b <= kReq) {
    if (tid < p.b) p.seqlens_out[tid] = len_out;
  } else {
    const Sums all = before;
    before = Sums{0u, 0u, 0u};
    n_in = p.seqlens[tid];
    x_in = p.new_tokens[tid];
#pragma unroll 1
    for (int r0 = 0; r0 < p.b; r0 += kReq) {
      const int n = scan(r0);
      if (r0 + tid < p.b) p.seqlens_out[r0 + tid] = n;
      before = s.carry;
      __syncthreads();
    }
    before = all;
  }
  if (tid == 0) {
    p.range_out[0] = head + s.taken;
    p.range_out[1] = tail + before.back;
  }
}

}  // namespace

cudaError_t launch_page_slots(const PageSlotsParams& p, cudaStream_t st) {
  const int64_t entries = p.packed ? p.rows : static_cast<int64_t>(p.b) * p.per;
  const int64_t want = (entries + kShare - 1) / kShare, most = p.in_place ? kCluster : kCtas;
  unsigned ctas = static_cast<unsigned>(want < 1 ? 1 : want > most ? most : want);
  if (p.in_place && ctas > 1) ctas = kCluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kReq);
  cfg.stream = st;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = ctas;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.in_place && ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, page_slots_kernel, p);
}

}  // namespace sdpa
