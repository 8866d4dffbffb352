// Attention of each sequence's newest tokens over a key/value cache in pages
// (sm_103a).
//
// For the R = (h / h_kv) s_q query rows x of a sequence and K/V head,
//   S = scale Q K^T (capped: softcap tanh(S / softcap)), P = softmax(S), O = P V
// over the sequence's keys j, of which row x of token t = x mod s_q sees
// p - left <= j <= p, p = len - s_q + t. Key j is row j mod page of page
// table[j / page].
//
// A decoding step reads each key once for a few rows, so the keys take the
// products' long side: S^T = K Q^T has a tile of 128 keys on the tensor cores'
// 128 lanes and N = 16, 32 or 64 rows as its columns, and O^T = V^T P^T the
// values' width on the lanes. A thread has one key: its rows' scores are its
// registers, P^T goes back through shared memory (a key's rows side by side), and
// only the maxima and sums cross threads: the sums once a unit, the maxima when
// one has grown by more than 2^8, which a vote of the warpgroup finds out.
// (With the rows on the lanes, as sdpa_prefix_kernel has them, a row of 8 keeps a
// warp busy with 128 columns while the others idle.)
//
// The lengths are known on the device only. All units (sequence, K/V head, row
// block) in a row, each as long as its key tiles, are one line, cut into equal
// runs, one for each CTA: any mix of lengths ends at the same time on all SMs. A
// unit that a run's end cuts leaves normalised fp32 rows and their log2-sum-exps,
// at most two slots a CTA, joined by a second kernel (paged_join.cu); the others
// are written as they are.
//
// One persistent CTA an SM. Roles: a warpgroup of softmax threads (two at N = 64,
// 32 rows each), a producer warp (walks the run, tells the others its units through a
// ring, copies pages by TMA, its lanes one box of a page each), an MMA issuer.
// Rows of a tile that no query sees (behind the last key, before the window,
// in pages that are not read) may hold anything: their scores are masked, and
// their values are zeroed in shared memory, since P's zeros would not cancel them.
#pragma once
#include "common.cuh"
#include "paged.cuh"

namespace sdpa {

template <int DQK, int DV, int N>
struct PagedCfg {
  static constexpr int BN = kPagedTile;
  static constexpr int GROUPS = N == 64 ? 2 : 1;       // softmax warpgroups
  static constexpr int NC = N / GROUPS;                // rows a thread
  static constexpr int SOFT = 128 * GROUPS;            // softmax threads
  static constexpr int THREADS = SOFT + 64;
  static constexpr int K_BYTES = BN * DQK * 2;
  static constexpr int V_BYTES = BN * DV * 2;
  static constexpr int Q_BYTES = N * DQK * 2;
  static constexpr int P_PITCH = N * 2;                // bytes a key of P^T: the swizzle's width
  static constexpr int P_BYTES = BN * P_PITCH;
  static constexpr int P_BUFS = N == 64 ? 1 : 2;
  static constexpr int MISC = 1024 + SOFT / 32 * 256;  // barriers and so on; two rows of 32 floats a softmax warp
  static constexpr int Q_BUFS = Q_BYTES > 16384 ? 1 : 2;
  static constexpr int AVAIL = 227 * 1024 - 1024 - Q_BUFS * Q_BYTES - P_BUFS * P_BYTES - MISC;
  static constexpr int FIT = AVAIL / (K_BYTES + V_BYTES);
  static constexpr int ST = FIT > 6 ? 6 : FIT;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + ST * K_BYTES;
  static constexpr int OFF_Q = OFF_V + ST * V_BYTES;
  static constexpr int OFF_P = OFF_Q + Q_BUFS * Q_BYTES;
  static constexpr int OFF_MISC = OFF_P + P_BUFS * P_BYTES;
  static constexpr int SMEM = OFF_MISC + MISC + 1024;
  static constexpr uint32_t TMEM_COLS = 4 * N;
  static constexpr uint32_t T_S = 0, T_O = 2 * N;      // two tiles of each
  static_assert(ST >= 2 && SMEM <= 227 * 1024, "shared memory");
};

// Barriers: rings of K and V, Q of a unit, S and P of a tile, P V done, O of a
// unit full and read, ring of units.
enum : int { GB_KF = 0, GB_KE = GB_KF + 6, GB_VF = GB_KE + 6, GB_VE = GB_VF + 6, GB_Q = GB_VE + 6, GB_QE = GB_Q + 2,
             GB_S = GB_QE + 2, GB_P = GB_S + 2, GB_PV = GB_P + 2, GB_O = GB_PV + 2, GB_OE = GB_O + 2,
             GB_I = GB_OE + 2, GB_IE = GB_I + 4, GB_DRAIN = GB_IE + 4, GB_COUNT = GB_DRAIN + 2 };

// One unit's part of a run, as the producer tells it.
struct PagedItem {
  int n;          // key tiles (0: the sequence has no key; -1: the run's end)
  int b, hk, rb;  // sequence, K/V head, row block
  int k0;         // first key tile
  int len;        // keys of the sequence
  int slot;       // partial slot, or -1: the whole unit
};

__device__ __forceinline__ uint64_t paged_desc_p(uint32_t saddr, int pitch) {
  // rows of P^T side by side (MN-major), 8 keys an atom as wide as the swizzle
  uint64_t d = sdesc_sw128(saddr, 16, 8 * pitch);
  if (pitch < 128) d = (d & ~(uint64_t{7} << 61)) | (static_cast<uint64_t>(pitch == 64 ? 4 : 6) << 61);
  return d;
}

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Keys of a sequence, and its key tiles [lo, lo + n) that some new token sees.
struct PagedSpan {
  int len, lo, n;
};
__device__ __forceinline__ PagedSpan paged_span(const PagedParams& p, int seqlen) {
  PagedSpan s;
  s.len = min(max(seqlen, 0), p.capacity);
  const int first = p.left < 0 ? 0 : max(0, s.len - p.s_q - p.left);
  s.lo = first / kPagedTile;
  s.n = s.len > 0 ? (s.len + kPagedTile - 1) / kPagedTile - s.lo : 0;
  return s;
}

template <int DQK, int DV, bool BF16, int N>
__global__ void __launch_bounds__(PagedCfg<DQK, DV, N>::THREADS, 1)
    sdpa_paged_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PagedParams p) {
  using C = PagedCfg<DQK, DV, N>;
  constexpr int ST = C::ST, NC = C::NC, BN = C::BN;
  constexpr int kWarpsAll = C::THREADS / 32, kSoftWarps = C::SOFT / 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  const uint32_t sK = smem_u32(smem + C::OFF_K), sV = smem_u32(smem + C::OFF_V);
  const uint32_t sQ = smem_u32(smem + C::OFF_Q), sP = smem_u32(smem + C::OFF_P);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_MISC);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + GB_COUNT);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  int* start = reinterpret_cast<int*>(tmem_slot + 2);              // sequence, place in it
  uint32_t* scan = reinterpret_cast<uint32_t*>(tmem_slot + 4);     // [warps] sums
  int* items = reinterpret_cast<int*>(tmem_slot + 4 + 16);         // ring of 4, 8 words each
  static_assert((GB_COUNT + 2 + 8 + 16) * 8 <= 1024 && GB_COUNT % 2 == 0, "barrier region");
  // [softmax warps][32] values of rows. While maxima are exchanged, sMax holds each
  // warp's and sRow is its own; at a unit's end sRow holds each warp's sums and sMax is
  // its own. Between the two uses lies a barrier of the warpgroup.
  float* sMax = reinterpret_cast<float*>(smem + C::OFF_MISC + 1024);
  float* sRow = sMax + kSoftWarps * 32;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // ---- this CTA's run: [lo, hi) of the line of all units
  // thread i has the sequences [i per, (i + 1) per)
  const int per = (p.B + C::THREADS - 1) / C::THREADS;
  const int units = p.H_kv * p.row_blocks;  // of a sequence
  uint32_t sum = 0;
  for (int i = tid * per; i < min(p.B, (tid + 1) * per); ++i)
    sum += static_cast<uint32_t>(paged_span(p, __ldg(p.seqlen + i)).n + kPagedCost);
  sum *= static_cast<uint32_t>(units);
  uint32_t upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += u;
  }
  if (lane == 31) scan[warp] = upto;
  if (tid == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    for (int i = 0; i < GB_COUNT; ++i) {
      uint32_t n = 1;
      if (i >= GB_P && i < GB_P + 2) n = kSoftWarps;
      if (i >= GB_OE && i < GB_OE + 2) n = kSoftWarps;
      if (i >= GB_IE && i < GB_DRAIN) n = kSoftWarps + 1;
      mbar_init(bar(i), n);
    }
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == kSoftWarps + 1) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  // rows of Q that no box fills stay 0
  for (int i = tid; i < C::Q_BUFS * C::Q_BYTES / 16; i += C::THREADS)
    reinterpret_cast<uint4*>(smem + C::OFF_Q)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  uint32_t total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kWarpsAll; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  const uint32_t run_lo = static_cast<uint32_t>(static_cast<uint64_t>(total) * blockIdx.x / gridDim.x);
  const uint32_t run_hi = static_cast<uint32_t>(static_cast<uint64_t>(total) * (blockIdx.x + 1) / gridDim.x);
  upto += before;
  if (run_lo < run_hi && run_lo >= upto - sum && run_lo < upto) {  // one thread of the CTA
    uint32_t at = run_lo - (upto - sum);
    int i = tid * per;
    for (;; ++i) {
      const uint32_t w = static_cast<uint32_t>(paged_span(p, __ldg(p.seqlen + i)).n + kPagedCost) * units;
      if (at < w) break;
      at -= w;
    }
    start[0] = i;
    start[1] = static_cast<int>(at);
  }
  __syncthreads();
  const uint32_t tbase = *tmem_slot;
  const ErrCtx ec{p.err, abort_flag};
  auto next_item = [&](int u, PagedItem* it) -> bool {
    if (!mbar_wait_w(bar(GB_I + (u & 3)), (u >> 2) & 1, ec, kSiteFwdSoftmax)) return false;
    const int4 a = *reinterpret_cast<const int4*>(items + (u & 3) * 8);
    const int4 b = *reinterpret_cast<const int4*>(items + (u & 3) * 8 + 4);
    *it = PagedItem{a.x, a.y, a.z, a.w, b.x, b.y, b.z};
    return true;
  };

  if (warp == kSoftWarps) {
    // ------------------------------------------------------------ producer
    int nk = 0, nv = 0, nu = 0, nq = 0;  // tiles of K and V, items, items with keys so far
    bool ok = true;
    int4 runs = make_int4(0, 0, 0, 0);
    auto tell = [&](const PagedItem& it) -> bool {
      if (!__all_sync(0xffffffffu,
                      mbar_wait(bar(GB_IE + (nu & 3)), ((nu >> 2) & 1) ^ 1, ec, kSiteFwdLoad, true, true)))
        return false;
      if (lane == 0) {
        *reinterpret_cast<int4*>(items + (nu & 3) * 8) = make_int4(it.n, it.b, it.hk, it.rb);
        *reinterpret_cast<int4*>(items + (nu & 3) * 8 + 4) = make_int4(it.k0, it.len, it.slot, 0);
        mbar_arrive(bar(GB_I + (nu & 3)));
      }
      __syncwarp();
      ++nu;
      return true;
    };
    uint32_t left = run_hi - run_lo;
    int i = 0, unit = 0, pos = 0;
    PagedSpan sp{0, 0, 0};
    if (left > 0) {
      i = start[0];
      sp = paged_span(p, __ldg(p.seqlen + i));
      const int w = sp.n + kPagedCost;
      unit = start[1] / w;
      pos = start[1] - unit * w;
    }
    while (left > 0) {
      const int w = sp.n + kPagedCost;
      const int take = static_cast<int>(min(left, static_cast<uint32_t>(w - pos)));
      const int t0 = max(pos - kPagedCost, 0), t1 = max(pos + take - kPagedCost, 0);
      const bool none = sp.n == 0 && pos == 0;
      if (t1 > t0 || none) {
        PagedItem it;
        it.n = t1 - t0;
        it.b = i;
        it.hk = unit / p.row_blocks;
        it.rb = unit - it.hk * p.row_blocks;
        it.k0 = sp.lo + t0;
        it.len = sp.len;
        it.slot = -1;
        const int id = i * units + unit + 1;
        if (t0 > 0) {
          it.slot = 2 * blockIdx.x;
          runs.x = id;
          runs.y = t1 == sp.n;
        } else if (t1 < sp.n) {
          it.slot = 2 * blockIdx.x + 1;
          runs.z = id;
        }
        if (!(ok = tell(it))) break;
        if (it.n > 0) {
          const int qb = nq % C::Q_BUFS;
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(GB_QE + qb), ((nq / C::Q_BUFS) & 1) ^ 1, ec, kSiteFwdLoad, true,
                                                       true))))
            break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(GB_Q + qb), (DQK / 64) * p.q_box);
#pragma unroll
            for (int c = 0; c < DQK / 64; ++c)
              tma_load_4d(sQ + qb * C::Q_BYTES + c * N * 128, &tmQ, bar(GB_Q + qb), c * 64, it.rb * N, it.b, it.hk);
          }
          ++nq;
          // Keys that some token sees: [seen, len). A tile's copies are boxes of a page,
          // of `box` keys each; lane l has the page of box b0 + l.
          const int seen = p.left < 0 ? 0 : max(0, sp.len - p.s_q - p.left);
          const int per_tile = BN >> p.box_shift;
          const int* row = p.table + i * p.table_stride;
          auto page_of = [&](int box) {
            const int key = box << p.box_shift;
            const int id = key < sp.len ? __ldg(row + (key >> p.page_shift)) : 0;
            // (the first page behind the pool reads as zeros)
            return static_cast<uint32_t>(id) < static_cast<uint32_t>(p.n_pages) ? id : p.n_pages;
          };
          int b0 = it.k0 * per_tile;
          int ids = page_of(b0 + lane), ahead = page_of(b0 + 32 + lane);
          for (int j = 0; j < it.n; ++j) {
            const int box0 = (it.k0 + j) * per_tile;
            if (box0 - b0 == 32) {
              b0 = box0;
              ids = ahead;
              ahead = page_of(b0 + 32 + lane);
            }
            const int s = nk % ST;
            const uint32_t ph = static_cast<uint32_t>(nk / ST) & 1u;
            // boxes of the tile with a visible key
            const int lo = max(box0, seen >> p.box_shift);
            const int hi = min(box0 + per_tile, (sp.len + p.box - 1) >> p.box_shift);
            const uint32_t bytes = static_cast<uint32_t>(hi - lo) * static_cast<uint32_t>(p.box) * 128u;
            // lane l copies column chunk l / per_tile (and further ones) of box l % per_tile
            const int my_box = box0 + (lane & (per_tile - 1));
            const int pg = __shfl_sync(0xffffffffu, ids, my_box - b0);
            const bool mine = my_box >= lo && my_box < hi;
            const int key = my_box << p.box_shift, in_page = key & ((1 << p.page_shift) - 1);
            const uint32_t dst = static_cast<uint32_t>(key - box0 * p.box) * 128u;
            auto copy = [&](int chunks, uint32_t base, const CUtensorMap* m, uint32_t b) {
              if (lane == 0) mbar_arrive_expect_tx(b, bytes * chunks);
              __syncwarp();
              if (mine)
                for (int c = lane / per_tile; c < chunks; c += 32 / per_tile)
                  tma_load_4d(base + c * BN * 128 + dst, m, b, c * 64, in_page, it.hk, pg);
              __syncwarp();
            };
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(GB_KE + s), ph ^ 1, ec, kSiteFwdLoad, true, true)))) break;
            copy(DQK / 64, sK + s * C::K_BYTES, &tmK, bar(GB_KF + s));
            ++nk;
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(GB_VE + s), ph ^ 1, ec, kSiteFwdLoad, true, true)))) break;
            copy(DV / 64, sV + s * C::V_BYTES, &tmV, bar(GB_VF + s));
            ++nv;
          }
          if (!ok) break;
        }
      }
      left -= static_cast<uint32_t>(take);
      pos = 0;
      if (++unit == units && left > 0) {
        unit = 0;
        ++i;
        sp = paged_span(p, __ldg(p.seqlen + i));
      }
    }
    if (ok) tell(PagedItem{-1, 0, 0, 0, 0, 0, 0});
    if (lane == 0) p.runs[blockIdx.x] = runs;
    // Every copy issued must land before the CTA can retire; on the healthy path they
    // did long ago.
    __syncwarp();
    if (*abort_flag) {
      for (int b = 0; b < C::Q_BUFS; ++b)
        if (nq > b) mbar_wait(bar(GB_Q + b), ((nq - 1 - b) / C::Q_BUFS) & 1, ec, kSiteDrain, false);
      for (int s = 0; s < ST; ++s) {
        if (nk > s) mbar_wait(bar(GB_KF + s), ((nk - 1 - s) / ST) & 1, ec, kSiteDrain, false);
        if (nv > s) mbar_wait(bar(GB_VF + s), ((nv - 1 - s) / ST) & 1, ec, kSiteDrain, false);
      }
    }
  } else if (warp == kSoftWarps + 1) {
    // ---------------------------------------------------------- MMA issuer
    constexpr uint32_t kIdS = idesc_f16(128, N, BF16, false, false);
    constexpr uint32_t kIdO = idesc_f16(DV, N, BF16, true, true);
    const uint64_t dK0 = sdesc_sw128(sK, 16, 1024);
    const uint64_t dQ0 = sdesc_sw128(sQ, 16, 1024);
    const uint64_t dV0 = sdesc_sw128(sV, BN * 128, 1024);
    const uint64_t dP0 = paged_desc_p(sP, C::P_PITCH);
    int u = 0, g = 0, q = 0;  // item, key tile, item with keys
    bool ok = true;
    // S of tile g, the j-th of an item of n
    auto issue_s = [&](int gs, int qs, bool first, bool last) -> bool {
      if (first && !mbar_wait_w(bar(GB_Q + qs % C::Q_BUFS), (qs / C::Q_BUFS) & 1, ec, kSiteFwdMma)) return false;
      if (!mbar_wait_w(bar(GB_KF + gs % ST), (gs / ST) & 1, ec, kSiteFwdMma)) return false;
      tc_fence_after();
      const uint64_t dK = opaque_u64(desc_adv(dK0, (gs % ST) * C::K_BYTES));
      const uint64_t dQ = opaque_u64(desc_adv(dQ0, (qs % C::Q_BUFS) * C::Q_BYTES));
#pragma unroll
      for (int kk = 0; kk < DQK / 16; ++kk)
        umma_ss_w(tbase + C::T_S + N * (gs & 1), desc_adv(dK, (kk >> 2) * (BN * 128) + (kk & 3) * 32),
                  desc_adv(dQ, (kk >> 2) * (N * 128) + (kk & 3) * 32), kIdS, kk > 0);
      umma_commit_w(bar(GB_S + (gs & 1)));
      umma_commit_w(bar(GB_KE + gs % ST));
      if (last) umma_commit_w(bar(GB_QE + qs % C::Q_BUFS));
      return true;
    };
    auto issue_pv = [&](int gv, int qv, bool first, bool last) -> bool {
      const int ob = qv & 1;
      // O's buffer has been read (of the item before the last one)
      if (first && !mbar_wait_w(bar(GB_OE + ob), ((qv >> 1) & 1) ^ 1, ec, kSiteFwdMma)) return false;
      if (!mbar_wait_w(bar(GB_VF + gv % ST), (gv / ST) & 1, ec, kSiteFwdMma)) return false;
      if (!mbar_wait_w(bar(GB_P + (gv & 1)), (gv >> 1) & 1, ec, kSiteFwdMma)) return false;
      tc_fence_after();
      const uint64_t dV = opaque_u64(desc_adv(dV0, (gv % ST) * C::V_BYTES));
      const uint64_t dP = opaque_u64(desc_adv(dP0, (C::P_BUFS == 2 ? (gv & 1) : 0) * C::P_BYTES));
#pragma unroll
      for (int kk = 0; kk < BN / 16; ++kk)
        umma_ss_w(tbase + C::T_O + N * ob, desc_adv(dV, kk * 2048), desc_adv(dP, kk * 16 * C::P_PITCH), kIdO,
                  !first || kk > 0);
      umma_commit_w(bar(GB_VE + gv % ST));
      umma_commit_w(bar(GB_PV + (gv & 1)));
      if (last) umma_commit_w(bar(GB_O + ob));
      return true;
    };
    for (;; ++u) {
      PagedItem it;
      if (!(ok = next_item(u, &it))) break;
      if (it.n >= 0) {
        if (it.n > 0) ok = issue_s(g, q, true, it.n == 1);
        for (int j = 0; ok && j < it.n; ++j, ++g) {
          // the next tile's S first, if its keys are there: it runs while the softmax does
          const bool more = j + 1 < it.n;
          const bool early =
              more && __all_sync(0xffffffffu, mbar_try_wait(bar(GB_KF + (g + 1) % ST), ((g + 1) / ST) & 1));
          if (early) ok = issue_s(g + 1, q, false, j + 2 == it.n);
          if (ok) ok = issue_pv(g, q, j == 0, !more);
          if (ok && more && !early) ok = issue_s(g + 1, q, false, j + 2 == it.n);
        }
        if (it.n > 0) ++q;
      }
      if (!ok) break;
      if (lane == 0) mbar_arrive(bar(GB_IE + (u & 3)));
      __syncwarp();
      if (it.n < 0) break;
    }
    umma_commit_w(bar(GB_DRAIN));
    mbar_wait(bar(GB_DRAIN), 0, ec, kSiteDrain, false);
  } else {
    // -------------------------------------------------------------- softmax
    const int t = warp >> 2, w4 = warp & 3;
    const int col0 = t * NC;            // first row of this warpgroup
    const int own_key = w4 * 32 + lane;  // this thread's key of a tile
    const uint32_t tS = tbase + C::T_S + col0 + (static_cast<uint32_t>(w4 * 32) << 16);
    const uint32_t tO = tbase + C::T_O + col0 + (static_cast<uint32_t>(w4 * 32) << 16);
    float* gMax = sMax + t * 128;
    float* gRow = sRow + t * 128;
    float* wMax = gMax + w4 * 32;
    float* wRow = gRow + w4 * 32;
    const float sl2 = p.scale_log2;
    const float hide = sl2 < 0.f ? -SDPA_NEG_INF : SDPA_NEG_INF;  // masked raw score
    // 16-byte chunk of a key's row of P^T, as the swizzle has it
    const int flip = C::P_PITCH == 128 ? own_key & 7 : C::P_PITCH == 64 ? (own_key >> 1) & 3 : (own_key >> 2) & 1;
    uint8_t* own_p = smem + C::OFF_P + own_key * C::P_PITCH;
    // A vote of the warpgroup. A warp whose wait ran out votes no until all leave
    // together: after a no comes a second vote, on whether all are well.
    auto vote = [&](bool yes) { return named_bar_and(1 + t, 128, yes); };
    auto load = [&](uint32_t at, float (&x)[NC]) {
      if constexpr (NC == 32) {
        tmem_ld32f(at, x);
      } else {
        uint32_t r[16];
        tmem_ld16(at, r);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(r[e]);
      }
      tmem_wait_ld();
    };
    auto spread = [&](float* own, float v, float (&x)[NC]) {  // lane e's value of row e to all lanes
      __syncwarp();
      if (lane < NC) own[lane] = v;
      __syncwarp();
#pragma unroll
      for (int e = 0; e < NC; e += 4) {
        const float4 f = *reinterpret_cast<const float4*>(own + e);
        x[e] = f.x, x[e + 1] = f.y, x[e + 2] = f.z, x[e + 3] = f.w;
      }
    };
    constexpr float kNone = 1e30f;  // -m of a row without a score: any score then grows it
    int u = 0, g = 0, q = 0;
    bool ok = true, left_all = false;
    PagedItem it;
    for (; (ok = next_item(u, &it)) && it.n >= 0; ++u) {
      const int base = it.rb * N + col0;  // of the K/V head's rows
      const int live = min(NC, p.R - base);
      const int64_t row0 = (static_cast<int64_t>(it.b) * p.H_kv + it.hk) * p.R + base;
      if (it.n == 0) {  // a sequence without a key
        for (int e = w4; e < live; e += 4) {
          for (int d = lane; d < DV / 2; d += 32) static_cast<uint32_t*>(p.o)[(row0 + e) * (DV / 2) + d] = 0u;
          if (lane == 0) p.lse[row0 + e] = SDPA_NEG_INF;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(GB_IE + (u & 3)));
        continue;
      }
      const int last0 = it.len - p.s_q;  // last key of token 0
      const int seen = p.left < 0 ? 0 : max(0, last0 - p.left);  // first key of token 0
      float nm[NC], l[NC], m = SDPA_NEG_INF;  // (m: row `lane`)
#pragma unroll
      for (int e = 0; e < NC; ++e) {
        nm[e] = kNone;
        l[e] = 0.f;
      }
      for (int j = 0; j < it.n; ++j, ++g) {
        const int key0 = (it.k0 + j) * BN, key = key0 + own_key;
        if (ok) ok = mbar_wait(bar(GB_S + (g & 1)), (g >> 1) & 1, ec, kSiteFwdSoftmax);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        float x[NC];
        load(tS + N * (g & 1), x);
        if (p.capped) {
#pragma unroll
          for (int e = 0; e < NC; ++e) x[e] = rcp(1.f + ex2(x[e] * p.cap_in));
        }
        if (key0 + BN - 1 > last0 || (p.left >= 0 && key0 < last0 + p.s_q - 1 - p.left)) {
          int tok = base % p.s_q;
#pragma unroll
          for (int e = 0; e < NC; ++e) {
            if (key > last0 + tok || (p.left >= 0 && key < last0 + tok - p.left)) x[e] = hide;
            tok = tok + 1 == p.s_q ? 0 : tok + 1;
          }
        }
        float most = SDPA_NEG_INF;
#pragma unroll
        for (int e = 0; e < NC; ++e) most = fmaxf(most, fmaf(x[e], sl2, nm[e]));
        if (!vote(ok && !(most > 8.f))) {
          // ---- some row's maximum has grown: exchange them
          float mine = SDPA_NEG_INF;
#pragma unroll
          for (int e = 0; e < NC; ++e) {
            const float r = warp_max(x[e] * sl2);
            if (lane == e) mine = r;
          }
          wMax[lane] = mine;
          if (!vote(ok)) {
            left_all = true;
            break;
          }
          const int e0 = lane & (NC - 1);
          const float mx = fmaxf(fmaxf(gMax[e0], gMax[32 + e0]), fmaxf(gMax[64 + e0], gMax[96 + e0]));
          float alpha = 1.f;
          if (mx > m + 8.f) {
            alpha = ex2(m - mx);
            m = mx;
          }
          spread(wRow, m == SDPA_NEG_INF ? kNone : -m, nm);
          float al[NC];
          spread(wRow, alpha, al);
#pragma unroll
          for (int e = 0; e < NC; ++e) l[e] *= al[e];
          if (j > 0) {
            if (ok) ok = mbar_wait(bar(GB_PV + ((g - 1) & 1)), ((g - 1) >> 1) & 1, ec, kSiteFwdSoftmax);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            float o[NC];
            load(tO + N * (q & 1), o);
#pragma unroll
            for (int e0 = 0; e0 < NC; e0 += 16) {
              uint32_t r[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(o[e0 + e] * al[e0 + e]);
              tmem_st16(tO + N * (q & 1) + e0, r);
            }
            tmem_wait_st();
          }
        }
#pragma unroll
        for (int e = 0; e < NC; ++e) {
          x[e] = ex2(fmaf(x[e], sl2, nm[e]));
          l[e] += x[e];
        }
        // P's buffer: the product that read it last is done
        if (ok) {
          if constexpr (C::P_BUFS == 2)
            ok = mbar_wait(bar(GB_PV + (g & 1)), ((g >> 1) & 1) ^ 1, ec, kSiteFwdSoftmax);
          else if (g > 0)
            ok = mbar_wait(bar(GB_PV + ((g - 1) & 1)), ((g - 1) >> 1) & 1, ec, kSiteFwdSoftmax);
        }
        uint8_t* to = own_p + (C::P_BUFS == 2 ? (g & 1) : 0) * C::P_BYTES;
#pragma unroll
        for (int e = 0; e < NC; e += 8)
          *reinterpret_cast<uint4*>(to + (((col0 + e) / 8) ^ flip) * 16) =
              make_uint4(pack2<BF16>(x[e], x[e + 1]), pack2<BF16>(x[e + 2], x[e + 3]),
                         pack2<BF16>(x[e + 4], x[e + 5]), pack2<BF16>(x[e + 6], x[e + 7]));
        // values of keys that no row sees
        const int front = min(BN, max(0, seen - key0)), back = min(BN, it.len - key0);
        if (front > 0 || back < BN) {
          if (ok) ok = mbar_wait(bar(GB_VF + g % ST), (g / ST) & 1, ec, kSiteFwdSoftmax);
          uint8_t* v = smem + C::OFF_V + (g % ST) * C::V_BYTES;
          for (int e = tid; e < (front + BN - back) * 8; e += C::SOFT) {
            const int r = e / 8 < front ? e / 8 : e / 8 - front + back;
#pragma unroll
            for (int c = 0; c < DV / 64; ++c)
              *reinterpret_cast<uint4*>(v + c * BN * 128 + r * 128 + (e & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(GB_P + (g & 1)));
      }
      if (left_all) break;
      // ---- the unit's rows: O / l, and the log of the sum of exponentials
      // sums over the warp's keys: lane e gets row e's
#pragma unroll
      for (int o = NC / 2; o > 0; o >>= 1) {
        const bool hi = (lane & o) != 0;
#pragma unroll
        for (int e = 0; e < o; ++e) {
          const float send = hi ? l[e] : l[e + o], keep = hi ? l[e + o] : l[e];
          l[e] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
      }
      if constexpr (NC == 16) l[0] += __shfl_xor_sync(0xffffffffu, l[0], 16);
      __syncwarp();
      wRow[lane] = l[0];
      if (!vote(ok)) {
        vote(false);
        left_all = true;
        break;
      }
      const int e0 = lane & (NC - 1);
      const float sum_l = (gRow[e0] + gRow[32 + e0]) + (gRow[64 + e0] + gRow[96 + e0]);
      float inv[NC];
      spread(wMax, sum_l == 0.f ? 0.f : 1.f / sum_l, inv);
      const float log_l = sum_l == 0.f ? SDPA_NEG_INF : m + __log2f(sum_l) + p.lse_shift;
      if (w4 == 0 && lane < live) {
        if (it.slot < 0)
          p.lse[row0 + lane] = log_l * kLn2;
        else
          p.part_lse[it.slot * N + col0 + lane] = log_l;
      }
      ok = mbar_wait_w(bar(GB_O + (q & 1)), (q >> 1) & 1, ec, kSiteFwdSoftmax);
      tc_fence_after();
      float o[NC];
      load(tO + N * (q & 1), o);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(GB_OE + (q & 1)));
        mbar_arrive(bar(GB_IE + (u & 3)));
      }
      // (64 value columns: the product's rows lie on each warp's first 16 lanes)
      const int d = DV == 128 ? own_key : w4 * 16 + lane;
      const bool has = DV == 128 || lane < 16;
#pragma unroll
      for (int e = 0; e < NC; ++e) o[e] = inv[e] == 0.f ? 0.f : o[e] * inv[e];
      if (it.slot >= 0) {
        float* dst = p.part + static_cast<int64_t>(it.slot * N + col0) * DV + d;
#pragma unroll
        for (int e = 0; e < NC; ++e)
          if (has && e < live) dst[e * DV] = o[e];
      } else {
        // two rows at a time: neighbouring lanes swap, and store two columns of a row each
        const bool odd = (lane & 1) != 0;
        uint32_t* dst = static_cast<uint32_t*>(p.o) + row0 * (DV / 2) + d / 2;
#pragma unroll
        for (int e = 0; e < NC; e += 2) {
          const float other = __shfl_xor_sync(0xffffffffu, odd ? o[e] : o[e + 1], 1);
          const uint32_t two = odd ? pack2<BF16>(other, o[e + 1]) : pack2<BF16>(o[e], other);
          if (has && e + (odd ? 1 : 0) < live) dst[(e + (odd ? 1 : 0)) * (DV / 2)] = two;
        }
      }
      ++q;
    }
    if (!left_all && !vote(ok)) vote(false);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kSoftWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tbase, C::TMEM_COLS);
  }
}

template <int DQK, int DV, bool BF16, int N>
cudaError_t launch_paged_n(const CUtensorMap (&m)[3], const PagedParams& p, cudaStream_t st) {
  using C = PagedCfg<DQK, DV, N>;
  auto kern = sdpa_paged_kernel<DQK, DV, BF16, N>;
  const cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(kern), C::SMEM, 0);
  if (e != cudaSuccess) return e;
  kern<<<p.grid, C::THREADS, C::SMEM, st>>>(m[0], m[1], m[2], p);
  return cudaGetLastError();
}

template <int DQK, int DV, bool BF16>
cudaError_t launch_paged_d(const CUtensorMap (&m)[3], const PagedParams& p, cudaStream_t st) {
  switch (paged_rows(p.R)) {
    case 16: return launch_paged_n<DQK, DV, BF16, 16>(m, p, st);
    case 32: return launch_paged_n<DQK, DV, BF16, 32>(m, p, st);
    default: return launch_paged_n<DQK, DV, BF16, 64>(m, p, st);
  }
}

}  // namespace sdpa
