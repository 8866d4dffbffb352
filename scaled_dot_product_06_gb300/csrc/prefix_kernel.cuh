// Attention of new tokens over a prefix that their whole batch shares and the
// keys of their own that each sequence has after it (sm_103a).
//
// For the rows x of K/V head hk (R = (h / h_kv) * s_q of them a sequence:
// query heads of the group times new tokens),
//   S = scale Q K^T (capped: softcap tanh(S / softcap)), P = softmax(S), O = P V
// over two key sets: the prefix, the same for all sequences, and the first
// seqlen[b] rows of the sequence's own cache, of which token t sees those up to
// seqlen[b] - s_q + t. The two are read separately: against the prefix all
// sequences' rows of a K/V head are one matrix of b * R rows, so that its keys
// and values are read once for the batch and the products fill tcgen05 tiles;
// the own keys are a stream of their own per sequence. Both are cut along the
// keys into work items; an item leaves normalised fp32 rows O_s and their
// log2-sum-exps L_s, and a second kernel joins them (prefix_join.cu):
//   L = log2 sum_s 2^L_s,   O = sum_s 2^(L_s - L) O_s.
// Items are handed out as CTAs ask for them, since the lengths are known on the
// device only: the producer takes a number from a counter, one ahead, and
// tells it to the other roles through a ring in shared memory. Which CTA has an
// item does not change its result.
//
// Measured (b64 h32 kv4 d128 bf16 behind 16384 keys, own lengths up to 1024, cap
// 50): 50 us, and 6.4 us the join, for 17 us of bytes and 9 us of products: the
// start (5 us), filling and emptying the pipeline at each item's ends (about 2 us)
// and the items' grain are the rest. Whole calls without a cap: own keys alone, 152
// sequences of 4096 keys, 61 us (5.2 TB/s); a prefix of 131072 for 512 rows of each
// of 4 K/V heads, 105 us (1.3 PFLOP/s). Equal runs of visits for each CTA instead of
// items (a stream cut at any tile, more partials, every row block's borders found by
// a scan of the lengths) took 51 us where the first form of this kernel took 41.
//
// One persistent CTA an SM, two softmax warpgroups, one MMA issuer, one TMA
// producer, as in the forward (fwd_kernel.cuh). An item runs in one of two
// ways:
//   dual    (more than 128 rows, d_qk up to 128) warpgroup t has the rows of tile t; both tiles
//           meet every key tile, which is loaded once for them;
//   single  (up to 128 rows: a decoding step's own keys, where the K/V stream
//           from memory is the limit) both warpgroups have the same rows and take
//           the item's key tiles in turns, each with its own running maximum,
//           sum and O in tensor memory, and each leaves a partial of its own;
//           one's softmax hides behind the other's products. Own keys of up to
//           32 rows go a step further (quart): Q lies four times in its tile, once
//           for each warp's lanes, and a warp takes a quarter of a tile's keys, P
//           of the others being 0: a warp alone with 128 columns of 8 rows would
//           be what the stream waits for. Each warp leaves a partial. (64
//           sequences of 512 own keys, 4 K/V heads: 21.1 us for 22.5 at 8 rows, 28.0
//           for 26.0 at 32 rows; with a cap 22.2 for 27.0, and 29.0 for 30.4.)
// MMA order per round: O_0 += P_0 V, S_0 of the next round, then the same for
// warpgroup 1.
#pragma once
#include <type_traits>

#include "common.cuh"
#include "prefix.cuh"

namespace sdpa {

template <int DQK, int DV>
struct PrefixCfg {
  static constexpr int BM = 128, BN = 128;
  static constexpr int Q_BYTES = BM * DQK * 2;
  static constexpr int K_BYTES = BN * DQK * 2;
  static constexpr int V_BYTES = BN * DV * 2;
  static constexpr int BAR_BYTES = 384;
  static constexpr int Q_TILES = DQK <= kPrefixDualMax ? 2 : 1;
  static constexpr int AVAIL = 227 * 1024 - Q_TILES * Q_BYTES - BAR_BYTES - 1024;
  static constexpr int FIT = AVAIL / (K_BYTES + V_BYTES);
  static constexpr int STAGES = FIT >= 4 ? 4 : FIT;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + Q_TILES * Q_BYTES;
  static constexpr int OFF_V = OFF_K + STAGES * K_BYTES;
  static constexpr int OFF_BAR = OFF_V + STAGES * V_BYTES;
  static constexpr int SMEM = OFF_BAR + BAR_BYTES + 1024;
  static constexpr int THREADS = 384;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t T_S = 0, T_O = 256;
  static constexpr int REG_LAUNCH = 168, REG_SOFTMAX = 216, REG_OTHER = 72;
  static_assert(STAGES >= 1 && SMEM <= 227 * 1024, "shared memory");
  static_assert(2 * 128 * REG_SOFTMAX + 128 * REG_OTHER == THREADS * REG_LAUNCH, "register split");
};

// Barriers: Q full and free, S / P / O per warpgroup, V landed (for the
// warpgroup that clears its rows behind the last key), rings of K and V, ring
// of item numbers.
enum : int { PB_Q = 0, PB_QE, PB_S, PB_P = PB_S + 2, PB_O = PB_P + 2, PB_VZ = PB_O + 2, PB_DRAIN = PB_VZ + 2, PB_KF,
             PB_KE = PB_KF + 4, PB_VF = PB_KE + 4, PB_VE = PB_VF + 4,
             PB_I = PB_VE + 4, PB_IE = PB_I + 4, PB_COUNT = PB_IE + 4 };

// One work item, decoded alike by every role.
struct PrefixItem {
  bool own;     // own keys (else the prefix)
  int hk, b;    // K/V head; sequence (own keys)
  int tile;     // first row tile
  bool has1;    // dual: the second row tile exists
  bool dual;
  bool quart;   // rows repeated for each warp's lanes, which take a quarter of the keys
  int k0, n;    // first key tile, key tiles (0: nothing to do)
  int keys;     // keys of the source
  int slot;     // partial slot of warpgroup 0 (single: warpgroup 1 has the next)
};

__device__ __forceinline__ PrefixItem prefix_item(const PrefixParams& p, int idx) {
  PrefixItem it;
  it.own = idx >= p.items_prefix;
  if (!it.own) {
    // row blocks of one key range next to one another: they share its keys in L2
    const int rb = idx % p.row_blocks_p;
    const int r = idx / p.row_blocks_p;
    const int sp = r % p.splits_p;
    it.hk = r / p.splits_p;
    it.b = 0;
    it.dual = p.dual_p != 0;
    it.tile = it.dual ? 2 * rb : rb;
    it.has1 = it.dual && it.tile + 1 < p.row_tiles_p;
    it.keys = p.s_prefix;
    it.k0 = sp * p.chunk_p;
    it.n = min(p.chunk_p, (it.keys + 127) / 128 - it.k0);
    it.quart = false;
    it.slot = it.dual ? sp : 2 * sp;
  } else {
    idx -= p.items_prefix;
    const int rb = idx % p.row_blocks_o;
    int r = idx / p.row_blocks_o;
    const int z = r % (p.B * p.H_kv);  // cache plane
    const int sp = r / (p.B * p.H_kv);
    it.b = z / p.H_kv;
    it.hk = z - it.b * p.H_kv;
    it.dual = p.dual_o != 0;
    it.tile = it.dual ? 2 * rb : rb;
    it.has1 = it.dual && it.tile + 1 < p.row_tiles_o;
    it.keys = min(max(__ldg(p.seqlen + it.b), 0), p.s_max);
    it.k0 = sp * p.chunk_o;
    it.n = max(0, min(p.chunk_o, (it.keys + 127) / 128 - it.k0));
    it.quart = p.quart_o != 0;
    it.slot = p.slots_p + (it.dual ? sp : it.quart ? 8 * sp : 2 * sp);
  }
  return it;
}

// Key tiles warpgroup t meets in round i: dual: tile i; single: tile 2 i + t.
__device__ __forceinline__ int prefix_tile(const PrefixItem& it, int t, int i) {
  return it.dual ? i : 2 * i + t;
}
// Whether warpgroup t clears the rows of key tile j's V behind the sequence's
// last key. They hold whatever the cache held before, NaN perhaps, and P's
// zeros would not cancel that. (The prefix's tensor map ends with its keys.)
__device__ __forceinline__ bool prefix_clears(const PrefixItem& it, int t, int j) {
  return it.own && (it.k0 + j + 1) * 128 > it.keys && (t == 0 || !it.dual);
}
__device__ __forceinline__ bool prefix_has(const PrefixItem& it, int t, int i) {
  return prefix_tile(it, t, i) < it.n && (t == 0 || !it.dual || it.has1);
}

template <int DQK, int DV, bool BF16, bool CAP>
__global__ void __launch_bounds__(384, 1)
    sdpa_prefix_kernel(const __grid_constant__ CUtensorMap tmQp, const __grid_constant__ CUtensorMap tmQo,
                       const __grid_constant__ CUtensorMap tmKp, const __grid_constant__ CUtensorMap tmVp,
                       const __grid_constant__ CUtensorMap tmKo, const __grid_constant__ CUtensorMap tmVo,
                       const PrefixParams p) {
  using C = PrefixCfg<DQK, DV>;
  constexpr int ST = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  const uint32_t sQ = smem_u32(smem + C::OFF_Q);
  const uint32_t sK = smem_u32(smem + C::OFF_K);
  const uint32_t sV = smem_u32(smem + C::OFF_V);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + PB_COUNT);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  volatile int* items = reinterpret_cast<volatile int*>(tmem_slot + 2);  // ring of 4
  static_assert((PB_COUNT + 3) * 8 <= C::BAR_BYTES, "barrier region");
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    if (p.items_prefix > 0) {
      tma_prefetch_desc(&tmQp);
      tma_prefetch_desc(&tmKp);
      tma_prefetch_desc(&tmVp);
    }
    if (p.items_own > 0) {
      tma_prefetch_desc(&tmQo);
      tma_prefetch_desc(&tmKo);
      tma_prefetch_desc(&tmVo);
    }
    // (a number is read by the MMA issuer and the eight softmax warps)
    for (int i = 0; i < PB_COUNT; ++i) mbar_init(bar(i), (i == PB_P || i == PB_P + 1) ? 128u : i >= PB_IE ? 9u : 1u);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  const ErrCtx ec{p.err, abort_flag};
  const int n_items = p.items_prefix + p.items_own;
  // The `u`-th item of this CTA (n_items: no more). Where there are more items
  // than CTAs the producer tells it; else each has one (which may be empty).
  auto next_item = [&](int u, int* idx) -> bool {
    if (p.next == nullptr) {
      *idx = u == 0 ? static_cast<int>(blockIdx.x) : n_items;
      return true;
    }
    if (!mbar_wait(bar(PB_I + (u & 3)), (u >> 2) & 1, ec, kSiteFwdSoftmax)) return false;
    *idx = items[u & 3];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(PB_IE + (u & 3)));
    return true;
  };

  if (warp >= 8) {
    setmaxnreg_dec<C::REG_OTHER>();
    if (warp == 8) {
      // ---------------------------------------------------------- producer
      int nq = 0;          // items loaded
      int nk = 0, nv = 0;  // key tiles loaded
      bool ok = true;
      int idx = blockIdx.x, ahead = 0;
      // (launched while the kernel that clears the counter runs)
      if (p.next != nullptr) asm volatile("griddepcontrol.wait;" ::: "memory");
      for (;; idx = __shfl_sync(0xffffffffu, ahead, 0)) {
        // the number after this one, asked for now and looked at afterwards
        ahead = n_items;
        if (lane == 0 && idx < n_items && p.next != nullptr)
          ahead = static_cast<int>(gridDim.x) + atomicAdd(p.next, 1);
        PrefixItem it;
        if (idx < n_items) it = prefix_item(p, idx);
        if (idx < n_items && it.n == 0) continue;
        if (p.next != nullptr) {
          if (!(ok = mbar_wait(bar(PB_IE + (nq & 3)), ((nq >> 2) & 1) ^ 1, ec, kSiteFwdLoad, true, true))) break;
          if (lane == 0) {
            items[nq & 3] = idx;
            mbar_arrive(bar(PB_I + (nq & 3)));
          }
          __syncwarp();
        }
        if (idx >= n_items) break;
        const CUtensorMap* mk = it.own ? &tmKo : &tmKp;
        const CUtensorMap* mv = it.own ? &tmVo : &tmVp;
        const int z = it.own ? it.b * p.H_kv + it.hk : it.hk;
        for (int j = 0; j < it.n; ++j) {
          const int s = nk % ST;
          const uint32_t ph = (nk / ST) & 1;
          const int row = (it.k0 + j) * C::BN;
          if (!(ok = mbar_wait(bar(PB_KE + s), ph ^ 1, ec, kSiteFwdLoad, true, true))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(PB_KF + s), C::K_BYTES);
#pragma unroll
            for (int c = 0; c < DQK / 64; ++c)
              tma_load_3d(sK + s * C::K_BYTES + c * C::BN * 128, mk, bar(PB_KF + s), c * 64, row, z);
          }
          ++nk;
          if (j == 0) {  // the item's Q, behind its first keys: they need not wait for Q's buffer
            if (!(ok = mbar_wait(bar(PB_QE), (nq & 1) ^ 1, ec, kSiteFwdLoad, true, true))) break;
            if (lane == 0) {
              const CUtensorMap* mq = it.own ? &tmQo : &tmQp;
              const uint32_t box = it.own ? p.q_box_o : p.q_box_p;  // bytes a 64-column box
              mbar_arrive_expect_tx(bar(PB_Q), (it.has1 ? 2 : it.quart ? 4 : 1) * (DQK / 64) * box);
              if (it.quart) {
#pragma unroll 1
                for (int w = 1; w < 4; ++w)
                  for (int c = 0; c < DQK / 64; ++c)
                    tma_load_4d(sQ + c * C::BM * 128 + w * 32 * 128, mq, bar(PB_Q), c * 64, 0, it.b, it.hk);
              }
#pragma unroll 1
              for (int t = 0; t < (it.has1 ? 2 : 1); ++t) {
                // rows of row tile `tile`: whole sequences' R rows each (R <= 128), else
                // 128 rows of one sequence
                int x0, b0;
                if (p.R <= 128) {
                  x0 = 0;
                  b0 = it.own ? it.b : (it.tile + t) * p.seqs_tile;
                } else {
                  const int per = (p.R + 127) / 128;
                  b0 = it.own ? it.b : (it.tile + t) / per;
                  x0 = (it.own ? it.tile + t : (it.tile + t) % per) * 128;
                }
                for (int c = 0; c < DQK / 64; ++c)
                  tma_load_4d(sQ + t * C::Q_BYTES + c * C::BM * 128, mq, bar(PB_Q), c * 64, x0, b0, it.hk);
              }
            }
            ++nq;
          }
          if (!(ok = mbar_wait(bar(PB_VE + s), ph ^ 1, ec, kSiteFwdLoad, true, true))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(PB_VF + s), C::V_BYTES);
#pragma unroll
            for (int c = 0; c < DV / 64; ++c)
              tma_load_3d(sV + s * C::V_BYTES + c * C::BN * 128, mv, bar(PB_VF + s), c * 64, row, z);
          }
          ++nv;
        }
        if (!ok) break;
      }
      __syncwarp();
      // Every copy issued must land before the CTA can retire; on the healthy
      // path they did long ago.
      if (*abort_flag) {
        if (nq > 0) mbar_wait(bar(PB_Q), (nq - 1) & 1, ec, kSiteDrain, false);
        for (int s = 0; s < ST; ++s) {
          if (nk > s) mbar_wait(bar(PB_KF + s), (((nk - 1 - s) / ST)) & 1, ec, kSiteDrain, false);
          if (nv > s) mbar_wait(bar(PB_VF + s), (((nv - 1 - s) / ST)) & 1, ec, kSiteDrain, false);
        }
      }
    } else if (warp == 9) {
      // ---------------------------------------------------------- MMA issuer
      constexpr uint32_t kIdS = idesc_f16(128, 128, BF16, false, false);
      constexpr uint32_t kIdO = idesc_f16(128, DV, BF16, false, true);
      const uint64_t dQ0 = sdesc_sw128(sQ, 16, 1024);
      const uint64_t dK0 = sdesc_sw128(sK, 16, 1024);
      const uint64_t dV0 = sdesc_sw128(sV, C::BN * 128, 1024);
      uint32_t pph[2] = {0u, 0u};  // P phases consumed
      int nq = 0, base = 0;        // items, key tiles before this item
      bool ok = true;
      for (int idx; (ok = next_item(nq, &idx)) && idx < n_items;) {
        const PrefixItem it = prefix_item(p, idx);
        if (it.n == 0) break;
        auto issue_s = [&](int t, int i) -> bool {  // S_t = Q K^T of its round i
          const int j = prefix_tile(it, t, i), g = base + j;
          if (!mbar_wait_w(bar(PB_KF + g % ST), (g / ST) & 1, ec, kSiteFwdMma)) return false;
          tc_fence_after();
          const uint64_t dQ = opaque_u64(desc_adv(dQ0, it.dual ? t * C::Q_BYTES : 0));
          const uint64_t dK = opaque_u64(desc_adv(dK0, (g % ST) * C::K_BYTES));
#pragma unroll
          for (int kk = 0; kk < DQK / 16; ++kk) {
            const uint32_t off = (kk >> 2) * (128 * 128) + (kk & 3) * 32;
            umma_ss_w(tbase + C::T_S + 128 * t, desc_adv(dQ, off), desc_adv(dK, off), kIdS, kk > 0);
          }
          umma_commit_w(bar(PB_S + t));
          // the key tile's last product of this kind frees it; the item's last, Q
          if (!it.dual || t == 1 || !it.has1) {
            umma_commit_w(bar(PB_KE + g % ST));
            if (j == it.n - 1) umma_commit_w(bar(PB_QE));
          }
          return true;
        };
        auto issue_pv = [&](int t, int i) -> bool {  // O_t += P_t V
          const int j = prefix_tile(it, t, i), g = base + j;
          if (!mbar_wait_w(bar(PB_VF + g % ST), (g / ST) & 1, ec, kSiteFwdMma)) return false;
          // (the warpgroup cannot watch V's own barrier: it runs up to a ring's
          // turn ahead of V, where the barrier's parity says nothing)
          if (prefix_clears(it, t, j) && lane == 0) mbar_arrive(bar(PB_VZ + t));
          if (!mbar_wait_w(bar(PB_P + t), pph[t], ec, kSiteFwdMma)) return false;
          pph[t] ^= 1u;
          tc_fence_after();
          const uint64_t dV = opaque_u64(desc_adv(dV0, (g % ST) * C::V_BYTES));
#pragma unroll
          for (int kk = 0; kk < C::BN / 16; ++kk)
            umma_ts_w(tbase + C::T_O + DV * t, tbase + C::T_S + 128 * t + kk * 8, desc_adv(dV, kk * 2048), kIdO,
                      (i > 0 || kk > 0));
          if (!it.dual || t == 1 || !it.has1) umma_commit_w(bar(PB_VE + g % ST));
          return true;
        };
        if (!(ok = mbar_wait_w(bar(PB_Q), nq & 1, ec, kSiteFwdMma))) break;
        if (!(ok = issue_s(0, 0))) break;
        if (prefix_has(it, 1, 0) && !(ok = issue_s(1, 0))) break;
        const int rounds = it.dual ? it.n : (it.n + 1) / 2;
        for (int i = 0; ok && i < rounds; ++i) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok || !prefix_has(it, t, i)) continue;
            ok = issue_pv(t, i);
            if (!ok) continue;
            if (prefix_has(it, t, i + 1))
              ok = issue_s(t, i + 1);
            else
              umma_commit_w(bar(PB_O + t));
          }
        }
        if (!ok) break;
        ++nq;
        base += it.n;
      }
      umma_commit_w(bar(PB_DRAIN));
      mbar_wait(bar(PB_DRAIN), 0, ec, kSiteDrain, false);
    }
  } else {
    setmaxnreg_inc<C::REG_SOFTMAX>();
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2;
    const int li = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tbase + C::T_S + 128 * t, tO = tbase + C::T_O + DV * t;
    const float sl2 = p.scale_log2;
    const uint64_t sl22 = f2(sl2, sl2);
    const float neg = (CAP || sl2 < 0.f) ? -SDPA_NEG_INF : SDPA_NEG_INF;  // masked raw score
    uint32_t sph = 0, oph = 0, zph = 0;  // S, O and V-landed phases
    int base = 0, ni = 0;
    bool ok = true;
    for (int idx; (ok = next_item(ni, &idx)) && idx < n_items; ++ni) {
      const PrefixItem it = prefix_item(p, idx);
      if (it.n == 0) break;
      // this thread's row: sequence b, row x of its R
      const int tile = it.tile + (it.dual ? t : 0);
      int b, x;
      bool row_ok;
      if (p.R <= 128) {
        const int off = (it.quart ? lane : li) / p.R;
        x = (it.quart ? lane : li) - off * p.R;
        b = it.own ? it.b : tile * p.seqs_tile + off;
        row_ok = it.own ? off == 0 : (off < p.seqs_tile && b < p.B);
      } else {
        const int per = (p.R + 127) / 128;
        b = it.own ? it.b : tile / per;
        x = (it.own ? tile : tile % per) * 128 + li;
        row_ok = x < p.R && b < p.B;
      }
      if (it.dual && t == 1 && !it.has1) row_ok = false;
      const bool warp_ok = __any_sync(0xffffffffu, row_ok);
      // last visible key: all of the prefix; own keys up to the token's place
      const int last = it.own ? it.keys - p.s_q + x % p.s_q : it.keys - 1;
      const int all_see = it.own ? it.keys - p.s_q : it.keys - 1;  // visible to every row
      float m = SDPA_NEG_INF, l = 0.f;
      // columns col .. col + N - 1 of the tile, whose first is key k0 + col; P of the
      // others is 0
      auto softmax = [&](auto width, int col, int k0, bool rescale) {
        constexpr int N = decltype(width)::value;
        k0 += col;
        float xs[N];
        if constexpr (CAP) {
          // Eight scores of a row share their reciprocals: what lies behind the last key
          // must not lend its roundings to those before it. Zeroed in tensor memory, by a
          // loop: the unrolled softmaxes already miss the instruction cache.
          const int behind = it.keys - k0;
          if (behind > 0 && behind < N) {
#pragma unroll 1
            for (int c = behind; c & 7; ++c) tmem_st1(tS + lane_off + col + c, 0u);
            tmem_wait_st();
          }
        }
#pragma unroll
        for (int q = 0; q < N / 32; ++q) tmem_ld32f(tS + lane_off + col + q * 32, xs + q * 32);
        tmem_wait_ld();
        float mx = SDPA_NEG_INF;
        const bool hidden = k0 + N - 1 > all_see;  // there are hidden keys
        if constexpr (CAP) mx = cap_scores<N>(xs, p.cap_in, sl2, row_ok);
        if (hidden) {
#pragma unroll
          for (int e = 0; e < N; ++e)
            if (k0 + e > last) xs[e] = neg;
        }
        if (!CAP && sl2 > 0.f)
          mx = extreme_of<false, N>(xs) * sl2;
        else if (!CAP || hidden)
          mx = extreme_of<true, N>(xs) * sl2;
        // O is rescaled only when the maximum grew by more than 2^8 (fwd_kernel.cuh)
        const bool grow = mx > m + 8.0f;
        float alpha = 1.0f;
        if (grow) {
          alpha = ex2(m - mx);
          m = mx;
        }
        if (rescale && __any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int q = 0; q < DV / 16; ++q) {
            uint32_t rr[16];
            tmem_ld16(tO + lane_off + q * 16, rr);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) rr[e] = __float_as_uint(__uint_as_float(rr[e]) * alpha);
            tmem_st16(tO + lane_off + q * 16, rr);
          }
        }
        l *= alpha;
        const float mu = (m == SDPA_NEG_INF) ? 0.f : m;
        const uint64_t nm2 = f2(-mu, -mu);
        uint64_t sa = f2(0.f, 0.f), sb = f2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < N; e += 4) {
          const float2 a = f2split(fma2(f2(xs[e], xs[e + 1]), sl22, nm2));
          const float2 c = f2split(fma2(f2(xs[e + 2], xs[e + 3]), sl22, nm2));
          xs[e] = ex2(a.x);
          xs[e + 1] = ex2(a.y);
          xs[e + 2] = ex2(c.x);
          xs[e + 3] = ex2(c.y);
          sa = add2(sa, f2(xs[e], xs[e + 1]));
          sb = add2(sb, f2(xs[e + 2], xs[e + 3]));
        }
        const float2 u = f2split(sa), w = f2split(sb);
        l += (u.x + u.y) + (w.x + w.y);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            pk[e] = N == 128 ? pack2<BF16>(xs[(q * 32 + 2 * e) % N], xs[(q * 32 + 2 * e + 1) % N]) : 0u;
          if (N == 128 || q * 32 != col) tmem_st16(tS + lane_off + q * 16, pk);
        }
        if constexpr (N == 32) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) pk[e] = pack2<BF16>(xs[2 * e], xs[2 * e + 1]);
          tmem_st16(tS + lane_off + col / 2, pk);
        }
        tmem_wait_st();
      };
      int i = 0;
      for (; ok && prefix_has(it, t, i); ++i) {
        const int j = prefix_tile(it, t, i);
        const int k0 = (it.k0 + j) * C::BN;
        if (prefix_clears(it, t, j)) {
          const int g = base + j;
          if (!(ok = mbar_wait(bar(PB_VZ + t), zph, ec, kSiteFwdSoftmax))) break;
          zph ^= 1u;
          uint8_t* v = smem + C::OFF_V + (g % ST) * C::V_BYTES;
          const int first = it.keys - k0;  // in [1, 127]
          for (int e = li; e < (C::BN - first) * 8; e += 128) {
#pragma unroll
            for (int c = 0; c < DV / 64; ++c)
              *reinterpret_cast<uint4*>(v + c * C::BN * 128 + first * 128 + e * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        if (!(ok = mbar_wait(bar(PB_S + t), sph, ec, kSiteFwdSoftmax))) break;
        sph ^= 1u;
        tc_fence_after();
        if (warp_ok) {
          if (it.quart)
            softmax(std::integral_constant<int, 32>{}, (warp & 3) * 32, k0, i > 0);
          else
            softmax(std::integral_constant<int, 128>{}, 0, k0, i > 0);
        }
        tc_fence_before();
        mbar_arrive(bar(PB_P + t));
      }
      if (!ok) break;
      base += it.n;
      // ---- the item's partial rows: O / l and log2 of the sum of exponentials
      // (single items of one key tile leave warpgroup 1 without one: L = -inf)
      if (i > 0) {
        if (!(ok = mbar_wait(bar(PB_O + t), oph, ec, kSiteFwdSoftmax))) break;
        oph ^= 1u;
        tc_fence_after();
      }
      const int64_t ri = (static_cast<int64_t>(row_ok ? b : 0) * p.H_kv + it.hk) * p.R + (row_ok ? x : 0);
      const int slot = it.slot + (it.dual ? 0 : it.quart ? 4 * t + (warp & 3) : t);
      const int64_t at = slot * p.rows + ri;
      if (i > 0 && warp_ok) {
        const float inv = l > 0.f ? 1.0f / l : 0.f;
        float4* dst = reinterpret_cast<float4*>(p.part) + prefix_part_index(slot, p.rows, ri, DV);
#pragma unroll
        for (int q = 0; q < DV / 32; ++q) {
          uint32_t rr[32];
          tmem_ld32(tO + lane_off + q * 32, rr);
          tmem_wait_ld();
          if (row_ok && l > 0.f) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[(q * 8 + e) * 8] = make_float4(__uint_as_float(rr[4 * e]) * inv, __uint_as_float(rr[4 * e + 1]) * inv,
                                           __uint_as_float(rr[4 * e + 2]) * inv,
                                           __uint_as_float(rr[4 * e + 3]) * inv);
          }
        }
      }
      // (a sum that is not a number leaves an L that is none: the join then makes the
      // row none, without reading the partial, which is not stored)
      if (row_ok) p.part_lse[at] = l == 0.f ? SDPA_NEG_INF : m + __log2f(l) + p.lse_shift;
      tc_fence_before();  // O has been read before the next item's P is announced
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tbase, C::TMEM_COLS);
  }
}

template <int DQK, int DV, bool BF16>
cudaError_t launch_prefix_t(const CUtensorMap (&m)[6], const PrefixParams& p, cudaStream_t st) {
  using C = PrefixCfg<DQK, DV>;
  auto kern = p.cap_in != 0.f || p.lse_shift != 0.f ? sdpa_prefix_kernel<DQK, DV, BF16, true>
                                                     : sdpa_prefix_kernel<DQK, DV, BF16, false>;
  cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(kern), C::SMEM, C::REG_LAUNCH);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.grid));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  // the launch overlaps the kernel that clears the counter
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = p.next != nullptr ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, m[0], m[1], m[2], m[3], m[4], m[5], p);
}

}  // namespace sdpa
