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
// 128 lanes and NR = 8, 16, 32 or 64 rows as its columns, and O^T = V^T P^T the
// values' width on the lanes. A thread has one key: its rows' scores are its
// registers, P^T goes back through shared memory (a key's rows side by side), and
// only the maxima and sums cross threads: the sums once a unit, the maxima when
// one has grown by more than 2^8, which a vote of the warpgroup finds out.
// (With the rows on the lanes, as sdpa_prefix_kernel has them, a row of 8 keeps a
// warp busy with 128 columns while the others idle.) The products read their long
// operand from shared memory, and a few columns more cost them nothing: P goes in
// as a high and a low part, each rounded to 16 bits, side by side, whose two O are
// added at the end, so that its rounding (2^-8 in bf16, as much as O's own) is gone. In
// fp16 the low part is held 2^18 times as large: what is below 2^-25, which the high part
// loses (131072 keys of 2^-25.4 beside one of 1 are 2^-8.4 of O), is in it down to 2^-43.
//
// The lengths are known on the device only. All units (sequence, K/V head, row
// block) in a row, each as long as its key tiles, are one line, cut into equal
// runs, one for each CTA: any mix of lengths ends at about the same time on all SMs. A
// unit that a run's end cuts leaves normalised fp32 rows O_s and their log2-sum-exps
// L_s, at most two slots a CTA, which are joined,
//   L = log2 sum_s 2^L_s,  O = sum_s 2^(L_s - L) O_s,
// in the order of the runs; the others are written as they are. Who leaves the last
// of a unit's parts joins them where there are two a unit or fewer (by the units there
// are): a kernel of its own for that (paged_join.cu) takes 6 us from the end of one to
// the next call's first look at memory: 96 sequences of up to 5000 keys on one K/V
// head 31.7 us for 33.6. Where there are more, that kernel does, with all SMs: one
// sequence of 131072 keys, 8 K/V heads, 19 parts each, 81.3 us for 84.2. Units of few
// tiles are not cut (paged.cuh).
//
// One persistent CTA an SM. Roles: two warpgroups of softmax threads (at NR = 8 and 16 they
// take the key tiles in turns, each with a maximum, sum and O of its own, joined at
// the unit's end by the one that had the last tile, while the other goes on; at 32
// and 64 each has half of the rows: in turns, 32 columns a thread spill, and 64 sequences
// of 4096 keys on 4 K/V heads of d64 took 75.7 us for 54.2), two producer warps, which
// both walk the run and copy pages by TMA, one the keys, the other the values (a copy of
// a small page takes its warp longer to issue than memory to deliver), and two MMA
// issuers, one for S^T, up to two tiles ahead, one for O^T: the products are so small that
// a tile's instructions and waits, not the tensor cores, bound an issuer (1900 cycles a
// tile of d = 64 for one warp with both). The keys' producer also copies the queries and
// tells the others the units through a ring.
// Rows of a tile that no query sees (behind the last key, before the window,
// in pages that are not read) may hold anything. Their scores are masked; their
// values, which P's zeros would not cancel, are left out of the product 16 keys at
// a time, and zeroed in shared memory within such a step, by the MMA issuer, which
// waits for the values anyway. (Zeroed by the softmax threads, which then had to wait
// for them too, 256 sequences of up to 777 keys took 209 us for 16 heads of their
// own, where whole tiles of as many bytes took 131.)
//
// Bound by memory: 152 sequences of 4096 keys, 8 heads on one K/V head of d128, take 50.0 us
// (6.4 TB/s, 94% of the copy rate), of which 2 pass before the first keys are asked for
// (lengths, then the table, then keys) and 3 with the last parts' join; one sequence of
// 131072 keys on 8 K/V heads 81.9 us (6.55 TB/s). Short units are bound by the keys'
// producer and the ends of units instead: 0.9 us each.
#pragma once
#include "common.cuh"
#include "paged.cuh"

namespace sdpa {

template <int DQK, int DV, int NR>
struct PagedCfg {
  static constexpr int BN = kPagedTile;
  static constexpr int N = NR < 16 ? 16 : NR;          // columns of S (an MMA of 128 lanes has 16 at least)
  static constexpr int NP = 2 * NR;                    // columns of P and O: the high parts' rows, the low parts'
  static constexpr bool TURNS = NR <= 16;              // the warpgroups take tiles in turns, else half of the rows each
  static constexpr int NC = TURNS ? NR : NR / 2;       // rows a thread
  static constexpr int SOFT = 256;                     // softmax threads
  static constexpr int THREADS = SOFT + 128;
  static constexpr int K_BYTES = BN * DQK * 2;
  static constexpr int V_BYTES = BN * DV * 2;
  static constexpr int Q_BYTES = N * DQK * 2;
  static constexpr int P_PITCH = NP < 64 ? NP * 2 : 128;  // bytes of a key in an atom of P^T: the swizzle's width
  static constexpr int P_BYTES = BN * NP * 2;
  static constexpr int P_BUFS = TURNS ? 2 : 1;
  // barriers and so on; two rows of NC floats a softmax warp; statistics handed over
  static constexpr int MISC = 1024 + SOFT / 32 * NC * 8 + (TURNS ? 4 * NR * 8 : 0);
  // Few rows: a unit's queries come with its first keys, into as many buffers as there
  // are stages. (A stage's wait for tile t - ST is then one for the queries' buffer: the ST - 1
  // units between have a tile each, so that of the unit which had it lies no later.) With a
  // ring of two and barriers of their own, as for more rows, whose buffers are larger, 256
  // sequences of up to 100 keys on 8 K/V heads took 21.3 us for 19.5: their many short units
  // are bound by the keys' producer and by the ends of units.
  static constexpr bool Q_WITH_K = TURNS;
  static constexpr int AVAIL = 227 * 1024 - 1024 - P_BUFS * P_BYTES - MISC;
  static constexpr int Q_RING = Q_BYTES > 16384 ? 1 : 2;
  static constexpr int FIT = Q_WITH_K ? AVAIL / (K_BYTES + V_BYTES + Q_BYTES)
                                      : (AVAIL - Q_RING * Q_BYTES) / (K_BYTES + V_BYTES);
  static constexpr int ST = FIT > 6 ? 6 : FIT;
  static constexpr int Q_BUFS = Q_WITH_K ? ST : Q_RING;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + ST * K_BYTES;
  static constexpr int OFF_Q = OFF_V + ST * V_BYTES;
  static constexpr int OFF_P = OFF_Q + Q_BUFS * Q_BYTES;
  static constexpr int OFF_MISC = OFF_P + P_BUFS * P_BYTES;
  static constexpr int SMEM = OFF_MISC + MISC + 1024;
  static constexpr int OS = TURNS ? 2 : 1;
  static constexpr uint32_t T_S = 0, T_O = 2 * N;      // S of two tiles; O of two units (of each warpgroup)
  static constexpr uint32_t T_END = T_O + 2 * OS * NP;
  static constexpr uint32_t TMEM_COLS = T_END <= 128 ? 128 : T_END <= 256 ? 256 : 512;
  static_assert(ST >= 2 && SMEM <= 227 * 1024, "shared memory");
};

// Barriers: rings of K and V, Q of a unit, S and P of a tile, P V done, O of a
// unit full and read, statistics handed over, ring of units.
enum : int { GB_KF = 0, GB_KE = GB_KF + 6, GB_VF = GB_KE + 6, GB_VE = GB_VF + 6, GB_Q = GB_VE + 6, GB_QE = GB_Q + 2,
             GB_S = GB_QE + 2, GB_P = GB_S + 2, GB_PV = GB_P + 2, GB_O = GB_PV + 2, GB_OE = GB_O + 2,
             GB_ST = GB_OE + 2, GB_I = GB_ST + 4, GB_IE = GB_I + 4, GB_DRAIN = GB_IE + 4, GB_START = GB_DRAIN + 2,
             GB_COUNT = GB_START + 2 };

// One unit's part of a run, as the producer tells it.
struct PagedItem {
  int n;          // key tiles (0: the sequence has no key; -1: the run's end)
  int b, hk, rb;  // sequence, K/V head, row block
  int k0;         // first key tile
  int len;        // keys of the sequence
  int slot;       // partial slot, or -1: the whole unit
  int parts;      // of a cut unit: its first run, its runs << 16
};

// P^T, a key's rows side by side (MN-major): atoms of 8 keys as wide as the swizzle.
__device__ __forceinline__ uint64_t paged_desc_p(uint32_t saddr, int pitch) {
  uint64_t d = sdesc_sw128(saddr, kPagedTile * 128, 8 * pitch);
  if (pitch < 128) d = (d & ~(uint64_t{7} << 61)) | (static_cast<uint64_t>(pitch == 64 ? 4 : 6) << 61);
  return d;
}

// tanh to 2^-22.2 relative (against 64 bits, all fp32 numbers from 2^-20 to 12): z + z^3
// q(z^2) up to 5/8, q a polynomial fitted to it by reweighted least squares (itself good to
// 2^-26.8; 2^-23.6 with its roundings), else 1 - 2 / (1 + e^(2 |z|)), which is at its worst
// just behind 5/8, 2^-22.3, and from 1 on good to 2^-23.1. (cap_r8's form is good to 2^-20
// of the cap, which a sum of many rows, LSE, shows; here the keys' stream leaves time for this one.)
__device__ __forceinline__ float paged_tanh(float z) {
  const float a = fabsf(z), z2 = z * z;
  const float far = copysignf(fmaf(-2.f, rcp(1.f + ex2(a * (2.f * kLog2e))), 1.f), z);
  float q = fmaf(z2, -0.00570499f, 0.02063909f);
  q = fmaf(z2, q, -0.05373972f);
  q = fmaf(z2, q, 0.13331442f);
  q = fmaf(z2, q, -0.3333328f);
  return a < 0.625f ? fmaf(z * z2, q, z) : far;
}

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// A bounded wait (mbar_wait), of which only the first look is inlined: there are
// some thirty waits, and the kernel's code has to stay in the instruction cache, whose
// misses queue behind the keys and values.
static __device__ __noinline__ bool paged_wait_on(uint32_t bar, uint32_t phase, uint32_t* err,
                                                  volatile uint32_t* abort, uint32_t site) {
  return mbar_wait(bar, phase, ErrCtx{err, abort}, site & ~(1u << 31), true, (site >> 31) != 0);
}
// By a converged warp; the same result in every lane. sleep: as in mbar_wait.
__device__ __forceinline__ bool paged_wait(uint32_t bar, uint32_t phase, const ErrCtx& e, uint32_t site,
                                           bool sleep = false) {
  bool ok = mbar_try_wait(bar, phase);
  if (!__all_sync(0xffffffffu, ok)) {
    if (!ok) ok = paged_wait_on(bar, phase, e.err_word, e.abort, site | (sleep ? 1u << 31 : 0u));
    ok = __all_sync(0xffffffffu, ok);
  }
  return ok;
}

// Of a cut unit: its first run, the group of parts that this CTA's is in, the words of
// both (of a half of the rows).
struct PagedParts {
  int first, groups, from, n;
  unsigned long long *word, *unit;
};
__device__ __forceinline__ PagedParts paged_parts(unsigned long long* words, int code, int half) {
  const int first = code & 0xffff, parts = code >> 16;
  const int group = (static_cast<int>(blockIdx.x) - first) / kPagedGroup, from = first + group * kPagedGroup;
  return PagedParts{first, (parts + kPagedGroup - 1) / kPagedGroup, from, min(kPagedGroup, parts - group * kPagedGroup),
                    words + 6 * from + (group == 0 ? 0 : 2) + half, words + 6 * first + 4 + half};
}
// A word of any former contents that parts are counted in at: nonce << 16 | count.
// Made ready when the kernel starts, by each that will count itself in (one of them
// succeeds; a compare-and-swap to count with would be tried again by all that come at
// once, and one just before waits as long as the memory's queue is).
__device__ __forceinline__ void paged_ready(unsigned long long* word, unsigned long long nonce) {
  const unsigned long long old = *reinterpret_cast<volatile unsigned long long*>(word);
  if (old >> 16 != nonce) atomicCAS(word, old, nonce << 16);
}
// True for the last of `parts`, which leaves a 0 behind, so that a captured call,
// whose nonce is the same in every replay, finds no count of the last replay.
__device__ __forceinline__ bool paged_count_in(unsigned long long* word, int parts) {
  const bool last = static_cast<int>((atomicAdd(word, 1ull) + 1) & 0xffff) == parts;
  if (last) atomicExch(word, 0ull);
  return last;
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

// The part of a cut unit has been written (by a warpgroup: half of the rows, or all of
// them): the last to write one of a group of kPagedGroup parts joins the group, the
// last to do that joins the groups. (A run may have the last part of a unit, a group by
// itself, and the first of another: first groups and later ones have words of their
// own.) False: a wait ran out, all leave. Not inlined: most units come without. o and
// lse are those of the warpgroup's first row.
template <int DV, bool BF16, int NR>
__device__ __noinline__ bool paged_join(float* part, float* part_lse, unsigned long long* words, uint8_t* o, float* lse,
                                        int code, int half, int bar_id, int col0, int live, bool ok, int* flag) {
  constexpr int LANES = DV / 4, W = 4;  // lanes a row; parts fetched at once
  const int lane = threadIdx.x & 31, w4 = (threadIdx.x >> 5) & 3;
  const PagedParts c = paged_parts(words, code, half);
  int from = c.from, n = c.n, step = 1;
  unsigned long long* word = c.word;
  bool final = c.groups == 1;
#pragma unroll 1
  for (;;) {
    // what the warpgroup wrote is in memory
    __threadfence();
    if (!named_bar_and(bar_id, 128, ok)) {
      named_bar_and(bar_id, 128, false);
      return false;
    }
    if ((threadIdx.x & 127) == 0) *flag = paged_count_in(word, n) ? 1 : 0;
    named_bar_and(bar_id, 128, true);
    if (*reinterpret_cast<volatile int*>(flag) == 0) return true;
    __threadfence();
#pragma unroll 1
    for (int e0 = w4; e0 < live; e0 += 8) {  // rows e0 and e0 + 4
      float m2[2] = {SDPA_NEG_INF, SDPA_NEG_INF}, l2[2] = {0.f, 0.f};
      float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll 1
      for (int s0 = 0; s0 < n; s0 += W) {
        float4 v[2][W];
        float L[2][W];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < W; ++i) {
            const int run = from + min(s0 + i, n - 1) * step, e = min(e0 + 4 * r, live - 1);
            const int64_t row = static_cast<int64_t>(2 * run + (run == c.first ? 1 : 0)) * NR + col0 + e;
            L[r][i] = s0 + i < n ? __ldcg(part_lse + row) : SDPA_NEG_INF;
            v[r][i] = __ldcg(reinterpret_cast<const float4*>(part + row * DV) + (lane & (LANES - 1)));
          }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < W; ++i) {
            // (a maximum that skips what is not a number: the weight then is none, and the row)
            const float mn = fmaxf(m2[r], L[r][i]), base = mn == SDPA_NEG_INF ? 0.f : mn;
            const float keep = ex2(m2[r] - base), w = ex2(L[r][i] - base);
            const bool some = w > 0.f;
            float4& a = acc[r];
            m2[r] = mn;
            l2[r] = fmaf(l2[r], keep, w);
            a.x = fmaf(w, some ? v[r][i].x : 0.f, a.x * keep), a.y = fmaf(w, some ? v[r][i].y : 0.f, a.y * keep);
            a.z = fmaf(w, some ? v[r][i].z : 0.f, a.z * keep), a.w = fmaf(w, some ? v[r][i].w : 0.f, a.w * keep);
          }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int e = e0 + 4 * r;
        if (e >= live) break;
        const float inv = l2[r] == 0.f ? 0.f : 1.f / l2[r], log_l = l2[r] == 0.f ? SDPA_NEG_INF : m2[r] + __log2f(l2[r]);
        const float4 a = make_float4(acc[r].x * inv, acc[r].y * inv, acc[r].z * inv, acc[r].w * inv);
        if (final) {
          if (lane < LANES)
            reinterpret_cast<uint2*>(o + e * (DV * 2))[lane] =
                make_uint2(pack2<BF16>(a.x, a.y), pack2<BF16>(a.z, a.w));
          if (lane == 0) lse[e] = log_l * kLn2;
        } else {  // to the group's first slot
          const int64_t row = static_cast<int64_t>(2 * from + (from == c.first ? 1 : 0)) * NR + col0 + e;
          __syncwarp();
          if (lane < LANES) reinterpret_cast<float4*>(part + row * DV)[lane] = a;
          if (lane == 0) part_lse[row] = log_l;
        }
      }
    }
    if (final) return true;
    from = c.first;
    n = c.groups;
    step = kPagedGroup;
    word = c.unit;
    final = true;
  }
}

// How long a unit of the sequence is on the line.
__device__ __forceinline__ int paged_weight(const PagedParams& p, const PagedSpan& s) {
  return p.whole == kUnitsAlike ? 1 : s.n + kPagedCost;
}

template <int DQK, int DV, bool BF16, int NR>
__global__ void __launch_bounds__(PagedCfg<DQK, DV, NR>::THREADS, 1)
    sdpa_paged_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PagedParams p) {
  using C = PagedCfg<DQK, DV, NR>;
  constexpr int ST = C::ST, N = C::N, NP = C::NP, NC = C::NC, BN = C::BN;
  constexpr int kWarpsAll = C::THREADS / 32, kSoftWarps = C::SOFT / 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  const uint32_t sK = smem_u32(smem + C::OFF_K), sV = smem_u32(smem + C::OFF_V);
  const uint32_t sQ = smem_u32(smem + C::OFF_Q), sP = smem_u32(smem + C::OFF_P);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_MISC);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + GB_COUNT);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  int* start = reinterpret_cast<int*>(tmem_slot + 4);              // sequence, place in it, its length
  uint32_t* scan = reinterpret_cast<uint32_t*>(tmem_slot + 8);     // [warps] sums
  int* items = reinterpret_cast<int*>(tmem_slot + 8 + 16);         // ring of 4, 8 words each
  int* sIds = items + 32;                                          // [producers][32] pages
  int* sFlag = sIds + 64;                                          // [warpgroups]
  static_assert(GB_COUNT * 8 + 96 + 128 + 256 + 16 <= 1024 && GB_COUNT % 2 == 0, "barrier region");
  // [softmax warps][NC] values of rows. While maxima are exchanged, sMax holds each
  // warp's and sRow is its own; at a unit's end sRow holds each warp's sums and sMax is
  // its own. Between the two uses lies a barrier of the warpgroup.
  float* sMax = reinterpret_cast<float*>(smem + C::OFF_MISC + 1024);
  float* sRow = sMax + kSoftWarps * NC;
  float* sStat = sRow + kSoftWarps * NC;  // [4][maximum, sum][NR]: statistics of the other warpgroup's tiles
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  if (warp == kSoftWarps) {
    for (int i = lane; i < GB_COUNT; i += 32) {
      uint32_t n = 1;
      if ((i >= GB_P && i < GB_P + 2) || (i >= GB_OE && i < GB_OE + 2)) n = C::TURNS ? kSoftWarps / 2 : kSoftWarps;
      if (i >= GB_IE && i < GB_DRAIN) n = kSoftWarps + 2;
      mbar_init(bar(i), n);
    }
    if (lane == 0) *abort_flag = 0u;
    fence_mbar_init();
  } else if (warp == kSoftWarps + 1) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  } else if (warp == kSoftWarps + 2) {
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
  }
  // rows of Q that no box fills stay 0
#pragma unroll 1
  for (int i = tid; i < C::Q_BUFS * C::Q_BYTES / 16; i += C::THREADS)
    reinterpret_cast<uint4*>(smem + C::OFF_Q)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  // (launched while the kernel before runs out: from here on its memory is looked at, by loads
  // that are not the read-only ones, which the compiler may put ahead of this)
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- this CTA's run: [lo, hi) of the line of all units
  // thread i has the sequences [i per, (i + 1) per)
  const int per = (p.B + C::THREADS - 1) / C::THREADS;
  const int units = p.H_kv * p.row_blocks;  // of a sequence
  uint32_t sum = 0;
#pragma unroll 1
  for (int i = tid * per; i < min(p.B, (tid + 1) * per); ++i)
    sum += p.whole == kUnitsAlike ? 1u : static_cast<uint32_t>(paged_weight(p, paged_span(p, p.seqlen[i])));
  sum *= static_cast<uint32_t>(units);
  uint32_t upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += u;
  }
  if (lane == 31) scan[warp] = upto;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t of_warp = lane < kWarpsAll ? scan[lane] : 0u;
  const uint32_t total = __reduce_add_sync(0xffffffffu, of_warp);
  const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? of_warp : 0u);
  // equal runs, the first ones longer by one
  const uint32_t each = total / gridDim.x, more = total - each * gridDim.x;
  const uint32_t run_lo = each * blockIdx.x + min(blockIdx.x, more);
  const uint32_t run_hi = run_lo + each + (blockIdx.x < more ? 1u : 0u);
  auto run_of = [&](uint32_t at) -> int {  // the run that has a place of the line
    const uint32_t longer = more * (each + 1);
    return static_cast<int>(at < longer ? at / (each + 1) : more + (at - longer) / each);
  };
  upto += before;
  if (run_lo < run_hi && run_lo >= upto - sum && run_lo < upto) {  // one thread of the CTA
    uint32_t at = run_lo - (upto - sum);
    int i = tid * per;
#pragma unroll 1
    for (;; ++i) {
      const int len = p.seqlen[i];
      const uint32_t w = static_cast<uint32_t>(paged_weight(p, paged_span(p, len))) * units;
      if (at < w) {
        start[2] = len;
        break;
      }
      at -= w;
    }
    start[0] = i;
    start[1] = static_cast<int>(at);
    mbar_arrive(bar(GB_START));
  }
  const uint32_t tbase = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const ErrCtx ec{p.err, abort_flag};
  auto next_item = [&](int u, PagedItem* it) -> bool {
    if (!paged_wait(bar(GB_I + (u & 3)), (u >> 2) & 1, ec, kSiteFwdSoftmax)) return false;
    const int4 a = *reinterpret_cast<const int4*>(items + (u & 3) * 8);
    const int4 b = *reinterpret_cast<const int4*>(items + (u & 3) * 8 + 4);
    auto one = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    *it = PagedItem{one(a.x), one(a.y), one(a.z), one(a.w), one(b.x), one(b.y), one(b.z), one(b.w)};
    return true;
  };

  if (warp == kSoftWarps || warp == kSoftWarps + 2) {
    // ----------------------------------------------------------- producers
    const bool keys = warp == kSoftWarps;
    const int width = keys ? DQK / 64 : DV / 64;  // 64-column chunks
    const uint32_t ring = keys ? sK : sV, stage_bytes = keys ? C::K_BYTES : C::V_BYTES;
    const int full = keys ? GB_KF : GB_VF, empty = keys ? GB_KE : GB_VE;
    const CUtensorMap* map = keys ? &tmK : &tmV;
    auto free_of = [&](int i, int round) {  // the round's use of barrier i's buffer may begin
      return paged_wait(bar(i), (round & 1) ^ 1, ec, kSiteFwdLoad, true);
    };
    int nt = 0, nu = 0, nq = 0;  // tiles copied, items told, items with keys so far
    int s = 0, round = 0;        // stage of the ring, and its uses
    bool ok = true;
    int4 record = make_int4(0, 0, 0, 0);
    auto tell = [&](const PagedItem& it) -> bool {
      if (!keys) return true;
      if (!free_of(GB_IE + (nu & 3), nu >> 2)) return false;
      if (lane == 0) {
        *reinterpret_cast<int4*>(items + (nu & 3) * 8) = make_int4(it.n, it.b, it.hk, it.rb);
        *reinterpret_cast<int4*>(items + (nu & 3) * 8 + 4) = make_int4(it.k0, it.len, it.slot, it.parts);
        mbar_arrive(bar(GB_I + (nu & 3)));
      }
      __syncwarp();
      ++nu;
      return true;
    };
    uint32_t left = run_hi - run_lo;
    if (left > 0 && !paged_wait(bar(GB_START), 0, ec, kSiteFwdLoad)) left = 0;
    int i = 0, hk = 0, rb = 0, pos = 0;  // sequence, K/V head, row block; place in the unit
    PagedSpan sp{0, 0, 0}, sp_next{0, 0, 0};
    // A tile's copies are boxes of a page, of `box` keys each. Lane l has the page of
    // box ib + l of sequence is (in shared memory too, for the lane that copies), and of
    // the batch of boxes that is wanted next.
    const int per_tile = BN >> p.box_shift;
    int is = -1, ib = 0, ids = 0, as = -1, ab = 0, ids_ahead = 0;
    int* own_ids = sIds + (keys ? 0 : 32);
    auto pages_of = [&](int i, int len, int b0) {  // (looked at, and held inside the pool, where it is used)
      const int key = (b0 + lane) << p.box_shift;
      return key < len ? p.table[i * p.table_stride + (key >> p.page_shift)] : 0;
    };
    int l0 = 0, lens = 0, lens_ahead = 0;
    auto length = [&](int i) { return i < p.B ? p.seqlen[i] : 0; };
    auto first_tile = [&]() { return sp.lo + (p.whole ? 0 : max(pos - kPagedCost, 0)); };
    if (left > 0) {
      i = l0 = start[0];
      sp = paged_span(p, start[2]);
      const int w = paged_weight(p, sp);
      const int unit = start[1] / w;
      pos = start[1] - unit * w;
      hk = unit / p.row_blocks;
      rb = unit - hk * p.row_blocks;
      // the first unit's pages at once, then the lengths of 32 sequences from l0 on, a
      // lane each, and of the 32 after them
      as = i;
      ab = first_tile() * per_tile;
      ids_ahead = pages_of(i, sp.len, ab);
      lens = length(l0 + lane);
      lens_ahead = length(l0 + 32 + lane);
    }
    auto span_of = [&](int i) {  // i in [l0, l0 + 64)
      const int near = __shfl_sync(0xffffffffu, lens, (i - l0) & 31);
      const int far = __shfl_sync(0xffffffffu, lens_ahead, (i - l0) & 31);
      return paged_span(p, i - l0 < 32 ? near : far);
    };
    bool ahead_known = false;  // sp_next is that of sequence i + 1
    while (left > 0) {
      const int w = paged_weight(p, sp);
      const int take = static_cast<int>(min(left, static_cast<uint32_t>(w - pos)));
      // (a unit that is not cut is all of the run's in which it begins)
      const int t0 = p.whole ? (pos > 0 ? sp.n : 0) : max(pos - kPagedCost, 0);
      const int t1 = p.whole ? sp.n : max(pos + take - kPagedCost, 0);
      const bool none = sp.n == 0 && pos == 0;
      if (t1 > t0 || none) {
        PagedItem it;
        it.n = t1 - t0;
        it.b = i;
        it.hk = hk;
        it.rb = rb;
        it.k0 = sp.lo + t0;
        it.len = sp.len;
        it.slot = -1;
        it.parts = 0;
        if (t0 > 0 || t1 < sp.n) {  // cut: the runs with its first and its last tile
          const uint32_t tile0 = run_hi - left - pos + kPagedCost;
          const int from = run_of(tile0), to = run_of(tile0 + sp.n - 1);
          it.slot = 2 * blockIdx.x + (t0 > 0 ? 0 : 1);
          it.parts = from | (to - from + 1) << 16;
          const int id = i * units + hk * p.row_blocks + rb + 1;
          if (t0 > 0)
            record.x = id, record.y = t1 == sp.n;
          else
            record.z = id;
        }
        if (!(ok = tell(it))) break;
        if (it.n > 0) {
          const int qb = nq % C::Q_BUFS;
          auto copy_q = [&](uint32_t b) {
#pragma unroll
            for (int c = 0; c < DQK / 64; ++c)
              tma_load_4d(sQ + qb * C::Q_BYTES + c * N * 128, &tmQ, b, c * 64, it.rb * NR, it.b, it.hk);
          };
          if (!C::Q_WITH_K && keys) {
            if (!(ok = free_of(GB_QE + qb, nq / C::Q_BUFS))) break;
            if (elect_one_sync()) {
              mbar_arrive_expect_tx(bar(GB_Q + qb), (DQK / 64) * p.q_box);
              copy_q(bar(GB_Q + qb));
            }
            __syncwarp();
          }
          ++nq;
          // boxes with a key that some token sees: [first, end)
          const int seen = p.left < 0 ? 0 : max(0, sp.len - p.s_q - p.left);
          const int first = seen >> p.box_shift, end = (sp.len + p.box - 1) >> p.box_shift;
          const bool again = hk + 1 < p.H_kv || rb + 1 < p.row_blocks;  // the next unit is of the same sequence
          for (int j = 0; j < it.n; ++j) {
            const int box0 = (it.k0 + j) * per_tile;
            const bool batch = j == 0 || box0 - ib == 32;  // another batch of pages
            if (batch && (is != i || ib != box0)) {
              ids = as == i && ab == box0 ? ids_ahead : pages_of(i, sp.len, box0);
              is = i;
              ib = box0;
              // (the first page behind the pool reads as zeros)
              own_ids[lane] = static_cast<uint32_t>(ids) < static_cast<uint32_t>(p.n_pages) ? ids : p.n_pages;
              __syncwarp();
            }
            if (!(ok = free_of(empty + s, round))) break;
            const int lo = max(box0, first), hi = min(box0 + per_tile, end);
            if (elect_one_sync()) {
              const uint32_t b = bar(full + s), rows = static_cast<uint32_t>(p.box) * 128u;  // bytes of a box
              const bool with_q = C::Q_WITH_K && keys && j == 0;
              mbar_arrive_expect_tx(b, static_cast<uint32_t>(hi - lo) * rows * width +
                                           (with_q ? (DQK / 64) * p.q_box : 0u));
              if (with_q) copy_q(b);
              uint32_t dst = ring + s * stage_bytes + static_cast<uint32_t>(lo - box0) * rows;
#pragma unroll 1
              for (int x = lo; x < hi; ++x, dst += rows) {
                const int pg = own_ids[x - ib], in_page = (x << p.box_shift) & ((1 << p.page_shift) - 1);
#pragma unroll
                for (int c = 0; c < DQK / 64; ++c)
                  if (c < width) tma_load_4d(dst + c * BN * 128, map, b, c * 64, in_page, it.hk, pg);
              }
            }
            __syncwarp();
            ++nt;
            if (++s == ST) {
              s = 0;
              ++round;
            }
            if (batch) {
              // the batch after this one: of this unit, of the next one of the sequence,
              // or of the next sequence
              if ((it.k0 + it.n) * per_tile > box0 + 32) {
                as = i, ab = box0 + 32;
                ids_ahead = pages_of(i, sp.len, ab);
              } else if (again && sp.lo * per_tile != box0) {
                as = i, ab = sp.lo * per_tile;
                ids_ahead = pages_of(i, sp.len, ab);
              } else if (as != i + 1 && i + 1 < p.B) {
                sp_next = span_of(i + 1);
                ahead_known = true;
                as = i + 1, ab = sp_next.lo * per_tile;
                ids_ahead = pages_of(i + 1, sp_next.len, ab);
              }
            }
          }
          if (!ok) break;
        }
      }
      left -= static_cast<uint32_t>(take);
      pos = 0;
      if (++rb == p.row_blocks) {
        rb = 0;
        ++hk;
      }
      if (hk == p.H_kv && left > 0) {
        hk = 0;
        ++i;
        if (i - l0 == 32) {
          l0 = i;
          lens = lens_ahead;
          lens_ahead = length(l0 + 32 + lane);
        }
        sp = ahead_known ? sp_next : span_of(i);
        ahead_known = false;
      }
    }
    if (keys && lane == 0 && p.runs != nullptr) p.runs[blockIdx.x] = record;
    // (the next kernel may come: it waits for this one's end before it looks at memory)
    if (keys) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (ok) tell(PagedItem{-1, 0, 0, 0, 0, 0, 0, 0});
    // Every copy issued must land before the CTA can retire; on the healthy path they
    // did long ago.
    __syncwarp();
    if (*abort_flag) {
#pragma unroll 1
      for (int b = 0; b < C::Q_BUFS; ++b)
        if (!C::Q_WITH_K && keys && nq > b)
          mbar_wait(bar(GB_Q + b), ((nq - 1 - b) / C::Q_BUFS) & 1, ec, kSiteDrain, false);
#pragma unroll 1
      for (int s = 0; s < ST; ++s)
        if (nt > s) mbar_wait(bar(full + s), ((nt - 1 - s) / ST) & 1, ec, kSiteDrain, false);
    }
  } else if (warp == kSoftWarps + 1) {
    // ------------------------------------------------- S^T = K Q^T
    constexpr uint32_t kIdS = idesc_f16(128, N, BF16, false, false);
    const uint64_t dK0 = sdesc_sw128(sK, 16, 1024), dQ0 = sdesc_sw128(sQ, 16, 1024);
    int g = 0, q = 0, s = 0;  // tile, item with keys, stage
    uint32_t ph = 0;          // the stage's phase
    bool ok = true;
    PagedItem it;
    if (p.words != nullptr && run_lo < run_hi) {
      // While the first keys are on their way: the words that this run's parts will be
      // counted in at, those of the unit that it ends within, and of the one that it begins
      // within (where there are such).
      ok = paged_wait(bar(GB_START), 0, ec, kSiteFwdMma);
      if (ok && lane < 8) {
        int code = static_cast<int>(blockIdx.x) | 1 << 16;
        if (lane >= 4) {
          const PagedSpan sp = paged_span(p, start[2]);
          const int pos = start[1] % paged_weight(p, sp);
          if (sp.n > 0) {
            const int from = run_of(run_lo - pos + kPagedCost);
            code = from | (run_of(run_lo - pos + kPagedCost + sp.n - 1) - from + 1) << 16;
          }
        }
        const PagedParts c = paged_parts(p.words, code, lane & 1);
        if (c.first <= static_cast<int>(blockIdx.x)) paged_ready((lane & 2) != 0 ? c.unit : c.word, p.nonce);
        __threadfence();
      }
      __syncwarp();
    }
    for (int u = 0; ok && (ok = next_item(u, &it)); ++u) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(GB_IE + (u & 3)));
      if (it.n < 0) break;
      if (it.n == 0) continue;
      const int qb = q % C::Q_BUFS;
      if (!C::Q_WITH_K && !(ok = paged_wait(bar(GB_Q + qb), (q / C::Q_BUFS) & 1, ec, kSiteFwdMma))) break;
      const uint64_t dQ = desc_adv(dQ0, qb * C::Q_BYTES);
      for (int j = 0; j < it.n; ++j, ++g) {
        // S's buffer: P of the tile before the last one, formed from it, is there
        if (!(ok = paged_wait(bar(GB_P + (g & 1)), ((g >> 1) & 1) ^ 1, ec, kSiteFwdMma))) break;
        if (!(ok = paged_wait(bar(GB_KF + s), ph, ec, kSiteFwdMma))) break;
        tc_fence_after();
        const uint64_t dK = desc_adv(dK0, s * C::K_BYTES);
        if (elect_one_sync()) {
#pragma unroll
          for (int kk = 0; kk < DQK / 16; ++kk)
            umma_ss(tbase + C::T_S + N * (g & 1), desc_adv(dK, (kk >> 2) * (BN * 128) + (kk & 3) * 32),
                    desc_adv(dQ, (kk >> 2) * (N * 128) + (kk & 3) * 32), kIdS, kk > 0);
          umma_commit(bar(GB_S + (g & 1)));
          umma_commit(bar(GB_KE + s));
          if (!C::Q_WITH_K && j + 1 == it.n) umma_commit(bar(GB_QE + qb));
        }
        __syncwarp();
        if (++s == ST) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (!ok) break;
      ++q;
    }
    umma_commit_w(bar(GB_DRAIN));
    mbar_wait(bar(GB_DRAIN), 0, ec, kSiteDrain, false);
  } else if (warp == kSoftWarps + 3) {
    // ------------------------------------------------- O^T = V^T P^T
    constexpr uint32_t kIdO = idesc_f16(DV, NP, BF16, true, true);
    const uint64_t dV0 = sdesc_sw128(sV, BN * 128, 1024), dP0 = paged_desc_p(sP, C::P_PITCH);
    int g = 0, q = 0, s = 0;
    uint32_t ph = 0;
    bool ok = true;
    PagedItem it;
    for (int u = 0; (ok = next_item(u, &it)); ++u) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(GB_IE + (u & 3)));
      if (it.n < 0) break;
      if (it.n == 0) continue;
      const int ob = q & 1;
      // O's buffer has been read (of the item before the last one)
      if (!(ok = paged_wait(bar(GB_OE + ob), ((q >> 1) & 1) ^ 1, ec, kSiteFwdMma))) break;
      const int seen = p.left < 0 ? 0 : max(0, it.len - p.s_q - p.left);
      for (int j = 0; j < it.n; ++j, ++g) {
        if (!(ok = paged_wait(bar(GB_VF + s), ph, ec, kSiteFwdMma))) break;
        // Keys [lo, hi) of the tile are seen by some row. Only the steps of 16 keys that
        // hold one of them are multiplied; what such a step has besides (the page's rows
        // behind the last key, say) may be anything: its values are zeroed first.
        const int key0 = (it.k0 + j) * BN, lo = max(0, seen - key0), hi = min(BN, it.len - key0);
        const int k0 = lo / 16, k1 = (hi + 15) / 16;
        if (((lo | hi) & 15) != 0) {
          uint8_t* v = smem + C::OFF_V + s * C::V_BYTES;
          const int front = lo & 15, rows = front + (-hi & 15);
#pragma unroll 1
          for (int e = lane; e < rows * 8; e += 32) {
            const int r = e / 8 < front ? lo - front + e / 8 : hi + e / 8 - front;
#pragma unroll
            for (int c = 0; c < DV / 64; ++c)
              *reinterpret_cast<uint4*>(v + c * BN * 128 + r * 128 + (e & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (!(ok = paged_wait(bar(GB_P + (g & 1)), (g >> 1) & 1, ec, kSiteFwdMma))) break;
        tc_fence_after();
        const uint64_t dV = desc_adv(dV0, s * C::V_BYTES);
        const uint64_t dP = desc_adv(dP0, (C::P_BUFS == 2 ? (g & 1) : 0) * C::P_BYTES);
        const uint32_t dO = tbase + C::T_O + NP * (C::TURNS ? 2 * ob + (g & 1) : ob);
        const bool first = j < C::OS;  // of the tiles that this O sums
        if (elect_one_sync()) {
          if (k1 - k0 == BN / 16) {
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)
              umma_ss(dO, desc_adv(dV, kk * 2048), desc_adv(dP, kk * 16 * C::P_PITCH), kIdO, !first || kk > 0);
          } else {
#pragma unroll 1
            for (int kk = k0; kk < k1; ++kk)
              umma_ss(dO, desc_adv(dV, kk * 2048), desc_adv(dP, kk * 16 * C::P_PITCH), kIdO, !first || kk > k0);
          }
          umma_commit(bar(GB_PV + (g & 1)));
          umma_commit(bar(GB_VE + s));
          if (j + 1 == it.n) umma_commit(bar(GB_O + ob));
        }
        __syncwarp();
        if (++s == ST) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (!ok) break;
      ++q;
    }
    umma_commit_w(bar(GB_DRAIN + 1));
    mbar_wait(bar(GB_DRAIN + 1), 0, ec, kSiteDrain, false);
  } else {
    // -------------------------------------------------------------- softmax
    const int t = warp >> 2, w4 = warp & 3;
    const int col0 = C::TURNS ? 0 : t * NC;  // first row of this warpgroup
    const int own_key = w4 * 32 + lane;       // this thread's key of a tile
    const uint32_t own_lanes = static_cast<uint32_t>(w4 * 32) << 16;
    const uint32_t tS = tbase + C::T_S + col0 + own_lanes;
    // O of the item's tiles (turns: those of warpgroup w)
    auto tO = [&](int q, int w) {
      return tbase + C::T_O + NP * (C::TURNS ? 2 * (q & 1) + w : (q & 1)) + col0 + own_lanes;
    };
    float* gMax = sMax + t * 4 * NC;
    float* gRow = sRow + t * 4 * NC;
    float* wMax = gMax + w4 * NC;
    float* wRow = gRow + w4 * NC;
    const int own_row = lane & (NC - 1);
    const float sl2 = p.scale_log2;
    const float hide = sl2 < 0.f ? -SDPA_NEG_INF : SDPA_NEG_INF;  // masked raw score
    // 16-byte chunk of a key's row of P^T (0 .. NP / 8 - 1), as the swizzle has it
    const int flip = C::P_PITCH == 128 ? own_key & 7 : C::P_PITCH == 64 ? (own_key >> 1) & 3 : (own_key >> 2) & 1;
    uint8_t* own_p = smem + C::OFF_P + own_key * C::P_PITCH;
    auto chunk_at = [&](int c) {
      return C::P_PITCH == 128 ? (c >> 3) * BN * 128 + (((c & 7) ^ flip) << 4) : (c ^ flip) << 4;
    };
    // A vote of the warpgroup. A warp whose wait ran out votes no until all leave
    // together: after a no comes a second vote, on whether all are well.
    auto vote = [&](bool yes) { return named_bar_and(1 + t, 128, yes); };
    auto load = [&](uint32_t at, float (&x)[NC]) {
      if constexpr (NC == 32) {
        tmem_ld32f(at, x);
      } else if constexpr (NC == 16) {
        uint32_t r[16];
        tmem_ld16(at, r);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(r[e]);
      } else {
        uint32_t r[8];
        tmem_ld8(at, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(r[e]);
      }
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
    // P = 2^(y - m) of the log2 scores y. m need not be the row's maximum: what P is
    // rounded to has to hold it with all its bits, and fp32 the sums. fp16 wants m
    // within 2^8; bf16 has fp32's exponents, and 2^60 either way is fine, so it begins
    // with m = 0 where all scores that a row sees of its first tile lie within that,
    // without asking for their maximum, which takes the warpgroup longer than the
    // softmax of the tile.
    constexpr float kFar = BF16 ? 60.f : 8.f;
    // Factor of P's low part. fp16: P is at most 2^kFar, what its high part leaves 2^-12 of
    // that, so the low part at most 2^14; bf16 has fp32's exponents and needs none.
    constexpr float kLow = BF16 ? 1.f : 0x1p18f;
    constexpr float kNone = 1e30f;  // -m of a row without a score: any score then grows it
    int u = 0, g0 = 0, q = 0, pairs = 0;  // item, its first tile, items with keys, items of both warpgroups
    bool ok = true, left_all = false;
    PagedItem it;
    for (; (ok = next_item(u, &it)) && it.n >= 0; ++u) {
      const int base = it.rb * NR + col0;  // of the K/V head's rows
      const int live = min(NC, p.R - base);
      const int64_t row0 = (static_cast<int64_t>(it.b) * p.H_kv + it.hk) * p.R + base;
      if (it.n == 0) {  // a sequence without a key
#pragma unroll 1
        for (int e = C::TURNS ? warp : w4; e < live; e += C::TURNS ? 8 : 4) {
#pragma unroll 1
          for (int d = lane; d < DV / 2; d += 32) static_cast<uint32_t*>(p.o)[(row0 + e) * (DV / 2) + d] = 0u;
          if (lane == 0) p.lse[row0 + e] = SDPA_NEG_INF;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(GB_IE + (u & 3)));
        continue;
      }
      const int last0 = it.len - p.s_q;  // last key of token 0
      float nm[NC], l[NC], m = BF16 ? 0.f : SDPA_NEG_INF;  // -m and sums of this key's; m: of row `own_row`
#pragma unroll
      for (int e = 0; e < NC; ++e) {
        nm[e] = BF16 ? 0.f : kNone;
        l[e] = 0.f;
      }
      const int j0 = C::TURNS ? (g0 ^ t) & 1 : 0;
      const bool ends = !C::TURNS || ((g0 + it.n - 1) & 1) == t;  // this warpgroup writes the rows
      for (int j = j0; j < it.n; j += C::OS) {
        const int g = g0 + j, key0 = (it.k0 + j) * BN, key = key0 + own_key;
        const bool first = j == j0;
        if (ok) ok = paged_wait(bar(GB_S + (g & 1)), (g >> 1) & 1, ec, kSiteFwdSoftmax);
        tc_fence_after();
        float x[NC];
        load(tS + N * (g & 1), x);
        tmem_wait_ld();
        if (p.capped) {
#pragma unroll
          for (int e = 0; e < NC; ++e) x[e] = paged_tanh(x[e] * p.cap_in);
        }
        const bool hidden = key0 + BN - 1 > last0 || (p.left >= 0 && key0 < last0 + p.s_q - 1 - p.left);
        bool out = false;  // a key that no row sees
        if (hidden) {
          out = key > last0 + p.s_q - 1 || (p.left >= 0 && key < last0 - p.left);
          if (p.s_q > 1) {  // or that only some tokens see
            int tok = base % p.s_q;
#pragma unroll
            for (int e = 0; e < NC; ++e) {
              if (key > last0 + tok || (p.left >= 0 && key < last0 + tok - p.left)) x[e] = hide;
              tok = tok + 1 == p.s_q ? 0 : tok + 1;
            }
          } else {
#pragma unroll
            for (int e = 0; e < NC; ++e) x[e] = out ? hide : x[e];
          }
        }
        float most = SDPA_NEG_INF, least = -SDPA_NEG_INF;
#pragma unroll
        for (int e = 0; e < NC; ++e) {
          const float y = fmaf(x[e], sl2, nm[e]);
          most = fmaxf(most, y);
          if constexpr (BF16) least = fminf(least, y);
        }
        // (rows of several tokens see a tile's keys only in part: such a tile says nothing of
        // the rows that see none of it)
        bool fine = most <= kFar;
        if (first) fine = fine && BF16 && (out || least >= -kFar) && (p.s_q == 1 || !hidden);
        if (!vote(ok && fine)) {
          // ---- the rows' maxima, of all keys of the tile
          float mine = SDPA_NEG_INF;
#pragma unroll
          for (int e = 0; e < NC; ++e) {
            const float r = warp_max(x[e] * sl2);
            if (own_row == e) mine = r;
          }
          if (lane < NC) wMax[lane] = mine;
          if (!vote(ok)) {
            left_all = true;
            break;
          }
          const float mx = fmaxf(fmaxf(gMax[own_row], gMax[NC + own_row]),
                                 fmaxf(gMax[2 * NC + own_row], gMax[3 * NC + own_row]));
          if (first) m = SDPA_NEG_INF;
          float alpha = 1.f;
          if (mx > m + kFar) {
            alpha = ex2(m - mx);
            m = mx;
          }
          spread(wRow, m == SDPA_NEG_INF ? kNone : -m, nm);
          if (!first) {
            float al[NC], o[NC];
            spread(wRow, alpha, al);
            // (the product of the warpgroup's tile before this one is done)
            const int before = g - C::OS;
            if (ok) ok = paged_wait(bar(GB_PV + (before & 1)), (before >> 1) & 1, ec, kSiteFwdSoftmax);
            tc_fence_after();
#pragma unroll
            for (int e = 0; e < NC; ++e) l[e] *= al[e];
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // the high parts' O, the low parts'
              load(tO(q, t) + h * NR, o);
              tmem_wait_ld();
#pragma unroll
              for (int e0 = 0; e0 < NC; e0 += 8) {
                uint32_t r[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) r[e] = __float_as_uint(o[e0 + e] * al[e0 + e]);
                tmem_st8(tO(q, t) + h * NR + e0, r);
              }
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
            ok = paged_wait(bar(GB_PV + (g & 1)), ((g >> 1) & 1) ^ 1, ec, kSiteFwdSoftmax);
          else if (g > 0)
            ok = paged_wait(bar(GB_PV + ((g - 1) & 1)), ((g - 1) >> 1) & 1, ec, kSiteFwdSoftmax);
        }
        uint8_t* to = own_p + (C::P_BUFS == 2 ? (g & 1) : 0) * C::P_BYTES;
#pragma unroll
        for (int e = 0; e < NC; e += 8) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            hi[i] = pack2<BF16>(x[e + 2 * i], x[e + 2 * i + 1]);
            const float2 f = unpack2<BF16>(hi[i]);
            lo[i] = pack2<BF16>((x[e + 2 * i] - f.x) * kLow, (x[e + 2 * i + 1] - f.y) * kLow);
          }
          *reinterpret_cast<uint4*>(to + chunk_at((col0 + e) / 8)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(to + chunk_at((NR + col0 + e) / 8)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(GB_P + (g & 1)));
      }
      if (left_all) break;
      const bool both = C::TURNS && it.n > 1;
      if (j0 < it.n) {
        // ---- sums over the warp's keys: lane e gets row e's
#pragma unroll
        for (int o = NC / 2; o > 0; o >>= 1) {
          const bool hi = (lane & o) != 0;
#pragma unroll
          for (int e = 0; e < o; ++e) {
            const float send = hi ? l[e] : l[e + o], keep = hi ? l[e + o] : l[e];
            l[e] = keep + __shfl_xor_sync(0xffffffffu, send, o);
          }
        }
#pragma unroll
        for (int o = NC; o < 32; o *= 2) l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
        __syncwarp();
        if (lane < NC) wRow[lane] = l[0];
        if (!vote(ok)) {
          vote(false);
          left_all = true;
          break;
        }
        float sum_l = (gRow[own_row] + gRow[NC + own_row]) + (gRow[2 * NC + own_row] + gRow[3 * NC + own_row]);
        float* stat = sStat + (pairs & 3) * 2 * NR;
        if (ends) {
          // ---- the unit's rows: O / l, and the log of the sum of exponentials
          float c_own = 1.f, c_other = 0.f;
          if (both) {  // join the other warpgroup's tiles
            ok = paged_wait(bar(GB_ST + (pairs & 3)), (pairs >> 2) & 1, ec, kSiteFwdSoftmax);
            const float m2 = stat[own_row], l2 = stat[NR + own_row], top = fmaxf(m, m2);
            const float b = top == SDPA_NEG_INF ? 0.f : top;
            c_own = ex2(m - b);
            c_other = ex2(m2 - b);
            sum_l = sum_l * c_own + l2 * c_other;
            m = top;
          }
          const float inv = sum_l == 0.f ? 0.f : 1.f / sum_l;
          float c[NC], c2[NC], o[NC];
          spread(wMax, c_own * inv, c);
          if (both) spread(wMax, c_other * inv, c2);
          const float log_l = sum_l == 0.f ? SDPA_NEG_INF : m + __log2f(sum_l);
          if (w4 == 0 && lane < live) {
            if (it.slot < 0)
              p.lse[row0 + lane] = log_l * kLn2;
            else
              p.part_lse[it.slot * NR + col0 + lane] = log_l;
          }
          ok = paged_wait(bar(GB_O + (q & 1)), (q >> 1) & 1, ec, kSiteFwdSoftmax) && ok;
          tc_fence_after();
          auto take = [&](int w, const float (&f)[NC], bool add) {  // o (+)= f times warpgroup w's O
            float hi[NC], lo[NC];
            load(tO(q, w), hi);
            load(tO(q, w) + NR, lo);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < NC; ++e) {
              // (an infinite value times a low part of 0 or below would make it NaN)
              const float sum = fabsf(hi[e]) < -SDPA_NEG_INF ? fmaf(lo[e], 1.f / kLow, hi[e]) : hi[e];
              const float v = f[e] == 0.f ? 0.f : sum * f[e];
              o[e] = add ? o[e] + v : v;
            }
          };
          take(t, c, false);
          if (both) take(t ^ 1, c2, true);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(GB_OE + (q & 1)));
          // (64 value columns: the product's rows lie on each warp's first 16 lanes)
          const int d = DV == 128 ? own_key : w4 * 16 + lane;
          const bool has = DV == 128 || lane < 16;
          if (it.slot >= 0) {
            float* dst = p.part + static_cast<int64_t>(it.slot * NR + col0) * DV + d;
#pragma unroll
            for (int e = 0; e < NC; ++e)
              if (has && e < live) dst[e * DV] = o[e];
            // (in turns, either warpgroup has all rows)
            if (p.runs == nullptr &&
                !paged_join<DV, BF16, NR>(p.part, p.part_lse, p.words, static_cast<uint8_t*>(p.o) + row0 * (DV * 2),
                                          p.lse + row0, it.parts, C::TURNS ? 0 : t, 1 + t, col0, live, ok, sFlag + t)) {
              left_all = true;
              break;
            }
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
        } else if (w4 == 0) {
          if (lane < NR) {
            stat[lane] = m;
            stat[NR + lane] = sum_l;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(GB_ST + (pairs & 3)));
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(GB_IE + (u & 3)));
      ++q;
      g0 += it.n;
      if (both) ++pairs;
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

template <int DQK, int DV, bool BF16, int NR>
cudaError_t launch_paged_n(const CUtensorMap (&m)[3], const PagedParams& p, cudaStream_t st) {
  using C = PagedCfg<DQK, DV, NR>;
  auto kern = sdpa_paged_kernel<DQK, DV, BF16, NR>;
  const cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(kern), C::SMEM, 0);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.grid));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, m[0], m[1], m[2], p);
}

template <int DQK, int DV, bool BF16>
cudaError_t launch_paged_d(const CUtensorMap (&m)[3], const PagedParams& p, cudaStream_t st) {
  switch (paged_rows(p.R)) {
    case 8: return launch_paged_n<DQK, DV, BF16, 8>(m, p, st);
    case 16: return launch_paged_n<DQK, DV, BF16, 16>(m, p, st);
    case 32: return launch_paged_n<DQK, DV, BF16, 32>(m, p, st);
    default: return launch_paged_n<DQK, DV, BF16, 64>(m, p, st);
  }
}

}  // namespace sdpa
