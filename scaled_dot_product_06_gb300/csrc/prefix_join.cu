// Joins the partial rows of the shared-prefix attention:
//   L = log2 sum_s 2^L_s,  O = sum_s 2^(L_s - L) O_s,  LSE = L ln 2
// over the slots a row has: the prefix's, and as many of the own keys' as its
// sequence's length fills. A row without a key gets O = 0 and LSE = -inf.
// Bound by the latency of reading the partials, which the first kernel has
// just left in L2: WARPS warps share a row's slots where there are many.
#include "common.cuh"
#include "prefix.cuh"

namespace sdpa {

namespace {

// Slots are read in the same order by the same warp whatever else runs, so a
// call's result does not depend on timing.
template <bool BF16, int DV, int WARPS>
__global__ void __launch_bounds__(256) prefix_join_kernel(const PrefixParams p) {
  constexpr int ROWS = 8 / WARPS;   // rows a block
  constexpr int EL = DV / 32;       // elements a lane: 2 or 4
  __shared__ float s_acc[WARPS > 1 ? 8 : 1][DV];
  __shared__ float s_ml[WARPS > 1 ? 8 : 1][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + warp / WARPS;
  const int w = warp % WARPS;
  const bool live = row < p.rows;
  int n = 0;
  if (live) {
    n = p.slots_p;
    if (p.slots_o > 0) {
      const int b = static_cast<int>(row / (static_cast<int64_t>(p.H_kv) * p.R));
      const int keys = min(max(__ldg(p.seqlen + b), 0), p.s_max);
      n += ((keys + 127) / 128 + p.chunk_o - 1) / p.chunk_o * (p.dual_o ? 1 : 2);
    }
  }
  float m = SDPA_NEG_INF, l = 0.f, acc[EL];
#pragma unroll
  for (int e = 0; e < EL; ++e) acc[e] = 0.f;
  // 32 slots at a time, one L a lane: their weights are known before the rows
  // are read, so the reads do not wait for one another
  for (int s0 = w * 32; s0 < n; s0 += WARPS * 32) {
    const int cnt = min(32, n - s0);
    const float L = lane < cnt ? p.part_lse[(s0 + lane) * p.rows + row] : SDPA_NEG_INF;
    float mx = L;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mn = fmaxf(m, mx);
    if (mn == SDPA_NEG_INF) continue;
    const float keep = ex2(m - mn), wt = ex2(L - mn);
    m = mn;
    float sum = wt;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = fmaf(l, keep, sum);
#pragma unroll
    for (int e = 0; e < EL; ++e) acc[e] *= keep;
    const float* src = p.part + (s0 * p.rows + row) * DV + lane * EL;
#pragma unroll 8
    for (int i = 0; i < cnt; ++i) {
      const float wi = __shfl_sync(0xffffffffu, wt, i);
      const bool some = __shfl_sync(0xffffffffu, L, i) != SDPA_NEG_INF;  // else its O was not written
      float v[EL];
#pragma unroll
      for (int e = 0; e < EL; ++e) v[e] = 0.f;
      if (some) {
        if constexpr (EL == 4) {
          const float4 f = *reinterpret_cast<const float4*>(src + i * p.rows * DV);
          v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
        } else {
          const float2 f = *reinterpret_cast<const float2*>(src + i * p.rows * DV);
          v[0] = f.x, v[1] = f.y;
        }
      }
#pragma unroll
      for (int e = 0; e < EL; ++e) acc[e] = fmaf(wi, v[e], acc[e]);
    }
  }
  if constexpr (WARPS > 1) {
#pragma unroll
    for (int e = 0; e < EL; ++e) s_acc[warp][lane * EL + e] = acc[e];
    if (lane == 0) {
      s_ml[warp][0] = m;
      s_ml[warp][1] = l;
    }
    __syncthreads();
    if (w != 0) return;
    for (int i = 1; i < WARPS; ++i) {
      const float mo = s_ml[warp + i][0], lo = s_ml[warp + i][1];
      if (mo == SDPA_NEG_INF) continue;
      const float mn = fmaxf(m, mo);
      const float keep = ex2(m - mn), add = ex2(mo - mn);
      m = mn;
      l = fmaf(l, keep, lo * add);
#pragma unroll
      for (int e = 0; e < EL; ++e) acc[e] = fmaf(acc[e], keep, add * s_acc[warp + i][lane * EL + e]);
    }
  }
  if (!live) return;
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint8_t* dst = static_cast<uint8_t*>(p.o) + (row * DV + lane * EL) * 2;
  if constexpr (EL == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<BF16>(acc[0] * inv, acc[1] * inv),
                                                pack2<BF16>(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack2<BF16>(acc[0] * inv, acc[1] * inv);
  if (lane == 0) p.lse[row] = l > 0.f ? (m + __log2f(l)) * kLn2 : SDPA_NEG_INF;
}

template <bool BF16, int DV>
cudaError_t launch_join_d(const PrefixParams& p, cudaStream_t st) {
  // one warp reads 32 slots at a time
  if (p.slots_p + p.slots_o > 32)
    prefix_join_kernel<BF16, DV, 8><<<static_cast<unsigned>(p.rows), 256, 0, st>>>(p);
  else
    prefix_join_kernel<BF16, DV, 1><<<static_cast<unsigned>((p.rows + 7) / 8), 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefix_join(bool bf16, int d_v, const PrefixParams& p, cudaStream_t st) {
  if (d_v == 64) return bf16 ? launch_join_d<true, 64>(p, st) : launch_join_d<false, 64>(p, st);
  return bf16 ? launch_join_d<true, 128>(p, st) : launch_join_d<false, 128>(p, st);
}

}  // namespace sdpa
