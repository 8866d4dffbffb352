// Joins the partial rows of units that runs' ends have cut into many (paged_kernel.cuh):
//   L = log2 sum_s 2^L_s,  O = sum_s 2^(L_s - L) O_s,  LSE = L ln 2.
// A block has one row of one run: it works if the run begins within a unit that
// also ends in it, and then joins all slots of the unit, in the order of their
// runs whatever else runs. The slots are in L2, just written; their latency is all
// there is to it, so the warps share them and each lane reads 16 bytes of a slot's
// row, four slots at once.
#include "common.cuh"
#include "paged.cuh"

namespace sdpa {

namespace {

constexpr int kJoinWarps = 8;

template <bool BF16, int DV>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_join_kernel(const __grid_constant__ PagedParams p, int rows) {
  constexpr int LANES = DV / 4, PER = 32 / LANES;  // lanes a slot's row, slots a warp reads side by side
  __shared__ int slots[kPagedGrid];
  __shared__ int count[kJoinWarps];
  __shared__ float4 s_acc[kJoinWarps * PER][LANES];
  __shared__ float s_m[kJoinWarps * PER], s_l[kJoinWarps * PER];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x, x = blockIdx.y;
  // (the next call's kernel may come: it waits for this one's end before it touches memory)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the partials are written
  const int4 mine = __ldcg(p.runs + c);
  if (mine.x == 0 || mine.y == 0) return;
  const int unit = mine.x - 1, rb = unit % p.row_blocks;
  const int row = rb * rows + x;  // of the K/V head's
  if (row >= p.R) return;
  // the unit's slots, in the order of their runs (run i by thread i)
  static_assert(kPagedGrid <= kJoinWarps * 32, "a thread each");
  int slot = -1;
  if (threadIdx.x <= c) {
    const int4 r = __ldcg(p.runs + threadIdx.x);
    slot = r.x == mine.x ? 2 * threadIdx.x : r.z == mine.x ? 2 * threadIdx.x + 1 : -1;
  }
  const unsigned has = __ballot_sync(0xffffffffu, slot >= 0);
  if (lane == 0) count[warp] = __popc(has);
  __syncthreads();
  int at = 0, n = 0;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    if (w < warp) at += count[w];
    n += count[w];
  }
  if (slot >= 0) slots[at + __popc(has & ((1u << lane) - 1u))] = slot;
  __syncthreads();
  const int sub = lane / LANES, l4 = lane % LANES;
  float m = SDPA_NEG_INF, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = warp * PER + sub; s0 < n; s0 += 4 * kJoinWarps * PER) {
    float4 v[4];
    float L[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = s0 + i * kJoinWarps * PER;
      const int64_t r = static_cast<int64_t>(slots[min(s, n - 1)]) * rows + x;
      v[i] = __ldcg(reinterpret_cast<const float4*>(p.part + r * DV) + l4);
      L[i] = s < n ? __ldcg(p.part_lse + r) : SDPA_NEG_INF;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // (a maximum that skips what is not a number: the weight then is none, and the row)
      const float mn = fmaxf(m, L[i]), base = mn == SDPA_NEG_INF ? 0.f : mn;
      const float keep = ex2(m - base), w = ex2(L[i] - base);
      m = mn;
      l = fmaf(l, keep, w);
      const bool some = w > 0.f;
      acc.x = fmaf(w, some ? v[i].x : 0.f, acc.x * keep), acc.y = fmaf(w, some ? v[i].y : 0.f, acc.y * keep);
      acc.z = fmaf(w, some ? v[i].z : 0.f, acc.z * keep), acc.w = fmaf(w, some ? v[i].w : 0.f, acc.w * keep);
    }
  }
  const int part = warp * PER + sub;
  s_acc[part][l4] = acc;
  if (l4 == 0) {
    s_m[part] = m;
    s_l[part] = l;
  }
  __syncthreads();
  if (threadIdx.x >= LANES) return;
  float mt = SDPA_NEG_INF;
#pragma unroll
  for (int i = 0; i < kJoinWarps * PER; ++i) mt = fmaxf(mt, s_m[i]);
  const float base = mt == SDPA_NEG_INF ? 0.f : mt;
  float lt = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kJoinWarps * PER; ++i) {
    const float w = ex2(s_m[i] - base);
    const float4 a = s_acc[i][l4];
    lt = fmaf(w, s_l[i], lt);
    acc.x = fmaf(w, a.x, acc.x), acc.y = fmaf(w, a.y, acc.y), acc.z = fmaf(w, a.z, acc.z), acc.w = fmaf(w, a.w, acc.w);
  }
  const float inv = lt == 0.f ? 0.f : 1.f / lt;
  const int64_t out = static_cast<int64_t>(unit / p.row_blocks) * p.R + row;
  reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.o) + out * DV * 2)[l4] =
      make_uint2(pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
  if (l4 == 0) p.lse[out] = lt == 0.f ? SDPA_NEG_INF : (mt + __log2f(lt)) * kLn2;
}

}  // namespace

cudaError_t launch_paged_join(bool bf16, int d_v, const PagedParams& p, cudaStream_t st) {
  const int rows = paged_rows(p.R);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.grid), static_cast<unsigned>(p.R < rows ? p.R : rows));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = st;
  // the launch itself overlaps the end of the kernel that leaves the partials
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (d_v == 64)
    return cudaLaunchKernelEx(&cfg, bf16 ? paged_join_kernel<true, 64> : paged_join_kernel<false, 64>, p, rows);
  return cudaLaunchKernelEx(&cfg, bf16 ? paged_join_kernel<true, 128> : paged_join_kernel<false, 128>, p, rows);
}

}  // namespace sdpa
