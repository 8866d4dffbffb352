// Joins the partial rows of the shared-prefix attention:
//   L = log2 sum_s 2^L_s,  O = sum_s 2^(L_s - L) O_s,  LSE = L ln 2
// over the slots a row has: the prefix's, and as many of the own keys' as its
// sequence's length fills. A row without a key gets O = 0 and LSE = -inf; a row
// with an L that is not a number (it sees such a score) is none itself.
// Bound by the latency of reading the partials, which the first kernel has
// just left in L2: a warp has 8 rows and 32 columns, whose partials are one line
// a column group (prefix_part_index), and reads 8 slots of them at once; warps
// share the slots where there are more. (A warp per row, its slots one after
// another behind their weights, took 45 us of 38 slots of 2048 rows d128 for
// 6 us now.)
#include "common.cuh"
#include "prefix.cuh"

namespace sdpa {

namespace {

// Slots are read in the same order by the same warp whatever else runs, so a
// call's result does not depend on timing.
template <bool BF16, int DV, int WARPS>
__global__ void __launch_bounds__(256) prefix_join_kernel(const PrefixParams p) {
  constexpr int UNITS = 8 / WARPS;  // slabs' column parts a block
  __shared__ float4 s_acc[WARPS > 1 ? 8 : 1][64];
  __shared__ float s_ml[WARPS > 1 ? 8 : 1][8][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * UNITS + warp / WARPS;
  const int w = warp % WARPS;
  constexpr int PARTS = DV / 32;
  const int64_t row = unit / PARTS * 8 + (lane & 7);    // this lane's row
  const int c0 = static_cast<int>(unit % PARTS) * 8 + (lane >> 3);  // its column groups: c0, c0 + 4
  const bool live = row < p.rows;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the partials are written
  int n = 0;  // slots of the row
  if (live) {
    n = p.slots_p;
    if (p.slots_o > 0) {
      const int b = static_cast<int>(row / (static_cast<int64_t>(p.H_kv) * p.R));
      const int keys = min(max(__ldg(p.seqlen + b), 0), p.s_max);
      const int tiles = (keys + 127) / 128, chunks = (tiles + p.chunk_o - 1) / p.chunk_o;
      n += chunks * (p.dual_o ? 1 : p.quart_o ? 8 : 2);
      // an item of one key tile: warpgroup 1 has none, nor have warps behind the last key
      if (!p.dual_o && chunks > 0 && tiles - (chunks - 1) * p.chunk_o == 1)
        n -= p.quart_o ? 8 - ((keys - 1) % 128 / 32 + 1) : 1;
    }
  }
  int most = n;  // of the slab's rows
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  float m = SDPA_NEG_INF, l = 0.f;
  float4 a0 = make_float4(0.f, 0.f, 0.f, 0.f), a1 = a0;
  const float4* part = reinterpret_cast<const float4*>(p.part) + c0 * 8;
  for (int s0 = w * 8; s0 < most; s0 += WARPS * 8) {
    // 8 slots, all read before their weights are known, and left out where the
    // row has none (what was not written may be NaN)
    float4 v0[8], v1[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4* at = part + prefix_part_index(min(s0 + i, most - 1), p.rows, min(row, p.rows - 1), DV);
      v0[i] = __ldcg(at);
      v1[i] = __ldcg(at + 32);
    }
    // lane: slots s0 + (lane >> 3) and 4 further of its row
    const int i0 = s0 + (lane >> 3), i1 = i0 + 4;
    const float L0 = i0 < n ? __ldcg(p.part_lse + i0 * p.rows + row) : SDPA_NEG_INF;
    const float L1 = i1 < n ? __ldcg(p.part_lse + i1 * p.rows + row) : SDPA_NEG_INF;
    float mx = fmaxf(L0, L1);
#pragma unroll
    for (int o = 16; o > 4; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mn = fmaxf(m, mx), base = mn == SDPA_NEG_INF ? 0.f : mn;
    const float keep = ex2(m - base), w0 = ex2(L0 - base), w1 = ex2(L1 - base);
    m = mn;
    l *= keep;
    a0.x *= keep, a0.y *= keep, a0.z *= keep, a0.w *= keep;
    a1.x *= keep, a1.y *= keep, a1.z *= keep, a1.w *= keep;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float wi = __shfl_sync(0xffffffffu, i < 4 ? w0 : w1, (i & 3) * 8 + (lane & 7));
      l += wi;
      const bool some = wi > 0.f;  // (not a number: O_s is not there, the row is none by the weight)
      a0.x = fmaf(wi, some ? v0[i].x : 0.f, a0.x), a0.y = fmaf(wi, some ? v0[i].y : 0.f, a0.y);
      a0.z = fmaf(wi, some ? v0[i].z : 0.f, a0.z), a0.w = fmaf(wi, some ? v0[i].w : 0.f, a0.w);
      a1.x = fmaf(wi, some ? v1[i].x : 0.f, a1.x), a1.y = fmaf(wi, some ? v1[i].y : 0.f, a1.y);
      a1.z = fmaf(wi, some ? v1[i].z : 0.f, a1.z), a1.w = fmaf(wi, some ? v1[i].w : 0.f, a1.w);
    }
  }
  if constexpr (WARPS > 1) {
    s_acc[warp][lane] = a0;
    s_acc[warp][lane + 32] = a1;
    if (lane < 8) {
      s_ml[warp][lane][0] = m;
      s_ml[warp][lane][1] = l;
    }
    __syncthreads();
    if (w != 0) return;
    for (int i = 1; i < WARPS; ++i) {
      const float mo = s_ml[warp + i][lane & 7][0], lo = s_ml[warp + i][lane & 7][1];
      const float mn = fmaxf(m, mo), base = mn == SDPA_NEG_INF ? 0.f : mn;
      const float keep = ex2(m - base), add = ex2(mo - base);
      m = mn;
      l = fmaf(l, keep, lo * add);
      const float4 b0 = s_acc[warp + i][lane], b1 = s_acc[warp + i][lane + 32];
      a0.x = fmaf(a0.x, keep, add * b0.x), a0.y = fmaf(a0.y, keep, add * b0.y);
      a0.z = fmaf(a0.z, keep, add * b0.z), a0.w = fmaf(a0.w, keep, add * b0.w);
      a1.x = fmaf(a1.x, keep, add * b1.x), a1.y = fmaf(a1.y, keep, add * b1.y);
      a1.z = fmaf(a1.z, keep, add * b1.z), a1.w = fmaf(a1.w, keep, add * b1.w);
    }
  }
  if (!live) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint2* dst = reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.o) + row * DV * 2);
  dst[c0] = make_uint2(pack2<BF16>(a0.x * inv, a0.y * inv), pack2<BF16>(a0.z * inv, a0.w * inv));
  dst[c0 + 4] = make_uint2(pack2<BF16>(a1.x * inv, a1.y * inv), pack2<BF16>(a1.z * inv, a1.w * inv));
  if (c0 == 0) p.lse[row] = l == 0.f ? SDPA_NEG_INF : (m + __log2f(l)) * kLn2;
}

template <bool BF16, int DV>
cudaError_t launch_join_d(const PrefixParams& p, cudaStream_t st) {
  // a warp reads 8 slots at a time; more than that are shared by up to 8 warps
  const int n = p.slots_p + p.slots_o;
  const int warps = n <= 8 ? 1 : n <= 16 ? 2 : n <= 32 ? 4 : 8;
  auto kern = warps == 1   ? prefix_join_kernel<BF16, DV, 1>
              : warps == 2 ? prefix_join_kernel<BF16, DV, 2>
              : warps == 4 ? prefix_join_kernel<BF16, DV, 4>
                           : prefix_join_kernel<BF16, DV, 8>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(((p.rows + 7) / 8 * (DV / 32) * warps + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  // the launch itself overlaps the end of the kernel that leaves the partials
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = p.items_prefix + p.items_own > 0 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

__global__ void prefix_zero_kernel(int* n) { *n = 0; }

}  // namespace

cudaError_t launch_prefix_zero(const PrefixParams& p, cudaStream_t st) {
  prefix_zero_kernel<<<1, 1, 0, st>>>(p.next);
  return cudaGetLastError();
}

cudaError_t launch_prefix_join(bool bf16, int d_v, const PrefixParams& p, cudaStream_t st) {
  if (d_v == 64) return bf16 ? launch_join_d<true, 64>(p, st) : launch_join_d<false, 64>(p, st);
  return bf16 ? launch_join_d<true, 128>(p, st) : launch_join_d<false, 128>(p, st);
}

}  // namespace sdpa
