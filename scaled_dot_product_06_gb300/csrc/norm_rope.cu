// Norms of queries and keys for each head with the position rotation, from the
// projection's layout to the attention's, and its backward.
//
// Forward, per row x of a head (d elements):
//   u = x * (mean(x^2) + eps)^-1/2 * w     (u = x without a weight)
//   y = R(pos) u: the first rot elements turned in pairs by the table's angles,
//       pairs (i, i + rot/2), or (2i, 2i + 1) when interleaved
// Backward, with g = R^T dy, xh = x r, r = (mean(x^2) + eps)^-1/2:
//   dx = r (g w - xh mean(g w xh)),   dw = sum over rows of g xh
// Everything between load and store is fp32; each output is rounded once.
//
// Both are bound by memory: each row is read once and written once (the
// backward reads x and dy). A row is spread over d / 8 lanes, 16 bytes each, so
// a warp holds a row each of 4, 2 or 1 consecutive tokens (d = 64, 128, 192)
// and walks `seg` heads of them: the angles, and their products with the
// weights, are formed once for those. Rows come through a ring of cp.async
// copies, each thread its own 16 bytes and reading back only those (no
// barrier), so the loads in flight hold no registers: with plain loads, four
// rows a thread ahead of their use, a call at b1 s16384 h32 + 2 x 4, d = 128
// took 74 us (68% of the copy rate; now 59 us, 85%) and its backward at b4
// s2048, 3 x 16 heads, 113 us (36%; now 65 us, 62%: no unit is near its limit,
// but a warp takes one row at a time, and wait for the copy, the partner's
// elements, four rounds of two sums' shuffles, the root and the store follow one
// another, 24 warps an SM). Shorter walks than 16 heads lose more to the angles
// than they gain in grain: 65 us at 8, 72 us at 4, for 60 us of the kernel alone.
#include <algorithm>

#include "common.cuh"
#include "norm_rope.cuh"

namespace sdpa {

namespace {

constexpr int kThreads = 256;

template <int D>
struct RowCfg {
  static constexpr int L = D / 8;          // lanes a row
  static constexpr int RPW = 32 / L;       // rows a warp
  static constexpr int WARPS = kThreads / 32;
};

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2<BF16>(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]), pack2<BF16>(x[4], x[5]),
                    pack2<BF16>(x[6], x[7]));
}

// Sum over the L lanes of a row (L = 24: over the warp, whose last 8 lanes hold 0).
template <int L>
__device__ __forceinline__ float row_sum(float v) {
  constexpr int W = L == 24 ? 32 : L;
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A lane's part of the turn of its row's elements e = [8 l, 8 l + 8): with the
// partner's elements p (of another lane, or its own pairs when interleaved)
// y = c u + s p. Lanes past rot keep their elements (c = 1, s = 0).
struct Turn {
  float c[8], s[8];
  int partner;  // lane of the partner's elements (half-split), else the lane itself
};

__device__ __forceinline__ Turn load_turn(const NormRopeParams& p, bool rotate, int64_t pos, int l, int lane) {
  Turn r;
  r.partner = lane;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    r.c[i] = 1.f;
    r.s[i] = 0.f;
  }
  if (rotate && 8 * l < p.rot) {
    pos = pos < 0 ? 0 : (pos >= p.n_pos ? p.n_pos - 1 : pos);
    const int half = p.rot / 2;
    const float* cr = p.cos + pos * half;
    const float* sr = p.sin + pos * half;
    if (p.interleaved) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(cr) + l);
      const float4 s = __ldg(reinterpret_cast<const float4*>(sr) + l);
      const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r.c[2 * i] = r.c[2 * i + 1] = cc[i];
        r.s[2 * i] = -ss[i];
        r.s[2 * i + 1] = ss[i];
      }
    } else {
      const bool second = 8 * l >= half;
      const int i0 = 8 * l - (second ? half : 0);
      r.partner = lane + (second ? -half / 8 : half / 8);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(cr + i0) + q);
        const float4 s = __ldg(reinterpret_cast<const float4*>(sr + i0) + q);
        const float m = second ? 1.f : -1.f;
        r.c[4 * q] = c.x, r.c[4 * q + 1] = c.y, r.c[4 * q + 2] = c.z, r.c[4 * q + 3] = c.w;
        r.s[4 * q] = m * s.x, r.s[4 * q + 1] = m * s.y, r.s[4 * q + 2] = m * s.z, r.s[4 * q + 3] = m * s.w;
      }
    }
  }
  return r;
}

// The partner's elements of a row given as 8 packed elements a lane: its own
// pairs swapped, or the partner lane's. Every lane of the warp calls it.
template <bool BF16>
__device__ __forceinline__ void partner8(bool interleaved, int partner, const uint4& v, float (&x)[8]) {
  uint4 p;
  if (interleaved) {
    p = make_uint4(__funnelshift_l(v.x, v.x, 16), __funnelshift_l(v.y, v.y, 16), __funnelshift_l(v.z, v.z, 16),
                   __funnelshift_l(v.w, v.w, 16));
  } else {
    p = make_uint4(__shfl_sync(0xffffffffu, v.x, partner), __shfl_sync(0xffffffffu, v.y, partner),
                   __shfl_sync(0xffffffffu, v.z, partner), __shfl_sync(0xffffffffu, v.w, partner));
  }
  unpack8<BF16>(p, x);
}

template <bool BF16>
__device__ __forceinline__ void load_weight(const NormRopeParams& p, const RowKind& k, int l, bool live,
                                            float (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.f;
  if (k.weight == nullptr || !live) return;
  if (p.weight_fp32) {
    const float4* w4 = static_cast<const float4*>(k.weight) + 2 * l;
    const float4 a = __ldg(w4), b = __ldg(w4 + 1);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  } else {
    unpack8<BF16>(__ldg(static_cast<const uint4*>(k.weight) + l), w);
  }
}

__device__ __forceinline__ int kind_of_block(const NormRopeParams& p, int block) {
  int k = 0;
  while (k + 1 < p.n_kinds && block >= p.kind[k + 1].block0) ++k;
  return k;
}

// 16 bytes from global to shared memory; zeros (no read) when not live.
__device__ __forceinline__ void copy16(uint4* dst, const uint16_t* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A warp's walk: work unit u of its kind is head segment u / n_tb of token block
// u % n_tb (RPW consecutive tokens, one a lane group).
struct Unit {
  int b, t, h0, n;  // sequence, token, first head, heads
  int64_t token;
  bool live;        // this lane moves data
};
template <int RPW>
__device__ __forceinline__ Unit unit_of(const NormRopeParams& p, const RowKind& k, uint32_t u, int sub,
                                        bool lane_ok) {
  const uint32_t n_tb = static_cast<uint32_t>((p.tokens + RPW - 1) / RPW);
  const uint32_t sg = u / n_tb, tb = u - sg * n_tb;
  Unit r;
  const uint32_t tok = tb * RPW + sub;
  r.live = lane_ok && tok < p.tokens;
  const uint32_t tk = r.live ? tok : 0;
  r.token = tk;
  r.b = static_cast<int>(tk / static_cast<uint32_t>(p.s));
  r.t = static_cast<int>(tk - static_cast<uint32_t>(r.b) * static_cast<uint32_t>(p.s));
  r.h0 = static_cast<int>(sg) * p.seg;
  r.n = min(p.seg, k.heads - r.h0);
  return r;
}

constexpr int kRing = 8;  // rows a thread has in flight

template <bool BF16, int D>
__global__ void __launch_bounds__(kThreads, 4) norm_rope_fwd_kernel(const __grid_constant__ NormRopeParams p) {
  using C = RowCfg<D>;
  __shared__ uint4 ring[kRing][kThreads];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / C::L, l = lane - sub * C::L;  // row of the warp, lane of the row
  const RowKind& k = p.kind[kind_of_block(p, blockIdx.x)];
  const uint32_t u = (blockIdx.x - k.block0) * C::WARPS + warp;
  if (u >= k.units) return;  // whole warps
  const Unit un = unit_of<C::RPW>(p, k, u, sub, sub < C::RPW && 8 * l < k.width);
  const uint16_t* src = static_cast<const uint16_t*>(k.token.ptr) + un.b * k.token.sb + un.t * k.token.st +
                        un.h0 * k.token.sh + 8 * l;
#pragma unroll
  for (int i = 0; i < kRing; ++i) {
    if (i < un.n) copy16(&ring[i][threadIdx.x], src + i * k.token.sh, un.live);
    copy_commit();
  }
  int64_t row = un.t;
  bool store = un.live;
  if (k.cached) {
    row += un.live ? __ldg(p.kv_rows + un.b) : 0;
    store = un.live && row >= 0 && row < p.cache_rows;
  }
  uint16_t* dst = static_cast<uint16_t*>(k.head.ptr) + un.b * k.head.sb + row * k.head.st + un.h0 * k.head.sh + 8 * l;
  const bool normed = k.weight != nullptr, rotate = k.rotate != 0;
  const int64_t pos = (rotate && p.positions != nullptr && un.live) ? __ldg(p.positions + un.token) : un.t;
  float cw[8], sw[8];  // the angles times the weights of the element and of its partner
  load_weight<BF16>(p, k, l, un.live, cw);
  const Turn turn = load_turn(p, rotate && un.live, pos, l, lane);
#pragma unroll
  for (int e = 0; e < 8; ++e) sw[e] = p.interleaved ? cw[e ^ 1] : __shfl_sync(0xffffffffu, cw[e], turn.partner);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    cw[e] *= turn.c[e];
    sw[e] *= turn.s[e];
  }
#pragma unroll 1
  for (int i = 0; i < un.n; ++i) {
    copy_wait<kRing - 1>();
    uint4* slot = &ring[i % kRing][threadIdx.x];
    uint4 v = *slot;
    if (normed || rotate) {  // uniform over the block
      float x[8], r = 1.f;
      unpack8<BF16>(v, x);
      if (normed) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
        r = rsqrtf(row_sum<C::L>(ss) * (1.f / D) + p.eps);
      }
      if (rotate) {
        float y[8];
        partner8<BF16>(p.interleaved, turn.partner, v, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = r * fmaf(cw[e], x[e], sw[e] * y[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = r * (cw[e] * x[e]);
      }
      v = pack8<BF16>(x);
    }
    if (store) *reinterpret_cast<uint4*>(dst) = v;
    dst += k.head.sh;
    if (i + kRing < un.n) copy16(slot, src + (i + kRing) * k.token.sh, un.live);
    copy_commit();
  }
}

template <bool BF16, int D>
__global__ void __launch_bounds__(kThreads, 3) norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p) {
  using C = RowCfg<D>;
  extern __shared__ uint4 bwd_ring[];  // [kRing][dy, x][kThreads]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / C::L, l = lane - sub * C::L;
  const int ki = kind_of_block(p, blockIdx.x);
  const RowKind& k = p.kind[ki];
  const RowSet& xs = p.x[ki];
  const uint32_t step = ((ki + 1 < p.n_kinds ? p.kind[ki + 1].block0 : gridDim.x) - k.block0) * C::WARPS;
  const bool lane_ok = sub < C::RPW && 8 * l < k.width;
  const bool normed = k.weight != nullptr, rotate = k.rotate != 0;
  float w[8], dw[8];
  load_weight<BF16>(p, k, l, lane_ok, w);
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[e] = 0.f;
  // the copies run ahead of the arithmetic by kRing rows, across units
  const uint32_t u0 = (blockIdx.x - k.block0) * C::WARPS + warp;
  uint32_t cu = u0;  // unit, row, and pointers of the next copy
  int ci = 0, cn = 0, slot_in = 0;
  bool c_live = false;
  const uint16_t *cg = nullptr, *cx = nullptr;
  auto copy_unit = [&]() {
    const Unit un = unit_of<C::RPW>(p, k, cu, sub, lane_ok);
    ci = 0;
    cn = un.n;
    c_live = un.live;
    cg = static_cast<const uint16_t*>(k.head.ptr) + un.b * k.head.sb + un.t * k.head.st + un.h0 * k.head.sh + 8 * l;
    if (normed)
      cx = static_cast<const uint16_t*>(xs.ptr) + un.b * xs.sb + un.t * xs.st + un.h0 * xs.sh + 8 * l;
  };
  if (cu < k.units) copy_unit();
  auto copy_next = [&]() {
    if (cu < k.units) {  // uniform over the warp
      uint4* slot = bwd_ring + (2 * slot_in) * kThreads + threadIdx.x;
      copy16(slot, cg, c_live);
      cg += k.head.sh;
      if (normed) {
        copy16(slot + kThreads, cx, c_live);
        cx += xs.sh;
      }
      if (++ci == cn) {
        cu += step;
        if (cu < k.units) copy_unit();
      }
    }
    copy_commit();
    slot_in = (slot_in + 1) % kRing;
  };
#pragma unroll 1
  for (int i = 0; i < kRing; ++i) copy_next();
  int slot_out = 0;
#pragma unroll 1
  for (uint32_t u = u0; u < k.units; u += step) {
    const Unit un = unit_of<C::RPW>(p, k, u, sub, lane_ok);
    const int64_t pos = (rotate && p.positions != nullptr && un.live) ? __ldg(p.positions + un.token) : un.t;
    const Turn turn = load_turn(p, rotate && un.live, pos, l, lane);
    uint16_t* dst = static_cast<uint16_t*>(k.token.ptr) + un.b * k.token.sb + un.t * k.token.st +
                    un.h0 * k.token.sh + 8 * l;
#pragma unroll 1
    for (int i = 0; i < un.n; ++i) {
      copy_wait<kRing - 1>();
      const uint4* slot = bwd_ring + (2 * slot_out) * kThreads + threadIdx.x;
      slot_out = (slot_out + 1) % kRing;
      uint4 v = slot[0];
      if (normed || rotate) {  // uniform over the block
        float g[8];
        unpack8<BF16>(v, g);
        if (rotate) {  // the transpose: the other way round
          float y[8];
          partner8<BF16>(p.interleaved, turn.partner, v, y);
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] = fmaf(-turn.s[e], y[e], turn.c[e] * g[e]);
        }
        if (normed) {
          float x[8], ss = 0.f, gx = 0.f;
          unpack8<BF16>(slot[kThreads], x);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            ss = fmaf(x[e], x[e], ss);
            gx = fmaf(g[e] * w[e], x[e], gx);
          }
          // (r^3, which an expanded form would need, overflows for tiny eps)
          const float r = rsqrtf(row_sum<C::L>(ss) * (1.f / D) + p.eps);
          const float m = row_sum<C::L>(gx) * (1.f / D) * r;  // mean(g w xh)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float xh = x[e] * r;
            dw[e] = fmaf(g[e], xh, dw[e]);
            g[e] = r * fmaf(-xh, m, g[e] * w[e]);
          }
        }
        v = pack8<BF16>(g);
      }
      if (un.live) *reinterpret_cast<uint4*>(dst) = v;
      dst += k.token.sh;
      copy_next();
    }
  }
  if (!normed) return;  // uniform over the block
  copy_wait<0>();
  __syncthreads();  // every warp is done with the ring
  float* part = reinterpret_cast<float*>(bwd_ring);  // [GROUPS][D]
  if (sub < C::RPW) {
#pragma unroll
    for (int e = 0; e < 8; ++e) part[(warp * C::RPW + sub) * D + 8 * l + e] = dw[e];
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float s = 0.f;
#pragma unroll
    for (int g = 0; g < C::WARPS * C::RPW; ++g) s += part[g * D + threadIdx.x];
    p.dw_part[static_cast<int64_t>(blockIdx.x) * D + threadIdx.x] = s;
  }
}
constexpr int kBwdSmem = kRing * 2 * kThreads * 16;

// dw[j] = sum of n partial rows in a fixed order: 32 columns a block, 32 threads a column.
template <bool BF16>
__global__ void __launch_bounds__(1024) dw_reduce_kernel(const float* __restrict__ part, int d, int q0, int k0,
                                                         int k1, int fp32, void* dw_q, void* dw_k) {
  __shared__ float sum[32][33];
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
  const bool keys = blockIdx.y != 0;
  void* dw = keys ? dw_k : dw_q;
  if (dw == nullptr) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the partial rows are written
  float s = 0.f;
  for (int i = (keys ? k0 : q0) + r; i < (keys ? k1 : k0); i += 32) s += part[static_cast<int64_t>(i) * d + col];
  sum[r][c] = s;
  __syncthreads();
  float v = sum[c][r];  // column r of the block, row c
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (c == 0) {
    const int j = blockIdx.x * 32 + r;
    if (fp32)
      static_cast<float*>(dw)[j] = v;
    else
      static_cast<uint16_t*>(dw)[j] = static_cast<uint16_t>(pack2<BF16>(v, 0.f) & 0xffffu);
  }
}

template <bool BF16, int D>
cudaError_t launch_fwd_d(const NormRopeParams& p, int blocks, cudaStream_t st) {
  norm_rope_fwd_kernel<BF16, D><<<blocks, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <bool BF16, int D>
cudaError_t launch_bwd_d(const NormRopeParams& p, int blocks, cudaStream_t st) {
  auto kern = norm_rope_bwd_kernel<BF16, D>;
  const cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(kern), kBwdSmem, 0);
  if (e != cudaSuccess) return e;
  kern<<<blocks, kThreads, kBwdSmem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

int norm_rope_plan(NormRopeParams* p, bool backward) {
  constexpr int W = kThreads / 32;
  const int rpw = p->d == 64 ? RowCfg<64>::RPW : (p->d == 128 ? RowCfg<128>::RPW : RowCfg<192>::RPW);
  const int64_t n_tb = (p->tokens + rpw - 1) / rpw;
  // heads a warp walks: sixteen, or the largest power of two below that leaves
  // 32 warps an SM
  auto warps = [&](int seg) {
    int64_t n = 0;
    for (int i = 0; i < p->n_kinds; ++i) n += n_tb * ((p->kind[i].heads + seg - 1) / seg);
    return n;
  };
  p->seg = 16;
  while (p->seg > 1 && warps(p->seg) < 32 * 152) p->seg /= 2;
  // the time of a kind's rows: with a norm backward 3 rows move and the sums
  // are taken, else 2 rows move
  auto cost = [&](int i) -> int64_t { return p->kind[i].heads * (p->kind[i].weight != nullptr ? 4 : 2); };
  int64_t need[3] = {0, 0, 0}, all = 0;
  for (int i = 0; i < p->n_kinds; ++i) {
    const int64_t units = n_tb * ((p->kind[i].heads + p->seg - 1) / p->seg);
    if (units >= (int64_t{1} << 31)) return -1;
    p->kind[i].units = static_cast<uint32_t>(units);
    need[i] = (units + W - 1) / W;
    all += cost(i);
  }
  // the backward's blocks loop, each leaving one partial row of dw: the three
  // resident an SM, shared among the kinds by their time (by their rows, b4 s2048
  // of 3 x 16 heads d128 took 67 us for 60: the values' blocks ended early)
  const int64_t most = 3 * 152;
  int64_t at = 0;
  for (int i = 0; i < p->n_kinds; ++i) {
    p->kind[i].block0 = static_cast<int>(at);
    const int64_t share = std::max<int64_t>(1, (most * cost(i) + all / 2) / all);
    at += backward ? std::min(need[i], share) : need[i];
    if (at > 0x7fffffff) return -1;
  }
  return static_cast<int>(at);
}

cudaError_t launch_norm_rope_fwd(bool bf16, const NormRopeParams& p, int blocks, cudaStream_t st) {
  if (p.d == 64) return bf16 ? launch_fwd_d<true, 64>(p, blocks, st) : launch_fwd_d<false, 64>(p, blocks, st);
  if (p.d == 128) return bf16 ? launch_fwd_d<true, 128>(p, blocks, st) : launch_fwd_d<false, 128>(p, blocks, st);
  if (p.d == 192) return bf16 ? launch_fwd_d<true, 192>(p, blocks, st) : launch_fwd_d<false, 192>(p, blocks, st);
  return cudaErrorInvalidValue;
}

cudaError_t launch_norm_rope_bwd(bool bf16, const NormRopeParams& p, int blocks, void* dw_q, void* dw_k,
                                 cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (blocks > 0) {
    if (p.d == 64)
      e = bf16 ? launch_bwd_d<true, 64>(p, blocks, st) : launch_bwd_d<false, 64>(p, blocks, st);
    else if (p.d == 128)
      e = bf16 ? launch_bwd_d<true, 128>(p, blocks, st) : launch_bwd_d<false, 128>(p, blocks, st);
    else
      e = bf16 ? launch_bwd_d<true, 192>(p, blocks, st) : launch_bwd_d<false, 192>(p, blocks, st);
  }
  if (e != cudaSuccess || (dw_q == nullptr && dw_k == nullptr)) return e;
  const int k1 = p.n_kinds > 2 ? p.kind[2].block0 : blocks;
  auto kern = bf16 ? dw_reduce_kernel<true> : dw_reduce_kernel<false>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.d / 32, 2);
  cfg.blockDim = dim3(1024);
  cfg.stream = st;
  // the launch itself overlaps the end of the kernel that leaves the partial rows
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = blocks > 0 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<const float*>(p.dw_part), p.d, p.kind[0].block0, p.kind[1].block0,
                            k1, p.weight_fp32, dw_q, dw_k);
}

}  // namespace sdpa
