// moe_layer.cuh -- a whole W8A8 mixture-of-experts layer for a few tokens.
//
// Token i's slot s names expert e = ids[i, s] with weight wt[i, s]; a pair is
// one (token, slot).  Per pair:
//     g, u = ((acc * sa) * sw) of the expert's gate and up rows
//     h    = silu(g) * u                      (the SiLU quantiser's arithmetic)
//     q, sh = per-token quantisation of h     (max(amax, 1e-12) / 127)
//     y    = ((acc * sh) * sw2) of the expert's down rows
// and out[i] = the chain f = fma(wt, y, f) over the slots, in order, rounded
// once.  A slot whose id lies outside [0, experts) adds nothing.
//
// Bound: reading the weights of the experts that are used, once each.  Four
// kernels, overlapped by programmatic dependent launch:
//   1. every CTA sorts the pairs by expert for itself (a few hundred integers:
//      no launch is spent on it) and streams gate and up rows past ALL tokens
//      (stream.cuh: up to 64 cost the tensor core nothing while it waits for
//      weights), keeping the columns of an expert's own tokens, so that no token
//      is gathered or copied;
//   2. scales, silu, the row's maximum and its quantisation, one CTA or cluster
//      per pair, into rows sorted by expert;
//   3. the down rows past each expert's rows; its first 200 KB of weights an SM
//      are requested while kernel 2 still runs;
//   4. the weighted sum.
#pragma once

#include "qk_common.cuh"
#include "quant.cuh"
#include "stream.cuh"

namespace qk {
namespace moe {

constexpr int kMaxPairs = 2048;    // 64 tokens x 32 slots
constexpr int kMaxExperts = 1024;

// The pairs sorted by expert: expert act[i] has pairs[off[i] .. off[i + 1]).
struct Routing {
  int active;
  short act[kMaxExperts];
  short off[kMaxExperts + 1];
  short pairs[kMaxPairs];
};

struct Args {
  int m, hidden, inter, experts, topk;
  int topk_inv;         // ceil(65536 / topk): pair / topk = (pair * topk_inv) >> 16 for pairs < 2048
  const float* sa;      // [m]
  const int32_t* ids;   // [m, topk]
  const float* wt;      // [m, topk]
  const float* s13;     // [experts, 2 inter]
  const float* s2;      // [experts, hidden]
  Routing* routing;     // workspace, like the following
  int32_t* gu;          // [slices, pairs, 2 inter]: the gate and up sums
  int8_t* q;            // [pairs, inter], sorted by expert
  float* sh;            // [pairs]
  int32_t* part;        // [slices, pairs, hidden]: the down sums
  void* out;            // [m, hidden]
  int out_bf16;
  stream::Plan up, down;
};

__device__ __forceinline__ int expert_of(const Args& p, int pair) {
  const int e = __ldg(p.ids + pair);
  return (e >= 0 && e < p.experts) ? e : -1;
}

// By all threads; `cnt` is scratch for kMaxExperts ints.
__device__ __forceinline__ void route(const Args& p, Routing& r, int* cnt) {
  const int tid = threadIdx.x, pairs = p.m * p.topk;
  for (int e = tid; e < p.experts; e += blockDim.x) cnt[e] = 0;
  __syncthreads();
  for (int i = tid; i < pairs; i += blockDim.x) {
    const int e = expert_of(p, i);
    if (e >= 0) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  if (tid < 32) {
    int active = 0, off = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 32) {
      const int e = e0 + tid, c = e < p.experts ? cnt[e] : 0;
      const unsigned used = __ballot_sync(0xFFFFFFFFu, c > 0);
      if (used == 0) continue;
      int sum = c;  // inclusive prefix over the warp
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (tid >= o) sum += v;
      }
      if (c > 0) {
        const int at = active + __popc(used & ((1u << tid) - 1u));
        r.act[at] = static_cast<short>(e);
        r.off[at] = static_cast<short>(off + sum - c);
        cnt[e] = off + sum - c;  // where the expert's next pair goes
      }
      active += __popc(used);
      off += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    if (tid == 0) {
      r.off[active] = static_cast<short>(off);
      r.active = active;
    }
    __syncwarp();
    // An expert's pairs in their own order, 32 at a time: every CTA must arrive at
    // the same order, so no atomic hands out the places.
    for (int i0 = 0; i0 < pairs; i0 += 32) {
      const int i = i0 + tid, e = i < pairs ? expert_of(p, i) : -1;
      const unsigned same = __match_any_sync(0xFFFFFFFFu, e), before = same & ((1u << tid) - 1u);
      const int at = e >= 0 ? cnt[e] : 0;
      __syncwarp();
      if (e >= 0) {
        r.pairs[at + __popc(before)] = static_cast<short>(i);
        if (before == 0) cnt[e] = at + __popc(same);
      }
      __syncwarp();
    }
  }
  __syncthreads();
}

// Units: expert by expert, a row block and K range at a time; an expert's token
// tiles (down) innermost, so that weights read again come from L2.
struct Walk {
  int i, base;  // active expert i, whose first unit is `base`
};

// Gate and up: rows of w13 past all tokens.
struct GateUp {
  static constexpr bool kEarlyWeights = false;
  using Walk = moe::Walk;
  const Args& p;
  const Routing& r;
  __device__ __forceinline__ Walk start() const { return {0, 0}; }
  __device__ __forceinline__ bool span(Walk& w, int u, stream::Span& s) const {
    const stream::Plan& pl = p.up;
    const int per = pl.row_blocks * pl.ksplit;
    w.i = u / per;
    if (w.i >= r.active) return false;
    const int j = u - w.i * per, rb = j / pl.ksplit, ks = j - rb * pl.ksplit;
    s.w_row = r.act[w.i] * pl.n + rb * stream::kRows;
    s.x_row = 0;
    s.kb0 = ks * pl.kbs;
    s.kb1 = min(pl.num_kb, s.kb0 + pl.kbs);
    return true;
  }
  // The columns of the expert's tokens, four at a time, to their pairs' rows.
  __device__ __forceinline__ void store(const Walk& w, int, const stream::Span& s, uint32_t tmem, int row) const {
    const stream::Plan& pl = p.up;
    const int col = s.w_row - r.act[w.i] * pl.n + row, lo = r.off[w.i], hi = r.off[w.i + 1];
    int32_t* out = p.gu + static_cast<int64_t>(s.kb0 / pl.kbs) * (p.m * p.topk) * pl.n + col;
    for (int j = lo; j < hi; j += 4) {
      uint32_t v[4];
      __syncwarp();
#pragma unroll
      for (int c = 0; c < 4; ++c)
        v[c] = stream::tmem_ld_x1(tmem + ((r.pairs[min(j + c, hi - 1)] * p.topk_inv) >> 16));
      tmem_ld_wait();
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (j + c < hi && col < pl.n) out[static_cast<int64_t>(r.pairs[j + c]) * pl.n] = static_cast<int>(v[c]);
    }
  }
};

// Down: rows of w2 past an expert's rows of q, nb at a time.
struct Down {
  static constexpr bool kEarlyWeights = true;
  using Walk = moe::Walk;
  const Args& p;
  const Routing& r;
  __device__ __forceinline__ Walk start() const { return {0, 0}; }
  __device__ __forceinline__ int tiles(int i) const {
    const int n = r.off[i + 1] - r.off[i];
    return n <= p.down.nb ? 1 : (n + p.down.nb - 1) / p.down.nb;
  }
  __device__ __forceinline__ bool span(Walk& w, int u, stream::Span& s) const {
    const stream::Plan& pl = p.down;
    const int per = pl.row_blocks * pl.ksplit;
    if (w.i >= r.active) return false;
    int t = tiles(w.i);
    while (u - w.base >= per * t) {
      w.base += per * t;
      if (++w.i >= r.active) return false;
      t = tiles(w.i);
    }
    const int j = u - w.base, b = t == 1 ? j : j / t, rb = b / pl.ksplit, ks = b - rb * pl.ksplit;
    s.w_row = r.act[w.i] * pl.n + rb * stream::kRows;
    s.x_row = r.off[w.i] + (j - b * t) * pl.nb;
    s.kb0 = ks * pl.kbs;
    s.kb1 = min(pl.num_kb, s.kb0 + pl.kbs);
    return true;
  }
  __device__ __forceinline__ void store(const Walk& w, int, const stream::Span& s, uint32_t tmem, int row) const {
    const stream::Plan& pl = p.down;
    const int col = s.w_row - r.act[w.i] * pl.n + row, left = r.off[w.i + 1] - s.x_row;
    int32_t* out = p.part + static_cast<int64_t>(s.kb0 / pl.kbs) * (p.m * p.topk) * pl.n + col;
    stream::each_column(tmem, left < pl.nb ? left : pl.nb, [&](int c, int v) {
      if (col < pl.n) out[static_cast<int64_t>(r.pairs[s.x_row + c]) * pl.n] = v;
    });
  }
};

__global__ void __launch_bounds__(stream::kThreads, 1)
    moe_gate_up_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                       const __grid_constant__ Args p) {
  extern __shared__ uint8_t raw[];
  __shared__ stream::Bars s;
  __shared__ Routing r;
  if (threadIdx.x == 0) {
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
  }
  stream::setup(s, p.up);
  griddep_wait();  // the previous kernel in the stream is done with our buffers
  griddep_launch_dependents();
  uint8_t* ring = stream::ring_of(raw);
  route(p, r, reinterpret_cast<int*>(ring));
  if (blockIdx.x == 0) {
    const int* src = reinterpret_cast<const int*>(&r);
    for (int i = threadIdx.x; i < static_cast<int>(sizeof(Routing) / 4); i += stream::kThreads)
      reinterpret_cast<int*>(p.routing)[i] = src[i];
  }
  fence_proxy_async_smem();  // the scratch above lies where copies will land
  __syncthreads();
  stream::run(GateUp{p, r}, p.up, s, ring, &tmW, &tmX);
  stream::teardown(s);
}

// What this kernel reads before its wait (the routing, weights) is complete: the
// quantiser before it has waited for the kernel that wrote the routing, and that
// one for whatever wrote the caller's data, before this one could start.
__global__ void __launch_bounds__(stream::kThreads, 1)
    moe_down_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                    const __grid_constant__ Args p) {
  extern __shared__ uint8_t raw[];
  __shared__ stream::Bars s;
  __shared__ Routing r;
  if (threadIdx.x == 0) {
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
  }
  for (int i = threadIdx.x; i < static_cast<int>(sizeof(Routing) / 4); i += stream::kThreads)
    reinterpret_cast<int*>(&r)[i] = __ldcg(reinterpret_cast<const int*>(p.routing) + i);
  stream::setup(s, p.down);
  stream::run(Down{p, r}, p.down, s, stream::ring_of(raw), &tmW, &tmX);
  stream::teardown(s);
}

// Row `pos` of q: h = silu(g) * u of pair pairs[pos], quantised.  One CTA or
// cluster per row; a thread keeps up to kQuantVec vectors of 4 values, or, when
// the row is longer, leaves h in the gate sums' place and reads it back.
constexpr int kQuantThreads = 256;
constexpr int kQuantVec = 4;

template <bool CLUSTER, bool LONG>
__global__ void __launch_bounds__(kQuantThreads) moe_quant_kernel(Args p) {
  __shared__ float red[33];
  griddep_wait();
  griddep_launch_dependents();
  int ranks = 1, rank = 0, pos = blockIdx.x;
  if constexpr (CLUSTER) {
    namespace cg = cooperative_groups;
    ranks = static_cast<int>(cg::this_cluster().num_blocks());
    rank = static_cast<int>(cg::this_cluster().block_rank());
    pos = blockIdx.x / ranks;
  }
  if (pos >= p.routing->off[p.routing->active]) return;  // (the whole cluster: slots without an expert)
  const int pair = p.routing->pairs[pos], e = __ldg(p.ids + pair), pairs = p.m * p.topk;
  const float sa = __ldg(p.sa + ((pair * p.topk_inv) >> 16));
  int32_t* gu = p.gu + static_cast<int64_t>(pair) * 2 * p.inter;
  const int64_t slice = static_cast<int64_t>(pairs) * 2 * p.inter;
  const float* s13 = p.s13 + static_cast<int64_t>(e) * 2 * p.inter;
  const int nvec = p.inter / 4, stride = ranks * kQuantThreads, t0 = rank * kQuantThreads + threadIdx.x;
  auto sums = [&](int at) {
    int4 v = *reinterpret_cast<const int4*>(gu + at);
    for (int k = 1; k < p.up.ksplit; ++k) {
      const int4 o = *reinterpret_cast<const int4*>(gu + k * slice + at);
      v.x += o.x;
      v.y += o.y;
      v.z += o.z;
      v.w += o.w;
    }
    return v;
  };
  auto row4 = [&](int j, float (&h)[4]) {
    const int4 g = sums(j), u = sums(p.inter + j);
    float a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int gi = i == 0 ? g.x : (i == 1 ? g.y : (i == 2 ? g.z : g.w));
      const int ui = i == 0 ? u.x : (i == 1 ? u.y : (i == 2 ? u.z : u.w));
      a[i] = __fmul_rn(__fmul_rn(__int2float_rn(gi), sa), __ldg(s13 + j + i));
      b[i] = __fmul_rn(__fmul_rn(__int2float_rn(ui), sa), __ldg(s13 + p.inter + j + i));
    }
    quant::silu_mul2(a[0], a[1], b[0], b[1], h[0], h[1]);
    quant::silu_mul2(a[2], a[3], b[2], b[3], h[2], h[3]);
  };
  float h[LONG ? 1 : kQuantVec][4], amax = 0.0f;
  if constexpr (LONG) {
    for (int v = t0; v < nvec; v += stride) {
      row4(v * 4, h[0]);
      *reinterpret_cast<float4*>(gu + v * 4) = make_float4(h[0][0], h[0][1], h[0][2], h[0][3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) amax = fmaxf(amax, fabsf(h[0][i]));
    }
  } else {
#pragma unroll
    for (int j = 0; j < kQuantVec; ++j) {
      const int v = t0 + j * stride;
      if (v < nvec) {
        row4(v * 4, h[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) amax = fmaxf(amax, fabsf(h[j][i]));
      }
    }
  }
  amax = quant::row_max<CLUSTER>(amax, red);
  const float scale = __fdiv_rn(fmaxf(amax, 1e-12f), 127.0f), inv = __fdiv_rn(1.0f, scale);
  int8_t* q = p.q + static_cast<int64_t>(pos) * p.inter;
  quant::Args qa = {};
  if constexpr (LONG) {
    for (int v = t0; v < nvec; v += stride) {
      const float4 f = *reinterpret_cast<const float4*>(gu + v * 4);
      h[0][0] = f.x;
      h[0][1] = f.y;
      h[0][2] = f.z;
      h[0][3] = f.w;
      quant::store_q<4>(qa, q + v * 4, h[0], inv);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kQuantVec; ++j) {
      const int v = t0 + j * stride;
      if (v < nvec) quant::store_q<4>(qa, q + v * 4, h[j], inv);
    }
  }
  if (t0 == 0) p.sh[pair] = scale;
  if constexpr (CLUSTER) quant::cluster_arrive_wait_relaxed();  // peers may still read red[32]
}

// out[i][j .. j + 3]: the slots in order.
__global__ void __launch_bounds__(128) moe_combine_kernel(Args p) {
  griddep_wait();
  griddep_launch_dependents();
  const int i = blockIdx.y, j = (blockIdx.x * 128 + threadIdx.x) * 4;
  if (j >= p.hidden) return;
  const int64_t slice = static_cast<int64_t>(p.m) * p.topk * p.hidden;
  float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int s = 0; s < p.topk; ++s) {
    const int pair = i * p.topk + s, e = expert_of(p, pair);
    if (e >= 0) {
      const int32_t* part = p.part + static_cast<int64_t>(pair) * p.hidden + j;
      int4 acc = __ldg(reinterpret_cast<const int4*>(part));
      for (int k = 1; k < p.down.ksplit; ++k) {
        const int4 v = __ldg(reinterpret_cast<const int4*>(part + k * slice));
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
      }
      const float* s2 = p.s2 + static_cast<int64_t>(e) * p.hidden + j;
      const float sh = __ldg(p.sh + pair), wt = __ldg(p.wt + pair);
      f[0] = __fmaf_rn(wt, __fmul_rn(__fmul_rn(__int2float_rn(acc.x), sh), __ldg(s2)), f[0]);
      f[1] = __fmaf_rn(wt, __fmul_rn(__fmul_rn(__int2float_rn(acc.y), sh), __ldg(s2 + 1)), f[1]);
      f[2] = __fmaf_rn(wt, __fmul_rn(__fmul_rn(__int2float_rn(acc.z), sh), __ldg(s2 + 2)), f[2]);
      f[3] = __fmaf_rn(wt, __fmul_rn(__fmul_rn(__int2float_rn(acc.w), sh), __ldg(s2 + 3)), f[3]);
    }
  }
  const int64_t o = static_cast<int64_t>(i) * p.hidden + j;
  if (p.out_bf16)
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + o) =
        make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
  else
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o) = make_float4(f[0], f[1], f[2], f[3]);
}

// Both products' plans.  Experts expected in use: no more than there are pairs.
// Tokens of a down unit: twice an expert's share of the pairs where the router
// spreads them evenly; an expert with more has its weights read again, from L2.
inline void plans(int m, int hidden, int inter, int experts, int topk, int num_sms, stream::Plan* up,
                  stream::Plan* down) {
  const int64_t pairs = static_cast<int64_t>(m) * topk, sets = pairs < experts ? pairs : experts;
  *up = stream::plan(m, sets, 2 * inter, hidden, num_sms);
  const int64_t share = (2 * pairs + experts - 1) / experts;
  *down = stream::plan(static_cast<int>(share < m ? share : m), sets, hidden, inter, num_sms);
}

inline cudaError_t launch_quant(const Args& a, int num_sms, cudaStream_t stream) {
  const int pairs = a.m * a.topk, per = kQuantThreads * kQuantVec * 4;  // values a CTA holds
  int cl = 1;
  while (cl < 8 && (a.inter > cl * per || (pairs * cl < 2 * num_sms && a.inter > cl * kQuantThreads * 4))) cl *= 2;
  const dim3 grid(static_cast<unsigned>(pairs * cl)), block(kQuantThreads);
  if (a.inter > cl * per)
    return launch_pdl(moe_quant_kernel<true, true>, grid, block, 0, stream, static_cast<unsigned>(cl), a);
  if (cl > 1)
    return launch_pdl(moe_quant_kernel<true, false>, grid, block, 0, stream, static_cast<unsigned>(cl), a);
  return launch_pdl(moe_quant_kernel<false, false>, grid, block, 0, stream, 1, a);
}

// Returns 0, 1 when a tensor map could not be made, 2 with *err set.
inline int launch(const Args& a, const int8_t* x, const int8_t* w13, const int8_t* w2, int dev, int num_sms,
                  cudaStream_t stream, cudaError_t* err) {
  const int pairs = a.m * a.topk;
  CUtensorMap tw13, tx, tw2, tq;
  if (!gemm::cached_tmap(&tw13, w13, a.experts * a.up.n, a.hidden, stream::kRows) ||
      !gemm::cached_tmap(&tx, x, a.m, a.hidden, a.up.nb) ||
      !gemm::cached_tmap(&tw2, w2, a.experts * a.down.n, a.inter, stream::kRows) ||
      !gemm::cached_tmap(&tq, a.q, pairs, a.inter, a.down.nb))
    return 1;
  const size_t most = stream::kRingBytes + 1024;
  if ((*err = gemm::set_smem_once(moe_gate_up_kernel, dev, 0, most)) != cudaSuccess) return 2;
  if ((*err = gemm::set_smem_once(moe_down_kernel, dev, 1, most)) != cudaSuccess) return 2;
  // units at most: every active expert's, and in the down product one token tile
  // more for every nb pairs
  const int64_t sets = pairs < a.experts ? pairs : a.experts;
  const int64_t up = sets * a.up.row_blocks * a.up.ksplit;
  const int64_t down = (sets + pairs / a.down.nb) * a.down.row_blocks * a.down.ksplit;
  *err = launch_pdl(moe_gate_up_kernel, dim3(static_cast<unsigned>(up < num_sms ? up : num_sms)),
                    dim3(stream::kThreads), stream::smem_bytes(a.up), stream, 1, tw13, tx, a);
  if (*err == cudaSuccess) *err = launch_quant(a, num_sms, stream);
  if (*err == cudaSuccess)
    *err = launch_pdl(moe_down_kernel, dim3(static_cast<unsigned>(down < num_sms ? down : num_sms)),
                      dim3(stream::kThreads), stream::smem_bytes(a.down), stream, 1, tw2, tq, a);
  if (*err == cudaSuccess)
    *err = launch_pdl(moe_combine_kernel, dim3((a.hidden + 511) / 512, a.m), dim3(128), 0, stream, 1, a);
  return *err == cudaSuccess ? 0 : 2;
}

}  // namespace moe
}  // namespace qk
