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
//      per pair, into rows sorted by expert; it starts beside kernel 1 and has
//      its place and its scales in hand when that ends;
//   3. the down rows past each expert's rows; a CTA starts, sorts the pairs and
//      requests its first 180 KB of weights as soon as one of kernel 1 has left
//      its SM, while the others and kernel 2 still run;
//   4. the weighted sum.
// Measured (8 experts of 4096 x 14336): one token with two experts 74 us (352 MB
// of weights, 4.8 TB/s, 0.73 of the copy rate: the SMs' shares of the bandwidth
// differ, kernel 1's CTAs end between 29 and 39 us, and kernel 3 cannot read
// before kernel 2 has the row's scale, about 8 us); 32 tokens 240 us (1.41 GB, 5.9
// TB/s, 0.90).
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
  int4* by_pair;        // workspace, like the following; [pairs]: {expert or -1, first tile of the down product,
                        // tiles from one row block to the next, blocks of a CTA there}
  int32_t* gu;          // [slices, pairs, 2 inter]: the gate and up sums
  int8_t* q;            // [pairs, inter], sorted by expert
  float* sh;            // [pairs]
  int32_t* part;        // [slices, pairs, hidden]: the down sums
  void* out;            // [m, hidden]
  int out_bf16;
  stream::Plan up, down;
  int up_grid, down_grid;
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

// Gate and up: rows of w13 past all tokens; tile t is row block t % row_blocks
// of active expert t / row_blocks.
struct GateUp {
  static constexpr bool kEarlyWeights = false;
  struct Walk {
    int i;
  };
  const Args& p;
  const Routing& r;
  __device__ __forceinline__ int tiles() const { return r.active * p.up.row_blocks; }
  __device__ __forceinline__ Walk start() const { return {0}; }
  __device__ __forceinline__ stream::Tile tile(Walk& w, int t) const {
    w.i = t / p.up.row_blocks;
    return {r.act[w.i] * p.up.n + (t - w.i * p.up.row_blocks) * stream::kRows, 0};
  }
  // The columns of the expert's tokens, four at a time, to their pairs' rows.
  __device__ __forceinline__ void store(const Walk& w, int, int slice, const stream::Tile& s, uint32_t tmem,
                                        int row) const {
    const stream::Plan& pl = p.up;
    const int col = s.w_row - r.act[w.i] * pl.n + row, lo = r.off[w.i], hi = r.off[w.i + 1];
    int32_t* out = p.gu + static_cast<int64_t>(slice) * (p.m * p.topk) * pl.n + col;
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

// Down: rows of w2 past an expert's rows of q, nb at a time: expert by expert, a
// row block's token tiles innermost, so that weights read again come from L2.
__device__ __forceinline__ int token_tiles(const Args& p, const Routing& r, int i) {
  const int n = r.off[i + 1] - r.off[i];
  return n <= p.down.nb ? 1 : (n + p.down.nb - 1) / p.down.nb;
}
__device__ __forceinline__ int down_tiles(const Args& p, const Routing& r) {
  int t = 0;
  for (int i = 0; i < r.active; ++i) t += token_tiles(p, r, i);
  return t * p.down.row_blocks;
}

struct Down {
  static constexpr bool kEarlyWeights = true;
  struct Walk {
    int i, base;  // active expert i, whose first tile is `base`
  };
  const Args& p;
  const Routing& r;
  __device__ __forceinline__ int tiles() const { return down_tiles(p, r); }
  __device__ __forceinline__ Walk start() const { return {0, 0}; }
  __device__ __forceinline__ stream::Tile tile(Walk& w, int t) const {
    int n = token_tiles(p, r, w.i);
    while (t - w.base >= p.down.row_blocks * n) {
      w.base += p.down.row_blocks * n;
      n = token_tiles(p, r, ++w.i);
    }
    const int j = t - w.base, rb = n == 1 ? j : j / n;
    return {r.act[w.i] * p.down.n + rb * stream::kRows, r.off[w.i] + (j - rb * n) * p.down.nb};
  }
  __device__ __forceinline__ void store(const Walk& w, int, int slice, const stream::Tile& s, uint32_t tmem,
                                        int row) const {
    const stream::Plan& pl = p.down;
    const int col = s.w_row - r.act[w.i] * pl.n + row, left = r.off[w.i + 1] - s.x_row;
    int32_t* out = p.part + static_cast<int64_t>(slice) * (p.m * p.topk) * pl.n + col;
    stream::each_column(tmem, left < pl.nb ? left : pl.nb, [&](int c, int v) {
      if (col < pl.n) out[static_cast<int64_t>(r.pairs[s.x_row + c]) * pl.n] = v;
    });
  }
};

// What kernel 4 needs of the routing (by all threads).
__device__ __forceinline__ void write_routing(const Args& p, const Routing& r) {
  const int tid = threadIdx.x, pairs = p.m * p.topk;
  const int per = stream::share(down_tiles(p, r), p.down.num_kb, p.down.cut, p.down_grid);
  for (int i = tid; i < pairs; i += blockDim.x)
    if (expert_of(p, i) < 0) p.by_pair[i] = make_int4(-1, 0, 0, 0);
  int base = 0;
  for (int i = 0; i < r.active; ++i) {
    const int n = token_tiles(p, r, i);
    for (int pos = r.off[i] + tid; pos < r.off[i + 1]; pos += blockDim.x)
      p.by_pair[r.pairs[pos]] = make_int4(r.act[i], base + (pos - r.off[i]) / p.down.nb, n, per);
    base += n * p.down.row_blocks;
  }
}

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
  if (blockIdx.x == gridDim.x - 1) write_routing(p, r);  // (the last CTA: its share is the smallest)
  fence_proxy_async_smem();  // the scratch above lies where copies will land
  __syncthreads();
  stream::run(GateUp{p, r}, p.up, s, ring, &tmW, &tmX);
  stream::teardown(s);
}

// It may start while kernel 1 runs (kernel 2 lets it, before its own wait).  What
// it reads before it waits for kernel 2, ids and weights, is the caller's and
// complete: kernel 1 has waited for whatever wrote them before it let kernel 2
// start.
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
  stream::setup(s, p.down);
  uint8_t* ring = stream::ring_of(raw);
  route(p, r, reinterpret_cast<int*>(ring));
  fence_proxy_async_smem();  // the scratch above lies where copies will land
  __syncthreads();
  stream::run(Down{p, r}, p.down, s, ring, &tmW, &tmX);
  stream::teardown(s);
}

// A pair's row of q: h = silu(g) * u, quantised.  One CTA or cluster per pair; a
// thread keeps kQuantVec vectors of 4 values, or, when the row is longer than
// that, leaves h in the gate sums' place and reads it back.  The row's place
// among the sorted pairs, how its sums are cut and its scales do not depend on
// kernel 1: they are found while that runs.
constexpr int kQuantThreads = 256;
constexpr int kQuantVec = 4;

template <bool CLUSTER, bool LONG>
__global__ void __launch_bounds__(kQuantThreads) moe_quant_kernel(Args p) {
  __shared__ float red[33];
  __shared__ unsigned used[kMaxExperts / 32];
  __shared__ int place;
  griddep_launch_dependents();  // kernel 3 may take the SMs that kernel 1 leaves
  int ranks = 1, rank = 0, pair = blockIdx.x;
  if constexpr (CLUSTER) {
    namespace cg = cooperative_groups;
    ranks = static_cast<int>(cg::this_cluster().num_blocks());
    rank = static_cast<int>(cg::this_cluster().block_rank());
    pair = blockIdx.x / ranks;
  }
  const int tid = threadIdx.x, pairs = p.m * p.topk, e = expert_of(p, pair);
  if (e < 0) {  // (the whole cluster) still, this kernel ends only after kernel 1
    griddep_wait();
    return;
  }
  // (ids and scales are the caller's: complete before kernel 1 let this one start)
  if (tid < kMaxExperts / 32) used[tid] = 0;
  if (tid == 0) place = 0;
  __syncthreads();
  int before = 0;
  for (int j = tid; j < pairs; j += kQuantThreads) {
    const int o = expert_of(p, j);
    if (o >= 0) atomicOr(&used[o >> 5], 1u << (o & 31));
    before += (o >= 0 && (o < e || (o == e && j < pair))) ? 1 : 0;
  }
  before = __reduce_add_sync(0xFFFFFFFFu, before);
  if ((tid & 31) == 0 && before > 0) atomicAdd(&place, before);
  __syncthreads();
  int active = 0, index = 0;  // experts in use, and among them those below e
  for (int i = 0; i < (p.experts + 31) / 32; ++i) {
    active += __popc(used[i]);
    index += i < (e >> 5) ? __popc(used[i]) : (i == (e >> 5) ? __popc(used[i] & ((1u << (e & 31)) - 1u)) : 0);
  }
  const int per = stream::share(active * p.up.row_blocks, p.up.num_kb, p.up.cut, p.up_grid);
  const float sa = __ldg(p.sa + ((pair * p.topk_inv) >> 16));
  int32_t* gu = p.gu + static_cast<int64_t>(pair) * 2 * p.inter;
  const int64_t slice = static_cast<int64_t>(pairs) * 2 * p.inter;
  const float* s13 = p.s13 + static_cast<int64_t>(e) * 2 * p.inter;
  const int nvec = p.inter / 4, stride = ranks * kQuantThreads, t0 = rank * kQuantThreads + tid;
  auto add_slices = [&](int4& v, int at) {
    const int n = stream::slices_of(index * p.up.row_blocks + at / stream::kRows, p.up.num_kb, per);
    for (int k = 1; k < n; ++k) {
      const int4 o = *reinterpret_cast<const int4*>(gu + k * slice + at);
      v.x += o.x;
      v.y += o.y;
      v.z += o.z;
      v.w += o.w;
    }
  };
  auto silu4 = [&](const int4& g, const int4& u, const float4& sg, const float4& su, float (&h)[4]) {
    auto val = [&](int acc, float sw) { return __fmul_rn(__fmul_rn(__int2float_rn(acc), sa), sw); };
    quant::silu_mul2(val(g.x, sg.x), val(g.y, sg.y), val(u.x, su.x), val(u.y, su.y), h[0], h[1]);
    quant::silu_mul2(val(g.z, sg.z), val(g.w, sg.w), val(u.z, su.z), val(u.w, su.w), h[2], h[3]);
  };
  auto scales4 = [&](int at) { return __ldg(reinterpret_cast<const float4*>(s13 + at)); };
  float h[LONG ? 1 : kQuantVec][4], amax = 0.0f;
  if constexpr (LONG) {
    griddep_wait();
    for (int v = t0; v < nvec; v += stride) {
      int4 g = *reinterpret_cast<const int4*>(gu + v * 4), u = *reinterpret_cast<const int4*>(gu + p.inter + v * 4);
      add_slices(g, v * 4);
      add_slices(u, p.inter + v * 4);
      silu4(g, u, scales4(v * 4), scales4(p.inter + v * 4), h[0]);
      *reinterpret_cast<float4*>(gu + v * 4) = make_float4(h[0][0], h[0][1], h[0][2], h[0][3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) amax = fmaxf(amax, fabsf(h[0][i]));
    }
  } else {
    float4 sg[kQuantVec], su[kQuantVec];
    int4 g[kQuantVec], u[kQuantVec];
#pragma unroll
    for (int j = 0; j < kQuantVec; ++j) {
      const int v = min(t0 + j * stride, nvec - 1);
      sg[j] = scales4(v * 4);
      su[j] = scales4(p.inter + v * 4);
    }
    griddep_wait();
#pragma unroll
    for (int j = 0; j < kQuantVec; ++j) {
      const int v = min(t0 + j * stride, nvec - 1);
      g[j] = *reinterpret_cast<const int4*>(gu + v * 4);
      u[j] = *reinterpret_cast<const int4*>(gu + p.inter + v * 4);
    }
#pragma unroll
    for (int j = 0; j < kQuantVec; ++j) {
      const int v = t0 + j * stride;
      if (v < nvec) {
        add_slices(g[j], v * 4);
        add_slices(u[j], p.inter + v * 4);
        silu4(g[j], u[j], sg[j], su[j], h[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) amax = fmaxf(amax, fabsf(h[j][i]));
      }
    }
  }
  amax = quant::row_max<CLUSTER>(amax, red);
  const float scale = __fdiv_rn(fmaxf(amax, 1e-12f), 127.0f), inv = __fdiv_rn(1.0f, scale);
  int8_t* q = p.q + static_cast<int64_t>(place) * p.inter;
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

// out[i][j .. j + 3]: the slots in order, eight at a time.  What does not come
// from the down product is read before the wait (the kernels before it have
// waited for whatever wrote it); the loads of all eight slots' sums are issued
// before any is used, of slots without an expert too (their rows of the
// workspace hold anything, and are not used).
__global__ void __launch_bounds__(128) moe_combine_kernel(Args p) {
  constexpr int S = 8;
  const int i = blockIdx.y, j = (blockIdx.x * 128 + threadIdx.x) * 4;
  if (j >= p.hidden) return;
  const int64_t slice = static_cast<int64_t>(p.m) * p.topk * p.hidden;
  float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s0 = 0; s0 < p.topk; s0 += S) {
    int4 rec[S], acc[S];
    float4 s2[S];
    float sh[S], wt[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int pair = i * p.topk + min(s0 + s, p.topk - 1);
      rec[s] = __ldg(p.by_pair + pair);
      sh[s] = __ldg(p.sh + pair);
      wt[s] = __ldg(p.wt + pair);
    }
#pragma unroll
    for (int s = 0; s < S; ++s)
      s2[s] = __ldg(reinterpret_cast<const float4*>(p.s2 + static_cast<int64_t>(max(rec[s].x, 0)) * p.hidden + j));
    if (s0 == 0) {
      griddep_wait();
      griddep_launch_dependents();
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int pair = i * p.topk + min(s0 + s, p.topk - 1);
      acc[s] = *reinterpret_cast<const int4*>(p.part + static_cast<int64_t>(pair) * p.hidden + j);
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if (s0 + s >= p.topk || rec[s].x < 0) continue;
      const int32_t* part = p.part + (static_cast<int64_t>(i) * p.topk + s0 + s) * p.hidden + j;
      const int n = stream::slices_of(rec[s].y + j / stream::kRows * rec[s].z, p.down.num_kb, rec[s].w);
      for (int k = 1; k < n; ++k) {
        const int4 v = *reinterpret_cast<const int4*>(part + k * slice);
        acc[s].x += v.x;
        acc[s].y += v.y;
        acc[s].z += v.z;
        acc[s].w += v.w;
      }
      f[0] = __fmaf_rn(wt[s], __fmul_rn(__fmul_rn(__int2float_rn(acc[s].x), sh[s]), s2[s].x), f[0]);
      f[1] = __fmaf_rn(wt[s], __fmul_rn(__fmul_rn(__int2float_rn(acc[s].y), sh[s]), s2[s].y), f[1]);
      f[2] = __fmaf_rn(wt[s], __fmul_rn(__fmul_rn(__int2float_rn(acc[s].z), sh[s]), s2[s].z), f[2]);
      f[3] = __fmaf_rn(wt[s], __fmul_rn(__fmul_rn(__int2float_rn(acc[s].w), sh[s]), s2[s].w), f[3]);
    }
  }
  const int64_t o = static_cast<int64_t>(i) * p.hidden + j;
  if (p.out_bf16)
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + o) =
        make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
  else
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + o) = make_float4(f[0], f[1], f[2], f[3]);
}

// Both products' plans.  Tokens of a down tile: twice an expert's share of the
// pairs where the router spreads them evenly; an expert with more has its
// weights read again, from L2.
inline void plans(Args& a, int num_sms) {
  const int64_t pairs = static_cast<int64_t>(a.m) * a.topk, share = (2 * pairs + a.experts - 1) / a.experts;
  a.up = stream::plan(a.m, 2 * a.inter, a.hidden, num_sms, 4, stream::kRingBytes);
  a.down = stream::plan(static_cast<int>(share < a.m ? share : a.m), a.hidden, a.inter, num_sms, 4,
                        stream::kRingBytes);
  a.up_grid = a.down_grid = num_sms;
}

inline cudaError_t launch_quant(const Args& a, int num_sms, cudaStream_t stream) {
  const int pairs = a.m * a.topk, per = kQuantThreads * kQuantVec * 4;  // values a CTA holds
  int cl = 1;
  while (cl < 8 && (a.inter > cl * per || (2 * pairs * cl <= num_sms && a.inter > cl * kQuantThreads * 4))) cl *= 2;
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
  if ((*err = stream::shares_sm_once(moe_quant_kernel<true, true>, dev, 0)) != cudaSuccess) return 2;
  if ((*err = stream::shares_sm_once(moe_quant_kernel<true, false>, dev, 1)) != cudaSuccess) return 2;
  if ((*err = stream::shares_sm_once(moe_quant_kernel<false, false>, dev, 2)) != cudaSuccess) return 2;
  if ((*err = stream::shares_sm_once(moe_combine_kernel, dev, 3)) != cudaSuccess) return 2;
  *err = launch_pdl(moe_gate_up_kernel, dim3(a.up_grid), dim3(stream::kThreads), stream::smem_bytes(a.up), stream, 1,
                    tw13, tx, a);
  if (*err == cudaSuccess) *err = launch_quant(a, num_sms, stream);
  if (*err == cudaSuccess)
    *err = launch_pdl(moe_down_kernel, dim3(a.down_grid), dim3(stream::kThreads), stream::smem_bytes(a.down), stream,
                      1, tw2, tq, a);
  if (*err == cudaSuccess)
    *err = launch_pdl(moe_combine_kernel, dim3((a.hidden + 511) / 512, a.m), dim3(128), 0, stream, 1, a);
  return *err == cudaSuccess ? 0 : 2;
}

}  // namespace moe
}  // namespace qk
