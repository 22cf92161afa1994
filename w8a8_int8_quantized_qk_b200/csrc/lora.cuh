// lora.cuh -- low-rank adapters of many requests beside the shared W8A8
// projection: out = epilogue(a b^T) + s B[id]^T, s = lora_scale[id] * x A[id]^T,
// where token i uses adapter id = ids[i] (none when outside [0, adapters)).
//
// Three kernels: s (the tokens into the adapters' ranks), the projection's
// int32 sums (the stream of stream.cuh up to 64 tokens, the GEMM beyond), and
// the output: the sums' epilogue plus s B^T, rounded once.
//
// Both small products run on the bf16 matrix instruction, 16 tokens a tile.
// A bf16 value is exact there; a binary32 one (s, and x when it is fp32) enters
// as three bf16 terms, x = h + m + l, each the rounding of what is left: 24 bits,
// so a product of 16 of them is as good as one of binary32 values.  Tokens of
// a tile may use different adapters: each adapter present is multiplied with
// the whole tile and the rows that use it take its result.  They take it by
// selection, not by multiplying with zero, so that an adapter that holds NaN
// or infinity reaches no row of another.
#pragma once

#include "qk_common.cuh"
#include "quant.cuh"
#include "stream.cuh"

namespace qk {
namespace lora {

struct Args {
  int m, n, k, rank, adapters;
  const void* x;              // [m, k] bf16 or fp32
  const __nv_bfloat16* la;    // [adapters, rank, k]
  const __nv_bfloat16* lb;    // [adapters, n, rank]
  const float* lscale;        // [adapters] or null
  const int32_t* ids;         // [m]
  const float* sa;            // [m]
  const float* sw;            // [n]
  float alpha;
  float* s;                   // [kparts, m, rank] workspace: parts over K
  int kparts, kpart;          // parts, and K elements of one (a multiple of 256)
  const int32_t* c;           // [slices, m, n] workspace: the int32 sums of the projection
  int num_kb, per;            // how c's tiles are cut into slices (per 0: not at all)
  void* out;
  int out_bf16;
};

constexpr int kTile = 16;  // tokens of a tile

__device__ __forceinline__ int adapter_of(const Args& p, int row) {
  const int id = row < p.m ? __ldg(p.ids + row) : -1;
  return (id >= 0 && id < p.adapters) ? id : -1;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two binary32 values as three pairs of bf16 terms.
__device__ __forceinline__ void split3(float lo, float hi, uint32_t (&t)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    t[i] = pack_bf16x2(lo, hi);
    lo = __fsub_rn(lo, bf16_lo(t[i]));
    hi = __fsub_rn(hi, bf16_hi(t[i]));
  }
}

// The tokens of tile `t` by adapter, by a whole warp: lane i < 16 holds token i's
// adapter in `id`, -1 for none and -2 past the last token.  Returns a mask of the
// lanes that show one first.
__device__ __forceinline__ unsigned tile_groups(const Args& p, int t, int& id) {
  const int lane = threadIdx.x & 31, row = t * kTile + lane;
  id = (lane < kTile && row < p.m) ? adapter_of(p, row) : -2;
  const unsigned same = __match_any_sync(0xFFFFFFFFu, id);
  return __ballot_sync(0xFFFFFFFFu, id >= -1 && (same & ((1u << lane) - 1u)) == 0);
}

// ---------------------------------------------------------------------------
// s: one CTA per (token tile, adapter in it, K part and 64 ranks); its 8 warps
// deal the part's K in steps of 32 and each multiplies all ranks.  The operands
// come straight from memory: a dot product may sum K in any order, so thread
// (g, q) takes elements 8 q .. 8 q + 7 of a step (16 bytes) of token g, of token
// g + 8 and of the adapter's row, four of them for each of two instructions, in
// the places (2 q, 2 q + 1) and (2 q + 8, 2 q + 9) those have for it.
// ---------------------------------------------------------------------------
constexpr int kShrinkThreads = 256;
constexpr int kShrinkStep = 32;
constexpr int kMaxRank = 128, kRankGroup = 64;

// Elements at .. at + 7 of x, as terms of four pairs.
template <bool BF16>
__device__ __forceinline__ void load_x(const void* x, int64_t at, bool in, uint32_t (&v)[4][BF16 ? 1 : 3]) {
  if constexpr (BF16) {
    const uint4 w = in ? __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(x) + at))
                       : make_uint4(0, 0, 0, 0);
    v[0][0] = w.x;
    v[1][0] = w.y;
    v[2][0] = w.z;
    v[3][0] = w.w;
  } else {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float4 a = in ? __ldg(f) : zero, b = in ? __ldg(f + 1) : zero;
    split3(a.x, a.y, v[0]);
    split3(a.z, a.w, v[1]);
    split3(b.x, b.y, v[2]);
    split3(b.z, b.w, v[3]);
  }
}

template <bool BF16, int RT>  // RT: tiles of 8 ranks
__global__ void __launch_bounds__(kShrinkThreads) lora_shrink_kernel(Args p) {
  constexpr int NW = kShrinkThreads / 32, TERMS = BF16 ? 1 : 3;
  __shared__ float red[NW][kTile][RT * 8 + 1];
  griddep_wait();
  griddep_launch_dependents();
  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  int id;
  const unsigned firsts = tile_groups(p, t, id) & __ballot_sync(0xFFFFFFFFu, id >= 0);
  if (static_cast<int>(blockIdx.y) >= __popc(firsts)) return;
  const int use = __shfl_sync(0xFFFFFFFFu, id, __fns(firsts, 0, blockIdx.y + 1));
  const unsigned mine = __ballot_sync(0xFFFFFFFFu, id == use);  // tokens of this adapter
  const int z = blockIdx.z % p.kparts, rg = blockIdx.z / p.kparts * kRankGroup, ranks = min(p.rank - rg, kRankGroup);
  const int k0 = z * p.kpart, k1 = min(p.k, k0 + p.kpart), r0 = t * kTile;
  const __nv_bfloat16* a = p.la + (static_cast<int64_t>(use) * p.rank + rg) * p.k;
  float acc[RT][4];
#pragma unroll
  for (int j = 0; j < RT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
  const bool in0 = (mine >> g) & 1u, in1 = (mine >> (g + 8)) & 1u;
#pragma unroll(RT <= 2 ? 4 : (RT <= 4 ? 2 : 1))
  for (int k = k0 + warp * kShrinkStep + q * 8; k < k1 + q * 8; k += NW * kShrinkStep) {
    const bool in = k < k1;  // (K is a multiple of 16: the last step may be half one)
    uint32_t x0[4][TERMS], x1[4][TERMS];
    uint4 b[RT];
    load_x<BF16>(p.x, static_cast<int64_t>(r0 + g) * p.k + k, in0 && in, x0);
    load_x<BF16>(p.x, static_cast<int64_t>(r0 + g + 8) * p.k + k, in1 && in, x1);
#pragma unroll
    for (int j = 0; j < RT; ++j)
      b[j] = (j * 8 < ranks && in) ? __ldg(reinterpret_cast<const uint4*>(a + static_cast<int64_t>(j * 8 + g) * p.k + k))
                                   : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < TERMS; ++i) {
      const uint32_t f0[4] = {x0[0][i], x1[0][i], x0[1][i], x1[1][i]};
      const uint32_t f1[4] = {x0[2][i], x1[2][i], x0[3][i], x1[3][i]};
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        mma_bf16(acc[j], f0, b[j].x, b[j].y);
        mma_bf16(acc[j], f1, b[j].z, b[j].w);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    red[warp][g][j * 8 + 2 * q] = acc[j][0];
    red[warp][g][j * 8 + 2 * q + 1] = acc[j][1];
    red[warp][g + 8][j * 8 + 2 * q] = acc[j][2];
    red[warp][g + 8][j * 8 + 2 * q + 1] = acc[j][3];
  }
  __syncthreads();
  const float ls = p.lscale ? __ldg(p.lscale + use) : 1.0f;
  float* s = p.s + static_cast<int64_t>(z) * p.m * p.rank + rg;
  for (int i = tid; i < kTile * ranks; i += kShrinkThreads) {
    const int row = i / ranks, r = i - row * ranks;
    if (!((mine >> row) & 1u)) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += red[w][row][r];
    s[static_cast<int64_t>(r0 + row) * p.rank + r] = ls * v;
  }
}

// ---------------------------------------------------------------------------
// out: a CTA takes 16 tokens by 256 columns, a warp 32 of the columns, and one
// group of tokens after another (those of an adapter, or of none); where the
// grid would be small the groups go to CTAs of their own.  Column 2 q + b of the
// j-th product of a warp stands for column 8 q + 2 j + b of its 32, so that a
// thread ends up with 8 consecutive columns of rows g and g + 8: 16-byte reads of
// the sums, 16-byte writes.  All but the sums is read, and multiplied, before
// the wait for the projection: it is the caller's, or the kernel's before that.
// ---------------------------------------------------------------------------
constexpr int kExpandThreads = 256;
constexpr int kExpandCols = 256;

inline size_t expand_smem(int rank) { return static_cast<size_t>(3) * kTile * ((rank + 15) / 16 * 8 + 4) * 4; }

__global__ void __launch_bounds__(kExpandThreads) lora_expand_kernel(Args p) {
  extern __shared__ uint32_t ss[];  // s: [term][token][rank / 2 words], rows padded by 16 bytes
  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const int r0 = t * kTile, steps = (p.rank + 15) / 16, pitch = steps * 8 + 4;
  const int col0 = blockIdx.y * kExpandCols + warp * 32, col = col0 + q * 8;
  const bool in = col < p.n;  // (n is a multiple of 8)
  bool waited = false;
  int id;
  const unsigned firsts = tile_groups(p, t, id);
  const int groups = __popc(firsts);
  const int id0 = __shfl_sync(0xFFFFFFFFu, id, g), id1 = __shfl_sync(0xFFFFFFFFu, id, g + 8);
  const float sa0 = id0 >= -1 ? __ldg(p.sa + r0 + g) : 0.0f, sa1 = id1 >= -1 ? __ldg(p.sa + r0 + g + 8) : 0.0f;
  const int slices = (in && p.per > 0) ? stream::slices_of(col / stream::kRows, p.num_kb, p.per) : 1;
  float4 sw[2] = {};
  if (in) {
    sw[0] = __ldg(reinterpret_cast<const float4*>(p.sw + col));
    sw[1] = __ldg(reinterpret_cast<const float4*>(p.sw + col) + 1);
  }
  for (int n = blockIdx.z; n < groups; n += gridDim.z) {
    const int use = __shfl_sync(0xFFFFFFFFu, id, __fns(firsts, 0, n + 1));
    const unsigned mine = __ballot_sync(0xFFFFFFFFu, id == use);
    float d[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) d[j][i] = 0.0f;
    if (use >= 0) {
      for (int i = tid; i < kTile * steps * 8; i += kExpandThreads) {
        const int row = i / (steps * 8), w = i - row * (steps * 8), r = 2 * w;
        if (!((mine >> row) & 1u)) continue;
        float lo = 0.0f, hi = 0.0f;
        if (r < p.rank) {
          const float* s = p.s + static_cast<int64_t>(r0 + row) * p.rank + r;
#pragma unroll 4
          for (int z = 0; z < p.kparts; ++z) {
            const float2 f = *reinterpret_cast<const float2*>(s + static_cast<int64_t>(z) * p.m * p.rank);
            lo += f.x;
            hi += f.y;
          }
        }
        uint32_t term[3];
        split3(lo, hi, term);
#pragma unroll
        for (int e = 0; e < 3; ++e) ss[(e * kTile + row) * pitch + w] = term[e];
      }
      __syncthreads();
      const __nv_bfloat16* b = p.lb + static_cast<int64_t>(use) * p.n * p.rank;
      const bool in0 = id0 == use, in1 = id1 == use;
#pragma unroll 2
      for (int st = 0; st < steps; ++st) {
        const int r = st * 16 + q * 4;
        uint2 bv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = col0 + (g >> 1) * 8 + j * 2 + (g & 1);
          bv[j] = (c < p.n && r < p.rank)
                      ? __ldg(reinterpret_cast<const uint2*>(b + static_cast<int64_t>(c) * p.rank + r))
                      : make_uint2(0, 0);
        }
#pragma unroll
        for (int e = 0; e < 3; ++e) {
          // (rows of other groups were not written: they must not be read as numbers)
          const uint2 zero = make_uint2(0, 0);
          const uint2 x0 = in0 ? *reinterpret_cast<const uint2*>(&ss[(e * kTile + g) * pitch + st * 8 + q * 2]) : zero;
          const uint2 x1 = in1 ? *reinterpret_cast<const uint2*>(&ss[(e * kTile + g + 8) * pitch + st * 8 + q * 2]) : zero;
          const uint32_t f[4] = {x0.x, x1.x, x0.y, x1.y};
#pragma unroll
          for (int j = 0; j < 4; ++j) mma_bf16(d[j], f, bv[j].x, bv[j].y);
        }
      }
    }
    if (!waited) {
      griddep_wait();
      griddep_launch_dependents();
      waited = true;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if ((h ? id1 : id0) != use || !in) continue;
      const int64_t o = static_cast<int64_t>(r0 + g + h * 8) * p.n + col;
      int4 c0 = *reinterpret_cast<const int4*>(p.c + o), c1 = *reinterpret_cast<const int4*>(p.c + o + 4);
      for (int i = 1; i < slices; ++i) {
        const int32_t* c = p.c + static_cast<int64_t>(i) * p.m * p.n + o;
        const int4 e0 = *reinterpret_cast<const int4*>(c), e1 = *reinterpret_cast<const int4*>(c + 4);
        c0 = make_int4(c0.x + e0.x, c0.y + e0.y, c0.z + e0.z, c0.w + e0.w);
        c1 = make_int4(c1.x + e1.x, c1.y + e1.y, c1.z + e1.z, c1.w + e1.w);
      }
      const float sa = h ? sa1 : sa0;
      auto val = [&](int acc, float s, float add) {
        const float v = __fmul_rn(__fmul_rn(__fmul_rn(__int2float_rn(acc), sa), s), p.alpha);
        return use >= 0 ? __fadd_rn(v, add) : v;
      };
      const float v0 = val(c0.x, sw[0].x, d[0][2 * h]), v1 = val(c0.y, sw[0].y, d[0][2 * h + 1]);
      const float v2 = val(c0.z, sw[0].z, d[1][2 * h]), v3 = val(c0.w, sw[0].w, d[1][2 * h + 1]);
      const float v4 = val(c1.x, sw[1].x, d[2][2 * h]), v5 = val(c1.y, sw[1].y, d[2][2 * h + 1]);
      const float v6 = val(c1.z, sw[1].z, d[3][2 * h]), v7 = val(c1.w, sw[1].w, d[3][2 * h + 1]);
      if (p.out_bf16) {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + o) =
            make_uint4(pack_bf16x2(v0, v1), pack_bf16x2(v2, v3), pack_bf16x2(v4, v5), pack_bf16x2(v6, v7));
      } else {
        float4* out = reinterpret_cast<float4*>(static_cast<float*>(p.out) + o);
        out[0] = make_float4(v0, v1, v2, v3);
        out[1] = make_float4(v4, v5, v6, v7);
      }
    }
    if (n + gridDim.z < groups) __syncthreads();  // s is rewritten
  }
  if (!waited) {
    griddep_wait();
    griddep_launch_dependents();
  }
}

// ---------------------------------------------------------------------------
// The projection's int32 sums for up to 64 tokens.
// ---------------------------------------------------------------------------
struct Dense {
  static constexpr bool kEarlyWeights = true;
  struct Walk {};
  int m;
  const stream::Plan& pl;
  int32_t* c;
  __device__ __forceinline__ int tiles() const { return pl.row_blocks; }
  __device__ __forceinline__ Walk start() const { return {}; }
  __device__ __forceinline__ stream::Tile tile(Walk&, int t) const { return {t * stream::kRows, 0}; }
  __device__ __forceinline__ void store(const Walk&, int, int slice, const stream::Tile& s, uint32_t tmem, int row) const {
    const int col = s.w_row + row;
    int32_t* out = c + static_cast<int64_t>(slice) * m * pl.n + col;
    stream::each_column(tmem, m, [&](int i, int v) {
      if (col < pl.n) out[static_cast<int64_t>(i) * pl.n] = v;
    });
  }
};

__global__ void __launch_bounds__(stream::kThreads, 1)
    lora_stream_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, int m,
                       const __grid_constant__ stream::Plan pl, int32_t* c) {
  extern __shared__ uint8_t raw[];
  __shared__ stream::Bars s;
  if (threadIdx.x == 0) {
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
  }
  stream::setup(s, pl);
  stream::run(Dense{m, pl, c}, pl, s, stream::ring_of(raw), &tmW, &tmX);
  stream::teardown(s);
}

inline bool streams(int m) { return m <= stream::kMaxTokens; }

inline stream::Plan stream_plan(int m, int n, int k, int num_sms) { return stream::plan(m, n, k, num_sms); }

// K parts of s: as many as keep its CTAs, one group a tile, within two an SM, no
// part under 256 (one step of each warp).
inline int shrink_parts(int m, int k, int num_sms) {
  const int tiles = (m + kTile - 1) / kTile, most = m < 4 ? m : 4;
  int parts = 1;
  while (parts < 16 && 2 * tiles * most * parts <= 2 * num_sms && k / (2 * parts) >= 256) parts *= 2;
  return parts;
}

template <bool BF16>
inline cudaError_t launch_shrink_t(const Args& a, cudaStream_t stream) {
  const int most = a.m < kTile ? a.m : kTile;
  const int groups = (a.rank + kRankGroup - 1) / kRankGroup;
  const dim3 grid((a.m + kTile - 1) / kTile, a.adapters < most ? a.adapters : most, a.kparts * groups);
  const dim3 block(kShrinkThreads);
  if (a.rank <= 16) return launch_pdl(lora_shrink_kernel<BF16, 2>, grid, block, 0, stream, 1, a);
  if (a.rank <= 32) return launch_pdl(lora_shrink_kernel<BF16, 4>, grid, block, 0, stream, 1, a);
  return launch_pdl(lora_shrink_kernel<BF16, 8>, grid, block, 0, stream, 1, a);
}

inline cudaError_t launch_shrink(const Args& a, bool x_bf16, cudaStream_t stream) {
  return x_bf16 ? launch_shrink_t<true>(a, stream) : launch_shrink_t<false>(a, stream);
}

// Returns 0, 1 when a tensor map could not be made, 2 with *err set.
inline int launch_stream(const Args& a, const int8_t* x, const int8_t* w, const stream::Plan& pl, int dev, int num_sms,
                         cudaStream_t stream, cudaError_t* err) {
  CUtensorMap tw, tx;
  if (!gemm::cached_tmap(&tw, w, a.n, a.k, stream::kRows) || !gemm::cached_tmap(&tx, x, a.m, a.k, pl.nb)) return 1;
  if ((*err = gemm::set_smem_once(lora_stream_kernel, dev, 0, stream::kRingBytes + 1024)) != cudaSuccess) return 2;
  *err = launch_pdl(lora_stream_kernel, dim3(num_sms), dim3(stream::kThreads), stream::smem_bytes(pl), stream, 1, tw, tx,
                    a.m, pl, const_cast<int32_t*>(a.c));
  return *err == cudaSuccess ? 0 : 2;
}

// Groups a tile can have go to CTAs of their own while the grid stays within
// sixteen CTAs an SM.
inline cudaError_t launch_expand(const Args& a, int num_sms, cudaStream_t stream) {
  const int64_t tiles = (a.m + kTile - 1) / kTile, cols = (a.n + kExpandCols - 1) / kExpandCols;
  const int most = a.m < kTile ? a.m : kTile, groups = a.adapters < most ? a.adapters + 1 : most;
  int64_t z = 16LL * num_sms / (tiles * cols);
  z = z < 1 ? 1 : (z > groups ? groups : z);
  return launch_pdl(lora_expand_kernel, dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(cols), static_cast<unsigned>(z)),
                    dim3(kExpandThreads), expand_smem(a.rank), stream, 1, a);
}

}  // namespace lora
}  // namespace qk
