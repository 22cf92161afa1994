// lora.cuh -- low-rank adapters of many requests beside the shared W8A8
// projection: out = epilogue(a b^T) + s B[id]^T, s = lora_scale[id] * x A[id]^T,
// where token i uses adapter id = ids[i] (none when outside [0, adapters)).
//
// Three kernels: the projection's int32 sums, s (the tokens into the adapters'
// ranks), and the output: the sums' epilogue plus s B^T, rounded once.  Up to 64
// tokens the sums are the stream of stream.cuh, which runs first and leaves room
// on its SMs: s is formed beside it (and waits for it at its end, so that the
// last kernel, which waits for s, waits for both).  Beyond, the GEMM fills the
// SMs, and s comes first, after a kernel that groups the tokens.
//
// Both small products run on the bf16 matrix instruction, 16 rows at a time.
// A bf16 value is exact there; a binary32 one (s, and x when it is fp32) enters
// as three bf16 terms, x = h + m + l, each the rounding of what is left: 24 bits,
// so a product of 16 of them is as good as one of binary32 values.  The 16 rows
// are tokens of ONE adapter, gathered from wherever they lie: from the whole batch
// up to 64 tokens (every CTA sorts them for itself), from 1024 tokens in a row
// beyond (a first kernel sorts those).  So an adapter is read for its own tokens
// only, however requests are mixed, and one that holds NaN or infinity reaches no
// other's rows.  (Tiles of 16 tokens in a row, an adapter present there after
// another, took 299 us for 1024 x 4096 x 4096, rank 128, 24 adapters in any order;
// groups take 73 us.)
//
// Bounds.  A few tokens: reading the weights, 4 x 14336 x 4096 rank 16 in 17 us (61
// MB); 64 x 4096 x 4096 with 32 adapters of rank 64 in 21.9 us (52 MB: the output
// kernel takes its half of the adapters from L2, but only after the sums).  A
// prompt: 4096 x 4096 x 4096 rank 16 in 94 us (98-100 under the power cap), of which the
// GEMM with int32 sums takes 52 (50.5 with bf16 output), s 13, the groups 3.5 and the
// output 29, which reads the 64 MB of sums: its registers leave four warps a scheduler,
// each in a chain of shared-memory reads, products and conversions (0.44 instructions a
// cycle of each scheduler).
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
  int beside;                 // the sums are formed before s, and beside it
  int32_t* units;             // workspace of a longer batch: [chunks, kMaxUnits] records of groups
  int32_t* counts;            // [chunks]: groups of a chunk
  int most;                   // groups a chunk can have with these adapters
};

constexpr int kTile = 16;     // rows of a group
constexpr int kChunk = 1024;  // tokens sorted together
constexpr int kMaxUnits = kChunk + kChunk / kTile;  // groups of a chunk, at most
constexpr int kRecord = 20;   // words of a group's record: the adapter, 16 tokens, 3 unused
constexpr int kMaxParts = 8;  // K parts of s

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

// Two binary32 values as three pairs of bf16 terms.  The first saturates: a value above
// the largest bf16 one leaves a finite rest (24 bits hold), and an infinite one an
// infinite rest, which is the second term; its own rest, inf - inf, counts as 0, so that
// the terms add up to the infinity.  (A NaN is in the first two terms already.)
__device__ __forceinline__ void split3(float lo, float hi, uint32_t (&t)[3]) {
  asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(t[0]) : "f"(hi), "f"(lo));
  lo = __fsub_rn(lo, bf16_lo(t[0]));
  hi = __fsub_rn(hi, bf16_hi(t[0]));
  t[1] = pack_bf16x2(lo, hi);
  lo = __fsub_rn(lo, bf16_lo(t[1]));
  hi = __fsub_rn(hi, bf16_hi(t[1]));
  t[2] = pack_bf16x2(lo == lo ? lo : 0.0f, hi == hi ? hi : 0.0f);
}

// 16 rows of one adapter (or of none: -1).
struct Group {
  int use;
  int tok[kTile];  // -1: no token
};

// Unit `u` of a batch of up to 64 tokens: adapters in the order of their first
// tokens, an adapter's tokens 16 to a unit.  By warp 0; false when there is none.
// Without `none`, tokens without an adapter are passed over.
__device__ __forceinline__ bool gather_unit(const Args& p, int u, bool none, Group& gr) {
  const int lane = threadIdx.x & 31;
  int id[2];
  uint64_t same[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    id[h] = h * 32 + lane < p.m ? adapter_of(p, h * 32 + lane) : -2;
    same[h] = 0;
  }
  const int halves = p.m > 32 ? 2 : 1;
  same[0] = __match_any_sync(0xFFFFFFFFu, id[0]);
  if (halves == 2) {
    same[1] = static_cast<uint64_t>(__match_any_sync(0xFFFFFFFFu, id[1])) << 32;
#pragma unroll 8
    for (int j = 0; j < 32; ++j) {
      const int lo = __shfl_sync(0xFFFFFFFFu, id[0], j), hi = __shfl_sync(0xFFFFFFFFu, id[1], j);
      if (id[1] == lo) same[1] |= 1ull << j;
      if (id[0] == hi) same[0] |= 1ull << (32 + j);
    }
  }
  int base = 0;
  bool found = false;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (h == halves) break;
    const bool leads = id[h] >= (none ? -1 : 0) && (same[h] & ((1ull << (32 * h + lane)) - 1ull)) == 0;
    const int units = leads ? (__popcll(same[h]) + kTile - 1) / kTile : 0;
    int sum = units;  // inclusive prefix
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
      if (lane >= o) sum += v;
    }
    const int at = base + sum - units;
    const unsigned here = __ballot_sync(0xFFFFFFFFu, u >= at && u < at + units);
    if (here != 0) {
      const int src = __ffs(here) - 1;
      uint64_t mask = __shfl_sync(0xFFFFFFFFu, same[h], src);
      const int skip = (u - __shfl_sync(0xFFFFFFFFu, at, src)) * kTile + lane;
      const int use = __shfl_sync(0xFFFFFFFFu, id[h], src);
      if (lane == 0) gr.use = use;
      if (lane < kTile) {
        for (int n = 0; n < skip && mask != 0; ++n) mask &= mask - 1ull;
        gr.tok[lane] = mask != 0 ? __ffsll(static_cast<long long>(mask)) - 1 : -1;
      }
      found = true;
    }
    base += __shfl_sync(0xFFFFFFFFu, sum, 31);
  }
  return found;
}

// This CTA's group (blockIdx.x), by all threads; false when there is none.
template <bool BESIDE>
__device__ __forceinline__ bool group_of_cta(const Args& p, bool none, Group& gr, int& ok) {
  const int tid = threadIdx.x;
  if constexpr (BESIDE) {
    if (tid < 32) {
      const bool found = gather_unit(p, blockIdx.x, none, gr);
      if (tid == 0) ok = found ? 1 : 0;
    }
  } else {
    const int chunk = blockIdx.x / p.most, u = blockIdx.x - chunk * p.most;
    const int32_t* rec = p.units + (static_cast<int64_t>(chunk) * kMaxUnits + u) * kRecord;
    const bool found = u < p.counts[chunk] && (none || rec[0] >= 0);
    if (tid == 0) {
      ok = found ? 1 : 0;
      if (found) gr.use = rec[0];
    }
    if (found && tid < kTile) gr.tok[tid] = rec[1 + tid];
  }
  __syncthreads();
  return ok != 0;
}

// The groups of 1024 tokens, one CTA.  A prompt's tokens lie together: where there
// are at most as many runs of an adapter's tokens as adapters, 32 at most, each run
// is taken as it stands.  Else a bitonic sort of (adapter + 1, token) in one word, 32
// apart through shared memory, nearer ones by shuffles.  Then a token's place in its
// run gives its group and its row there.
__global__ void __launch_bounds__(kChunk) lora_units_kernel(Args p) {
  __shared__ uint32_t buf[kChunk + 1];
  __shared__ int warp_start[kChunk / 32], warp_units[kChunk / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5, row = blockIdx.x * kChunk + i;
  uint32_t key = row < p.m ? (static_cast<uint32_t>(adapter_of(p, row) + 1) << 10) | static_cast<uint32_t>(i) : 0xFFFFFFFFu;
  buf[i] = key;
  __syncthreads();
  const int runs = __syncthreads_count(i > 0 && row < p.m && (buf[i - 1] >> 10) != (key >> 10)) + 1;
  for (int k = runs <= min(p.adapters + 1, 32) ? 2 * kChunk : 2; k <= kChunk; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      uint32_t other;
      if (j >= 32) {
        __syncthreads();
        buf[i] = key;
        __syncthreads();
        other = buf[i ^ j];
      } else {
        other = __shfl_xor_sync(0xFFFFFFFFu, key, j);
      }
      const bool smaller = ((i & j) == 0) == ((i & k) == 0);
      key = smaller ? min(key, other) : max(key, other);
    }
  }
  __syncthreads();
  buf[i] = key;
  if (i == 0) buf[kChunk] = 0xFFFFFFFFu;
  __syncthreads();
  const bool valid = key != 0xFFFFFFFFu;
  const uint32_t id = key >> 10;
  const bool first = valid && (i == 0 || (buf[i - 1] >> 10) != id), last = valid && (buf[i + 1] >> 10) != id;
  // the run's first token: a running maximum of first tokens' places
  int start = first ? i : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, start, o);
    if (lane >= o) start = max(start, v);
  }
  if (lane == 31) warp_start[warp] = start;
  __syncthreads();
  start = max(start, __reduce_max_sync(0xFFFFFFFFu, lane < warp ? warp_start[lane] : 0));
  const int pos = i - start, slot = pos & (kTile - 1);
  const bool opens = valid && slot == 0;
  const unsigned open = __ballot_sync(0xFFFFFFFFu, opens);
  if (lane == 0) warp_units[warp] = __popc(open);
  __syncthreads();
  const int units = warp_units[lane], before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? units : 0);
  const int unit = before + __popc(open & ((2u << lane) - 1u)) - 1, all = __reduce_add_sync(0xFFFFFFFFu, units);
  if (i == 0) p.counts[blockIdx.x] = all;
  if (valid) {
    int32_t* rec = p.units + (static_cast<int64_t>(blockIdx.x) * kMaxUnits + unit) * kRecord;
    if (opens) rec[0] = static_cast<int>(id) - 1;
    rec[1 + slot] = blockIdx.x * kChunk + static_cast<int>(key & (kChunk - 1));
    if (last)
      for (int e = slot + 1; e < kTile; ++e) rec[1 + e] = -1;
  }
}

// ---------------------------------------------------------------------------
// s: one CTA per (group, K part and 64 ranks); its 8 warps deal the part's K in
// steps of 32 and each multiplies all ranks.  The operands come straight from
// memory: a dot product may sum K in any order, so thread (g, q) takes elements
// 8 q .. 8 q + 7 of a step (16 bytes) of rows g and g + 8 and of the adapter's row,
// four of them for each of two instructions, in the places (2 q, 2 q + 1) and
// (2 q + 8, 2 q + 9) those have for it.
// ---------------------------------------------------------------------------
constexpr int kShrinkThreads = 256;
constexpr int kShrinkStep = 32;
constexpr int kRankGroup = 64;

// Elements at .. at + 7 of x, and their four pairs as bf16 terms.
template <bool BF16>
__device__ __forceinline__ void load_x(const void* x, int64_t at, bool in, uint4 (&v)[BF16 ? 1 : 2]) {
  const char* p = static_cast<const char*>(x) + at * (BF16 ? 2 : 4);
#pragma unroll
  for (int i = 0; i < (BF16 ? 1 : 2); ++i)
    v[i] = in ? ld_nc_v4(p + i * 16) : vec4(0, 0, 0, 0);
}
template <bool BF16>
__device__ __forceinline__ void terms_x(const uint4 (&v)[BF16 ? 1 : 2], uint32_t (&t)[4][BF16 ? 1 : 3]) {
  if constexpr (BF16) {
    t[0][0] = v[0].x;
    t[1][0] = v[0].y;
    t[2][0] = v[0].z;
    t[3][0] = v[0].w;
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      split3(__uint_as_float(v[i].x), __uint_as_float(v[i].y), t[2 * i]);
      split3(__uint_as_float(v[i].z), __uint_as_float(v[i].w), t[2 * i + 1]);
    }
  }
}

// RT: tiles of 8 ranks.  BESIDE: the sums are formed before s, and beside it; a kernel of
// its own, since the split of shared memory it asks for to stand beside them stays with a
// kernel (as one of both, a short batch slowed the long ones after it in the process: 4096
// x 4096 x 4096 rank 16 from 93 to 101 us, 1024 x 4096 x 4096 rank 128 from 73 to 81).
template <bool BF16, int RT, bool BESIDE>
__global__ void __launch_bounds__(kShrinkThreads, 2) lora_shrink_kernel(Args p) {
  constexpr int NW = kShrinkThreads / 32, TERMS = BF16 ? 1 : 3, XV = BF16 ? 1 : 2;
  __shared__ float red[NW][kTile][RT * 8 + 1];
  __shared__ Group gr;
  __shared__ int ok;
  // (beside the sums: x, the adapters and ids are the caller's, complete before the
  // kernel of the sums let this one start, and s is free)
  if constexpr (!BESIDE) griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  if (!group_of_cta<BESIDE>(p, false, gr, ok)) {
    if constexpr (BESIDE) griddep_wait();
    return;
  }
  const int use = gr.use, tok0 = gr.tok[g], tok1 = gr.tok[g + 8];
  const int z = blockIdx.z % p.kparts, rg = blockIdx.z / p.kparts * kRankGroup, ranks = min(p.rank - rg, kRankGroup);
  const int k0 = z * p.kpart, k1 = min(p.k, k0 + p.kpart);
  const __nv_bfloat16* a = p.la + (static_cast<int64_t>(use) * p.rank + rg) * p.k;
  float acc[RT][4];
#pragma unroll
  for (int j = 0; j < RT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
  // U steps' loads are issued together (ld_nc_v4 and mma_bf16 are volatile: they
  // keep their order)
  constexpr int U = RT <= 2 ? 4 : ((RT <= 4 || BF16) ? 2 : 1), ROW = NW * kShrinkStep;
  for (int k = k0 + warp * kShrinkStep + q * 8; k < k1 + q * 8; k += U * ROW) {
    uint4 x0[U][XV], x1[U][XV], b[U][RT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int ku = k + u * ROW;
      const bool in = ku < k1;  // (K is a multiple of 16: the last step may be half one)
      load_x<BF16>(p.x, static_cast<int64_t>(tok0) * p.k + ku, tok0 >= 0 && in, x0[u]);
      load_x<BF16>(p.x, static_cast<int64_t>(tok1) * p.k + ku, tok1 >= 0 && in, x1[u]);
#pragma unroll
      for (int j = 0; j < RT; ++j)
        b[u][j] = (j * 8 < ranks && in) ? ld_nc_v4(a + static_cast<int64_t>(j * 8 + g) * p.k + ku) : vec4(0, 0, 0, 0);
    }
    // The instruction truncates as it accumulates: a batch's products are summed on
    // their own, the smallest terms first, and added to the rest with rounding (300
    // fp32 tokens of 8192 values, rank 128, all positive: s is within 1.9e-7 of the exact
    // value, relative, and within 9.6e-7 as a single chain).
    float part[RT][4];
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[j][i] = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t t0[4][TERMS], t1[4][TERMS];
      terms_x<BF16>(x0[u], t0);
      terms_x<BF16>(x1[u], t1);
#pragma unroll
      for (int i = TERMS - 1; i >= 0; --i) {
        const uint32_t f0[4] = {t0[0][i], t1[0][i], t0[1][i], t1[1][i]};
        const uint32_t f1[4] = {t0[2][i], t1[2][i], t0[3][i], t1[3][i]};
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          mma_bf16(part[j], f0, b[u][j].x, b[u][j].y);
          mma_bf16(part[j], f1, b[u][j].z, b[u][j].w);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = __fadd_rn(acc[j][i], part[j][i]);
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
    if (gr.tok[row] < 0) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += red[w][row][r];
    s[static_cast<int64_t>(gr.tok[row]) * p.rank + r] = ls * v;
  }
  if constexpr (BESIDE) {
    // The next kernel has no room beside these before the sums are done: its rows of
    // the adapter are brought into L2 meanwhile, a part by each CTA of the group,
    // where that part is no more than its work here (64 x 4096 x 4096 rank 64, 32
    // adapters: 22.7 -> 22.1 us, 32 x 8192 x 8192 rank 128, 8 adapters: 34.5 -> 32.9;
    // 256 KB of 450 KB each for 64 x 14336 x 4096 rank 64: 44.8 -> 45.7, against the
    // weights' own stream).
    const int64_t bytes = static_cast<int64_t>(p.n) * p.rank * 2, part = (bytes + gridDim.z - 1) / gridDim.z;
    if (part <= 256 * 1024) {
      const char* lb = reinterpret_cast<const char*>(p.lb) + static_cast<int64_t>(use) * bytes;
      const int64_t from = part * blockIdx.z, to = min(bytes, from + part);
      for (int64_t i = from + tid * 128; i < to; i += kShrinkThreads * 128) prefetch_l2(lb + i);
    }
    griddep_wait();
  }
}

// ---------------------------------------------------------------------------
// out, up to 64 tokens: a CTA takes the 16 rows of a group by 512 columns, a warp
// 32 of each half.  Column 2 q + b of the j-th product of a warp stands for column
// 8 q + 2 j + b of its 32, so that a thread ends up with 8 consecutive columns of
// rows g and g + 8: 16-byte reads of the sums, 16-byte writes.  The adapter's rows
// and the scales of both halves are requested before the wait (they are the
// caller's), then the sums and s.
// ---------------------------------------------------------------------------
constexpr int kExpandThreads = 256;
constexpr int kHalves = 2;
constexpr int kExpandCols = 256 * kHalves;
constexpr int kSlices = 3;  // of the sums, at most (a CTA takes at least half of a tile)

inline size_t expand_smem(int rank) { return static_cast<size_t>(3) * kTile * ((rank + 31) / 32 * 16 + 4) * 4; }

// Columns col .. col + 7 of row `row`: the sums' epilogue, in the GEMM's order, and
// the adapter's part.
__device__ __forceinline__ void store8(const Args& p, int row, int col, const int4& c0, const int4& c1, float sa,
                                       const float4& w0, const float4& w1, bool adapter, float d0, float d1, float d2,
                                       float d3, float d4, float d5, float d6, float d7) {
  auto val = [&](int acc, float sw, float add) {
    const float f = __fmul_rn(__fmul_rn(__fmul_rn(__int2float_rn(acc), sa), sw), p.alpha);
    return adapter ? __fadd_rn(f, add) : f;
  };
  const float v0 = val(c0.x, w0.x, d0), v1 = val(c0.y, w0.y, d1), v2 = val(c0.z, w0.z, d2), v3 = val(c0.w, w0.w, d3);
  const float v4 = val(c1.x, w1.x, d4), v5 = val(c1.y, w1.y, d5), v6 = val(c1.z, w1.z, d6), v7 = val(c1.w, w1.w, d7);
  const uint64_t o = static_cast<uint64_t>(static_cast<uint32_t>(row)) * static_cast<uint32_t>(p.n) + static_cast<uint32_t>(col);
  if (p.out_bf16) {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + o) =
        vec4(pack_bf16x2(v0, v1), pack_bf16x2(v2, v3), pack_bf16x2(v4, v5), pack_bf16x2(v6, v7));
  } else {
    float4* out = reinterpret_cast<float4*>(static_cast<float*>(p.out) + o);
    out[0] = make_float4(v0, v1, v2, v3);
    out[1] = make_float4(v4, v5, v6, v7);
  }
}

__global__ void __launch_bounds__(kExpandThreads, 2) lora_expand_kernel(Args p) {
  extern __shared__ uint32_t ss[];  // s: [term][row][rank / 2 words], rows padded by 16 bytes
  __shared__ Group gr;
  __shared__ int ok;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const int steps = (p.rank + 31) / 32, pitch = steps * 16 + 4;
  const int col0 = blockIdx.y * kExpandCols + warp * 32;  // of the first half
  const int64_t slice = static_cast<int64_t>(p.m) * p.n;
  float4 sw[kHalves][2];
#pragma unroll
  for (int v = 0; v < kHalves; ++v) {
    const int col = col0 + v * 256 + q * 8;
    const bool in = col < p.n;  // (n is a multiple of 8)
    sw[v][0] = in ? __ldg(reinterpret_cast<const float4*>(p.sw + col)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    sw[v][1] = in ? __ldg(reinterpret_cast<const float4*>(p.sw + col) + 1) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  if (!group_of_cta<true>(p, true, gr, ok)) {
    griddep_wait();
    return;
  }
  const int use = gr.use;
  const __nv_bfloat16* b = p.lb + static_cast<int64_t>(use) * p.n * p.rank;
  uint4 bv[kHalves][4];
  auto request = [&](int v, int st) {  // 32 ranks of the adapter's rows
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = st * 32 + q * 8, c = col0 + v * 256 + (g >> 1) * 8 + j * 2 + (g & 1);
      bv[v][j] = (c < p.n && r < p.rank) ? ld_nc_v4(b + static_cast<int64_t>(c) * p.rank + r) : vec4(0, 0, 0, 0);
    }
  };
  if (use >= 0) {
#pragma unroll
    for (int v = 0; v < kHalves; ++v) request(v, 0);
  }
  float sa[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int tok = gr.tok[g + h * 8];
    sa[h] = tok >= 0 ? __ldg(p.sa + tok) : 0.0f;
  }
  // s of pair of ranks w of a row, its K parts
  auto s_of = [&](int i, float2 (&f)[kMaxParts]) {
    const int row = i / (steps * 16), w = i - row * (steps * 16), tok = gr.tok[row];
    const bool on = tok >= 0 && 2 * w < p.rank;
    const float* s = p.s + static_cast<int64_t>(on ? tok : 0) * p.rank + (on ? 2 * w : 0);
#pragma unroll
    for (int z = 0; z < kMaxParts; ++z)
      f[z] = on && z < p.kparts ? *reinterpret_cast<const float2*>(s + static_cast<int64_t>(z) * p.m * p.rank)
                                : make_float2(0.0f, 0.0f);
  };
  griddep_wait();
  griddep_launch_dependents();
  float2 f[kMaxParts];  // (requested before the sums: its use comes first)
  if (use >= 0) s_of(tid, f);
  int4 c0[kHalves][2], c1[kHalves][2];  // the sums of rows g and g + 8
#pragma unroll
  for (int v = 0; v < kHalves; ++v) {
    const int col = col0 + v * 256 + q * 8;
    const int slices = p.per > 0 ? stream::slices_of(min(col, p.n - 1) / stream::kRows, p.num_kb, p.per) : 1;
    int4 e0[2][kSlices - 1], e1[2][kSlices - 1];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int tok = gr.tok[g + h * 8];
      const bool in = tok >= 0 && col < p.n;
      const int4 zero = make_int4(0, 0, 0, 0);
      const int32_t* c = p.c + static_cast<int64_t>(in ? tok : 0) * p.n + (in ? col : 0);
      c0[v][h] = in ? *reinterpret_cast<const int4*>(c) : zero;
      c1[v][h] = in ? *reinterpret_cast<const int4*>(c + 4) : zero;
#pragma unroll
      for (int i = 0; i < kSlices - 1; ++i) {
        const bool on = in && i + 1 < slices;
        e0[h][i] = on ? *reinterpret_cast<const int4*>(c + (i + 1) * slice) : zero;
        e1[h][i] = on ? *reinterpret_cast<const int4*>(c + (i + 1) * slice + 4) : zero;
      }
    }
    auto add = [](int4& x, const int4& y) { x = make_int4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w); };
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < kSlices - 1; ++i) {
        add(c0[v][h], e0[h][i]);
        add(c1[v][h], e1[h][i]);
      }
  }
  if (use >= 0) {
    for (int i = tid; i < kTile * steps * 16; i += kExpandThreads) {
      const int row = i / (steps * 16), w = i - row * (steps * 16);
      if (i != tid) s_of(i, f);
#pragma unroll
      for (int z = 1; z < kMaxParts; ++z) {
        f[0].x += f[z].x;
        f[0].y += f[z].y;
      }
      uint32_t term[3];
      split3(f[0].x, f[0].y, term);
#pragma unroll
      for (int e = 0; e < 3; ++e) ss[(e * kTile + row) * pitch + w] = term[e];
    }
    __syncthreads();
  }
#pragma unroll
  for (int v = 0; v < kHalves; ++v) {
    const int col = col0 + v * 256 + q * 8;
    float d[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) d[j][i] = 0.0f;
    if (use >= 0) {
      for (int st = 0; st < steps; ++st) {
        if (st > 0) request(v, st);
        const int at = st * 16 + q * 4;
#pragma unroll
        for (int e = 2; e >= 0; --e) {
          const uint4 x0 = *reinterpret_cast<const uint4*>(&ss[(e * kTile + g) * pitch + at]);
          const uint4 x1 = *reinterpret_cast<const uint4*>(&ss[(e * kTile + g + 8) * pitch + at]);
          const uint32_t f0[4] = {x0.x, x1.x, x0.y, x1.y}, f1[4] = {x0.z, x1.z, x0.w, x1.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            mma_bf16(d[j], f0, bv[v][j].x, bv[v][j].y);
            mma_bf16(d[j], f1, bv[v][j].z, bv[v][j].w);
          }
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int tok = gr.tok[g + h * 8];
      if (tok < 0 || col >= p.n) continue;
      store8(p, tok, col, c0[v][h], c1[v][h], sa[h], sw[v][0], sw[v][1], use >= 0, d[0][2 * h], d[0][2 * h + 1],
             d[1][2 * h], d[1][2 * h + 1], d[2][2 * h], d[2][2 * h + 1], d[3][2 * h], d[3][2 * h + 1]);
    }
  }
}

// ---------------------------------------------------------------------------
// out, longer batches: a CTA walks its share of the groups, in order, at its 256
// columns, with the next group's s and the next groups' sums in flight while the
// current one is multiplied and stored, so that it reads and writes without a pause.
// (A warp copies the sums it will use itself, asynchronously, eight lanes a row so
// that each fetches whole sectors: no registers, no barrier of the CTA.)  Consecutive
// groups mostly share their adapter, whose rows stay where they are until it changes:
// in registers up to 32 ranks, in a thread's own places in shared memory beyond.
// ---------------------------------------------------------------------------
constexpr int kSumBytes = kTile * 256 * 4;  // of one group
constexpr int kRecords = 8, kRecordsAhead = 7;

// Groups' sums in shared memory, and buffers of s: two CTAs an SM at 128 ranks too
// (4096 x 2048 x 2048, 24 mixed adapters: 106 us with one CTA and four groups, 97 us
// so).
template <int RK>
constexpr int kSumTiles = RK > 64 ? 2 : 4;
template <int RK>
constexpr int kTermBuffers = RK > 64 ? 1 : 2;

template <int RK>
constexpr size_t long_smem() {
  return static_cast<size_t>(kSumTiles<RK>) * kSumBytes + (RK > 32 ? kExpandThreads * RK * 2 : 0);
}

template <int RK>  // ranks, rounded up to 16, 32, 64 or 128
__global__ void __launch_bounds__(kExpandThreads, 2) lora_expand_long_kernel(Args p) {
  // ranks a thread takes of a step (as two instructions' operands, or one's)
  constexpr int STEP = RK < 32 ? 16 : 32, STEPS = RK / STEP, HALVES = STEP / 16, VEC = STEP / 4;
  constexpr int TILES = kSumTiles<RK>, BUFS = kTermBuffers<RK>;
  constexpr int WORDS = RK / 2, PITCH = WORDS + 4, SV = (kTile * WORDS + kExpandThreads - 1) / kExpandThreads;
  // the sums: [group][warp][row][8 pieces of 16 bytes, a pair exchanged in odd rows];
  // the adapter's rows: [step][product][thread][16 bytes]
  extern __shared__ __align__(16) uint8_t cs[];
  __shared__ __align__(16) uint32_t ss[BUFS][3][kTile][PITCH];  // s: [buffer][term][row][pair of ranks]
  __shared__ __align__(16) int recs[kRecords][kRecord];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const int col0 = blockIdx.y * 256 + warp * 32, col = col0 + q * 8;
  const bool in = col < p.n;  // (n is a multiple of 8)
  float4 sw[2] = {};
  if (in) {
    sw[0] = __ldg(reinterpret_cast<const float4*>(p.sw + col));
    sw[1] = __ldg(reinterpret_cast<const float4*>(p.sw + col) + 1);
  }
  // (every kernel from the groups to the product lets the next one start only after
  // its own wait: groups and s are complete, only the sums are not)
  // this CTA's groups: [walk, end) of all chunks' together
  const int chunks = (p.m + kChunk - 1) / kChunk;
  int total = 0;
  for (int c = 0; c < chunks; ++c) total += __ldg(p.counts + c);
  int walk = static_cast<int>(static_cast<int64_t>(total) * blockIdx.x / gridDim.x);
  const int end = static_cast<int>(static_cast<int64_t>(total) * (blockIdx.x + 1) / gridDim.x);
  const unsigned mine = end - walk;
  if (mine == 0) {
    griddep_wait();
    return;
  }
  int chunk = 0, base = 0, count = __ldg(p.counts);
  auto record = [&](unsigned i) {  // requests the record of this CTA's group i (they are asked for in order)
    if (walk >= end) return;
    while (walk - base >= count) {
      base += count;
      count = __ldg(p.counts + ++chunk);
    }
    const int32_t* src = p.units + (static_cast<int64_t>(chunk) * kMaxUnits + walk - base) * kRecord;
    if (tid < kRecord / 4) cp_async16(smem_addr(&recs[i % kRecords][tid * 4]), src + tid * 4, true);
    ++walk;
  };
  // (a row of c or out is less than 2^26 bytes: an address is one multiply-add)
  const int r0 = lane >> 3, piece = lane & 7;
  const bool piece_in = col0 + piece * 4 < p.n;
  const char* c_col = reinterpret_cast<const char*>(p.c + (piece_in ? col0 + piece * 4 : 0));
  const uint32_t c_row = static_cast<uint32_t>(p.n) * 4u;
  const uint32_t cs_put = smem_addr(cs) + warp * (kTile * 128) + r0 * 128 + (piece ^ (r0 & 1)) * 16;
  auto sums = [&](unsigned i) {  // requests the sums of group i
    if (i >= mine) return;
    const int* rec = recs[i % kRecords] + 1 + r0;
    const uint32_t dst = cs_put + (i % TILES) * kSumBytes;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int tok = rec[h * 4];
      cp_async16(dst + h * 512, c_col + static_cast<uint64_t>(static_cast<uint32_t>(max(tok, 0))) * c_row,
                 piece_in && tok >= 0);
    }
  };
  float sa_n[2];
  float2 s_n[SV];
  auto fetch = [&](unsigned i) {  // s and the tokens' scales of group i
    if (i >= mine) return;
    const int* rec = recs[i % kRecords];
    const bool has = rec[0] >= 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int tok = rec[1 + g + h * 8];
      sa_n[h] = tok >= 0 ? __ldg(p.sa + tok) : 0.0f;
    }
#pragma unroll
    for (int v = 0; v < SV; ++v) {
      const int at = tid + v * kExpandThreads, row = at / WORDS, r = 2 * (at % WORDS);
      s_n[v] = make_float2(0.0f, 0.0f);
      if (row < kTile && r < p.rank && has) {
        const int tok = rec[1 + row];
        if (tok >= 0) {
          const float* s = p.s + static_cast<int64_t>(tok) * p.rank + r;
          s_n[v] = *reinterpret_cast<const float2*>(s);
          for (int z = 1; z < p.kparts; ++z) {
            const float2 f = *reinterpret_cast<const float2*>(s + static_cast<int64_t>(z) * p.m * p.rank);
            s_n[v].x += f.x;
            s_n[v].y += f.y;
          }
        }
      }
    }
  };
  for (unsigned i = 0; i < kRecordsAhead; ++i) record(i);
  cp_async_commit();
  cp_async_wait_all();
  __syncthreads();
  fetch(0);
  griddep_wait();
  griddep_launch_dependents();
  for (unsigned i = 0; i < TILES - 1; ++i) {
    sums(i);
    cp_async_commit();
  }
  uint32_t bv[4][VEC / 2];
  int held = -1;  // the adapter whose rows are held
  for (unsigned i = 0; i < mine; ++i) {
    const int* rec = recs[i % kRecords];
    const int use = rec[0], par = i % BUFS;
    const float sa[2] = {sa_n[0], sa_n[1]};
    if (BUFS == 1 && i > 0) __syncthreads();  // (s of the last group has been read)
    if (use >= 0) {
#pragma unroll
      for (int v = 0; v < SV; ++v) {
        const int at = tid + v * kExpandThreads;
        if (at < kTile * WORDS) {
          uint32_t term[3];
          split3(s_n[v].x, s_n[v].y, term);
#pragma unroll
          for (int e = 0; e < 3; ++e) ss[par][e][at / WORDS][at % WORDS] = term[e];
        }
      }
    }
    // (s and the records that were waited for below are there for every thread)
    __syncthreads();
    sums(i + TILES - 1);
    record(i + kRecordsAhead);
    cp_async_commit();
    fetch(i + 1);
    float d[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) d[j][e] = use >= 0 ? 0.0f : -0.0f;  // (x + -0 is x, for -0 too)
    if (use >= 0) {
      uint8_t* bs = cs + TILES * kSumBytes + tid * 16;
      if (held != use) {
        const __nv_bfloat16* b = p.lb + static_cast<int64_t>(use) * p.n * p.rank;
#pragma unroll
        for (int st = 0; st < STEPS; ++st) {
          if (RK > 64 && st * STEP >= p.rank) break;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = st * STEP + q * VEC, cb = col0 + (g >> 1) * 8 + j * 2 + (g & 1);
            const bool on = cb < p.n && r < p.rank;
            const __nv_bfloat16* at = on ? b + static_cast<int64_t>(cb) * p.rank + r : b;
            if constexpr (RK > 32) {
              cp_async16(smem_addr(bs) + (st * 4 + j) * kExpandThreads * 16, at, on);
            } else if constexpr (HALVES == 2) {
              const uint4 v = on ? __ldg(reinterpret_cast<const uint4*>(at)) : vec4(0, 0, 0, 0);
              bv[j][0] = v.x;
              bv[j][1] = v.y;
              bv[j][2] = v.z;
              bv[j][3] = v.w;
            } else {
              const uint2 v = on ? __ldg(reinterpret_cast<const uint2*>(at)) : make_uint2(0, 0);
              bv[j][0] = v.x;
              bv[j][1] = v.y;
            }
          }
        }
        if constexpr (RK > 32) {
          cp_async_commit();
          cp_async_wait_all();
        }
        held = use;
      }
#pragma unroll
      for (int st = 0; st < STEPS; ++st) {
        if (RK > 64 && st * STEP >= p.rank) break;
        if constexpr (RK > 32) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 v = *reinterpret_cast<const uint4*>(bs + (st * 4 + j) * kExpandThreads * 16);
            bv[j][0] = v.x;
            bv[j][1] = v.y;
            bv[j][2] = v.z;
            bv[j][3] = v.w;
          }
        }
#pragma unroll
        for (int e = 2; e >= 0; --e) {  // the smallest terms first
          uint32_t x0[VEC / 2], x1[VEC / 2];
          const uint32_t* a0 = &ss[par][e][g][st * (STEP / 2) + q * (VEC / 2)];
          const uint32_t* a1 = &ss[par][e][g + 8][st * (STEP / 2) + q * (VEC / 2)];
          if constexpr (HALVES == 2) {
            const uint4 v0 = *reinterpret_cast<const uint4*>(a0), v1 = *reinterpret_cast<const uint4*>(a1);
            x0[0] = v0.x, x0[1] = v0.y, x0[2] = v0.z, x0[3] = v0.w;
            x1[0] = v1.x, x1[1] = v1.y, x1[2] = v1.z, x1[3] = v1.w;
          } else {
            const uint2 v0 = *reinterpret_cast<const uint2*>(a0), v1 = *reinterpret_cast<const uint2*>(a1);
            x0[0] = v0.x, x0[1] = v0.y;
            x1[0] = v1.x, x1[1] = v1.y;
          }
#pragma unroll
          for (int h = 0; h < HALVES; ++h) {
            const uint32_t f[4] = {x0[2 * h], x1[2 * h], x0[2 * h + 1], x1[2 * h + 1]};
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_bf16(d[j], f, bv[j][2 * h], bv[j][2 * h + 1]);
          }
        }
      }
    }
    cp_async_wait_but<TILES - 1>();
    __syncwarp();  // (the warp's lanes copied them for one another)
    const uint8_t* c = cs + (i % TILES) * kSumBytes + warp * (kTile * 128) + g * 128;
    const int e0 = ((2 * q) ^ (g & 1)) * 16, e1 = ((2 * q + 1) ^ (g & 1)) * 16;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int tok = rec[1 + g + h * 8];
      if (tok >= 0 && in)
        store8(p, tok, col, *reinterpret_cast<const int4*>(c + h * 1024 + e0),
               *reinterpret_cast<const int4*>(c + h * 1024 + e1), sa[h], sw[0], sw[1], true,
               d[0][2 * h], d[0][2 * h + 1], d[1][2 * h], d[1][2 * h + 1], d[2][2 * h], d[2][2 * h + 1], d[3][2 * h],
               d[3][2 * h + 1]);
    }
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
                       const __grid_constant__ stream::Plan pl, int32_t* c, const int32_t* ids) {
  extern __shared__ uint8_t raw[];
  __shared__ stream::Bars s;
  if (threadIdx.x == 0) {
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
    if (blockIdx.x == 0) {  // (the next kernel's first read)
      prefetch_l2(ids);
      prefetch_l2(ids + m - 1);
    }
  }
  stream::setup(s, pl);
  stream::run(Dense{m, pl, c}, pl, s, stream::ring_of(raw), &tmW, &tmX);
  stream::teardown(s);
}

inline bool streams(int m) { return m <= stream::kMaxTokens; }

// (a ring of 172 KB leaves room for a CTA of s, with its 33 KB for 64 ranks)
constexpr size_t kRing = 172 * 1024;
inline stream::Plan stream_plan(int m, int n, int k, int num_sms) {
  return stream::plan(m, n, k, num_sms, kSlices - 1, kRing);
}

inline int chunks_of(int m) { return (m + kChunk - 1) / kChunk; }

// Groups at most of `tokens` sorted together (those without an adapter make groups
// of their own, for the output): every adapter's last one may be partly filled.
inline int most_groups(int tokens, int adapters, bool none) {
  const int a = adapters + (none ? 1 : 0);
  return (a < tokens ? a : tokens) + tokens / kTile;
}

// K parts of s: as many as keep its CTAs within one an SM, no part under 512.
// `adapters` 1 gives the most parts.
inline int shrink_parts(int m, int k, int adapters, int num_sms) {
  const int ctas = streams(m) ? most_groups(m, adapters, false) : (m + kTile - 1) / kTile;
  int parts = 1;
  while (parts < kMaxParts && 2 * ctas * parts <= num_sms && k / (2 * parts) >= 512) parts *= 2;
  return parts;
}

template <bool BF16, int RT>
inline cudaError_t launch_shrink_rt(const Args& a, dim3 grid, int dev, cudaStream_t stream) {
  if (!a.beside) return launch_pdl(lora_shrink_kernel<BF16, RT, false>, grid, dim3(kShrinkThreads), 0, stream, 1, a);
  const cudaError_t e = stream::shares_sm_once(lora_shrink_kernel<BF16, RT, true>, dev, (BF16 ? 8 : 0) + RT / 4);
  if (e != cudaSuccess) return e;
  return launch_pdl(lora_shrink_kernel<BF16, RT, true>, grid, dim3(kShrinkThreads), 0, stream, 1, a);
}

template <bool BF16>
inline cudaError_t launch_shrink_t(const Args& a, int dev, cudaStream_t stream) {
  const int groups = a.beside ? most_groups(a.m, a.adapters, false) : chunks_of(a.m) * a.most;
  const dim3 grid(groups, 1, a.kparts * ((a.rank + kRankGroup - 1) / kRankGroup));
  if (a.rank <= 16) return launch_shrink_rt<BF16, 2>(a, grid, dev, stream);
  if (a.rank <= 32) return launch_shrink_rt<BF16, 4>(a, grid, dev, stream);
  return launch_shrink_rt<BF16, 8>(a, grid, dev, stream);
}

inline cudaError_t launch_shrink(const Args& a, bool x_bf16, int dev, cudaStream_t stream) {
  return x_bf16 ? launch_shrink_t<true>(a, dev, stream) : launch_shrink_t<false>(a, dev, stream);
}

inline cudaError_t launch_units(const Args& a, cudaStream_t stream) {
  return launch_pdl(lora_units_kernel, dim3(chunks_of(a.m)), dim3(kChunk), 0, stream, 1, a);
}

// Returns 0, 1 when a tensor map could not be made, 2 with *err set.
inline int launch_stream(const Args& a, const int8_t* x, const int8_t* w, const stream::Plan& pl, int dev, int num_sms,
                         cudaStream_t stream, cudaError_t* err) {
  CUtensorMap tw, tx;
  if (!gemm::cached_tmap(&tw, w, a.n, a.k, stream::kRows) || !gemm::cached_tmap(&tx, x, a.m, a.k, pl.nb)) return 1;
  if ((*err = gemm::set_smem_once(lora_stream_kernel, dev, 0, stream::kRingBytes + 1024)) != cudaSuccess) return 2;
  if ((*err = stream::shares_sm_once(lora_stream_kernel, dev, 0)) != cudaSuccess) return 2;
  *err = launch_pdl(lora_stream_kernel, dim3(num_sms), dim3(stream::kThreads), stream::smem_bytes(pl), stream, 1, tw, tx,
                    a.m, pl, const_cast<int32_t*>(a.c), a.ids);
  return *err == cudaSuccess ? 0 : 2;
}

template <int RK>
inline cudaError_t launch_long(const Args& a, dim3 grid, int dev, cudaStream_t stream) {
  constexpr size_t bytes = long_smem<RK>();
  const cudaError_t e = gemm::set_smem_once(lora_expand_long_kernel<RK>, dev, RK / 16, bytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(lora_expand_long_kernel<RK>, grid, dim3(kExpandThreads), bytes, stream, 1, a);
}

inline cudaError_t launch_expand(const Args& a, int dev, int num_sms, cudaStream_t stream) {
  if (a.beside) {
    const dim3 grid(most_groups(a.m, a.adapters, true), (a.n + kExpandCols - 1) / kExpandCols);
    return launch_pdl(lora_expand_kernel, grid, dim3(kExpandThreads), expand_smem(a.rank), stream, 1, a);
  }
  // as many CTAs as are resident at once (two an SM), at least one a column block
  const int most = chunks_of(a.m) * a.most, cols = (a.n + 255) / 256;
  int x = 2 * num_sms / cols;
  x = x < 1 ? 1 : (x > most ? most : x);
  const dim3 grid(x, cols);
  if (a.rank <= 16) return launch_long<16>(a, grid, dev, stream);
  if (a.rank <= 32) return launch_long<32>(a, grid, dev, stream);
  if (a.rank <= 64) return launch_long<64>(a, grid, dev, stream);
  return launch_long<128>(a, grid, dev, stream);
}

}  // namespace lora
}  // namespace qk
