// stream.cuh -- int8 weights streamed past at most 64 int8 tokens on the
// tensor core: the core of the MoE layer for a few tokens and of the
// projection with adapters for small batches.
//
// The products are bound by reading the weights once, so the weight rows take
// the M side of the MMA (128 rows) and the tokens its N side (16 .. 64), and
// 128-row tiles of 128 K bytes flow through a ring that holds about 200 KB on
// every SM: the loads need no registers and no thread waits for them.  The
// warp matrix instruction (mma.m16n8k32, fed from registers) was built first;
// it takes 32 cycles a warp for 512 weight bytes on this part, which is 47 %
// of the pipe at full HBM rate for 8 tokens and the bound beyond 16: 32 tokens,
// two each of 8 experts of 4096 x 14336, took 310 us with it, 236 us here.
//
// Every CTA takes the same number of 128 x 128-byte blocks, in the order of
// the tiles (128 rows by all of K), so no SM idles in a last round: a tile that
// two CTAs share leaves as two partial sums.  The sums are int32, one slice for
// each part a tile is cut into; what reads them adds the slices, exactly.
#pragma once

#include "gemm_sm100.cuh"
#include "qk_common.cuh"

namespace qk {
namespace stream {

constexpr int kThreads = 192;      // producer warp, MMA warp, 4 epilogue warps
constexpr int kRows = 128;         // weight rows of a unit
constexpr int kK = 128;            // K bytes of a stage
constexpr int kMaxStages = 12;
constexpr int kMaxTokens = 64;     // N side of one unit
constexpr int kTmemCols = 128;     // two accumulators of 64 columns
constexpr size_t kRingBytes = 212 * 1024;

struct Plan {
  int nb;          // tokens of a tile: 16, 32, 48 or 64
  int stages;
  int num_kb;      // K blocks of a tile
  int row_blocks;
  int n;           // weight rows (per expert)
  int cut;         // a CTA takes at least 1 / cut of a tile
  int max_slices;  // parts a tile is then cut into, at most
};

__host__ __device__ inline int stage_bytes(int nb) { return kRows * kK + nb * kK; }

// Blocks a CTA takes of `tiles` tiles: an equal share, but no fewer than four
// (64 KB), and no less than 1 / cut of a tile (its sums are read slice by slice).
__host__ __device__ inline int share(int tiles, int num_kb, int cut, int grid) {
  const int64_t all = static_cast<int64_t>(tiles) * num_kb;
  int per = static_cast<int>((all + grid - 1) / grid);
  if (per < 4) per = 4;
  const int least = (num_kb + cut - 1) / cut;
  return per < least ? least : per;
}

// Slices of a tile, and the slice of the part that CTA `bid` holds of it.  (The
// host has checked that all blocks together are fewer than 2^32.)
__device__ __forceinline__ int slices_of(int tile, int num_kb, int per) {
  const uint32_t f = static_cast<uint32_t>(tile) * num_kb, d = static_cast<uint32_t>(per);
  return static_cast<int>((f + num_kb - 1) / d - f / d) + 1;
}
__device__ __forceinline__ int slice_of(int tile, int num_kb, int per, int bid) {
  return bid - static_cast<int>(static_cast<uint32_t>(tile) * num_kb / static_cast<uint32_t>(per));
}

// `tokens`: N side wanted of sets of n rows (experts) by k; `cut` as above;
// `ring`: bytes of the ring.  The grid is one CTA an SM; the fewest blocks a CTA can get, those of one
// set, bound the slices.
inline Plan plan(int tokens, int n, int k, int num_sms, int cut, size_t ring) {
  Plan p;
  p.nb = tokens >= kMaxTokens ? kMaxTokens : (tokens + 15) / 16 * 16;
  const int fit = static_cast<int>(ring / stage_bytes(p.nb));
  p.stages = fit < kMaxStages ? fit : kMaxStages;
  p.num_kb = (k + kK - 1) / kK;
  p.row_blocks = (n + kRows - 1) / kRows;
  p.n = n;
  p.cut = cut;
  const int per = share(p.row_blocks, p.num_kb, cut, num_sms);
  // a part starts at the tile's start or at a multiple of `per` inside it
  p.max_slices = (p.num_kb - 1) / per + 2;
  return p;
}

inline size_t smem_bytes(const Plan& p) {
  return 1024 + static_cast<size_t>(p.stages) * stage_bytes(p.nb);
}

struct Bars {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

// A tile in the two tensor maps.
struct Tile {
  int w_row, x_row;
};

__device__ __forceinline__ uint32_t tmem_ld_x1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr) : "memory");
  return r;
}

// The blocks [f, end) of a CTA, tile by tile.
struct Range {
  uint32_t f, end;
  __device__ __forceinline__ Range(int tiles, int num_kb, int per) {
    const uint64_t all = static_cast<uint64_t>(tiles) * num_kb, at = static_cast<uint64_t>(blockIdx.x) * per;
    f = static_cast<uint32_t>(at < all ? at : all);
    end = static_cast<uint32_t>(at + per < all ? at + per : all);
  }
  // the part of the next tile: K blocks [kb0, kb1)
  __device__ __forceinline__ bool next(int num_kb, int& tile, int& kb0, int& kb1) {
    if (f >= end) return false;
    tile = static_cast<int>(f / static_cast<uint32_t>(num_kb));
    kb0 = static_cast<int>(f - static_cast<uint32_t>(tile) * num_kb);
    const int left = static_cast<int>(end - f);
    kb1 = left < num_kb - kb0 ? kb0 + left : num_kb;
    f += kb1 - kb0;
    return true;
  }
};

// The roles.  P has:
//   static constexpr bool kEarlyWeights   the first weights are requested before
//                                     the wait for the previous kernel (which must
//                                     not write them)
//   int tiles()
//   Walk start(); Tile tile(Walk&, int t)   tile t (a Walk goes upward only)
//   void store(Walk, int t, int slice, Tile, uint32_t tmem, int row)   a part's
//                                     sums: row `row` of the tile, tokens in TMEM
//                                     columns
template <class P>
__device__ __forceinline__ void run(const P& prob, const Plan& pl, Bars& s, uint8_t* ring, const CUtensorMap* tmW,
                                    const CUtensorMap* tmX) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = pl.stages, sb = stage_bytes(pl.nb), num_kb = pl.num_kb;
  const int tiles = prob.tiles(), per = share(tiles, num_kb, pl.cut, static_cast<int>(gridDim.x));
  const uint32_t ring0 = smem_addr(ring);
  Range parts(tiles, num_kb, per);
  typename P::Walk w = prob.start();
  int t, kb0, kb1;
  if (warp == 0) {
    if (lane == 0) {
      int stage = 0, pre = 0;
      uint32_t phase = 0, issued = 0;
      bool ok = true;
      if constexpr (P::kEarlyWeights) {
        Range early = parts;
        typename P::Walk we = prob.start();
        while (pre < stages && early.next(num_kb, t, kb0, kb1)) {
          const Tile u = prob.tile(we, t);
          for (int kb = kb0; kb < kb1 && pre < stages; ++kb, ++pre) {
            const uint32_t fb = smem_addr(&s.full[pre]);
            mbar_arrive_expect_tx(fb, static_cast<uint32_t>(sb));
            tma_load_2d(ring0 + pre * sb, tmW, fb, kb * kK, u.w_row);
          }
        }
        griddep_wait();
      }
      while (ok && parts.next(num_kb, t, kb0, kb1)) {
        const Tile u = prob.tile(w, t);
        for (int kb = kb0; kb < kb1; ++kb) {
          const uint32_t fb = smem_addr(&s.full[stage]);
          if (pre > 0) {
            --pre;  // this stage's weights are on their way
          } else {
            if (!mbar_wait(smem_addr(&s.empty[stage]), phase ^ 1u, &s.abort)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(fb, static_cast<uint32_t>(sb));
            tma_load_2d(ring0 + stage * sb, tmW, fb, kb * kK, u.w_row);
          }
          tma_load_2d(ring0 + stage * sb + kRows * kK, tmX, fb, kb * kK, u.x_row);
          ++issued;
          if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // No copy may still be landing in shared memory when the CTA exits: wait
      // (bounded, ignoring the abort flag) for the last copies issued.
      const uint32_t n = static_cast<uint32_t>(stages);
      for (uint32_t i = issued > n ? issued - n : 0u; i < issued; ++i)
        mbar_wait(smem_addr(&s.full[i % n]), (i / n) & 1u, nullptr);
    }
    __syncwarp();
    if constexpr (P::kEarlyWeights) griddep_launch_dependents();
  } else if (warp == 1) {
    if constexpr (P::kEarlyWeights) {
      griddep_wait();
      griddep_launch_dependents();
    }
    if (lane == 0) {
      const uint32_t idesc = idesc_i8(kRows, pl.nb);
      int stage = 0;
      uint32_t phase = 0, abuf = 0, aphase = 0;
      bool ok = true;
      while (ok && parts.next(num_kb, t, kb0, kb1)) {
        if (!mbar_wait(smem_addr(&s.acc_empty[abuf]), aphase ^ 1u, &s.abort)) break;
        tc_fence_after();
        const uint32_t d = s.tmem_base + abuf * kMaxTokens;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(smem_addr(&s.full[stage]), phase, &s.abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = ring0 + stage * sb, b0 = a0 + kRows * kK;
#pragma unroll
          for (int kk = 0; kk < kK / gemm::UMMA_K; ++kk)
            mma_i8(d, sdesc_k_sw128(a0 + kk * gemm::UMMA_K), sdesc_k_sw128(b0 + kk * gemm::UMMA_K), idesc,
                   kb > kb0 || kk > 0);
          mma_commit(smem_addr(&s.empty[stage]));
          if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) {
          mma_commit(smem_addr(&s.acc_full[abuf]));
          abuf ^= 1u;
          if (abuf == 0) aphase ^= 1u;
        }
      }
      // Every MMA issued must be complete before the TMEM can be released.
      mma_commit(smem_addr(&s.drain));
      mbar_wait(smem_addr(&s.drain), 0u, nullptr);
    }
    __syncwarp();
  } else {
    if constexpr (P::kEarlyWeights) {
      griddep_wait();
      griddep_launch_dependents();
    }
    const int quad = warp & 3;
    uint32_t abuf = 0, aphase = 0;
    while (parts.next(num_kb, t, kb0, kb1)) {
      const Tile u = prob.tile(w, t);
      if (!gemm::warp_wait(smem_addr(&s.acc_full[abuf]), aphase, &s.abort)) break;
      tc_fence_after();
      prob.store(w, t, slice_of(t, num_kb, per, static_cast<int>(blockIdx.x)), u,
                 s.tmem_base + abuf * kMaxTokens + (static_cast<uint32_t>(quad * 32) << 16), quad * 32 + lane);
      tc_fence_before();
      if (lane == 0) mbar_arrive(smem_addr(&s.acc_empty[abuf]));
      abuf ^= 1u;
      if (abuf == 0) aphase ^= 1u;
    }
  }
}

__device__ __forceinline__ void setup(Bars& s, const Plan& pl) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < pl.stages; ++i) {
      mbar_init(smem_addr(&s.full[i]), 1);
      mbar_init(smem_addr(&s.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&s.acc_full[i]), 1);
      mbar_init(smem_addr(&s.acc_empty[i]), 4);
    }
    mbar_init(smem_addr(&s.drain), 1);
    s.abort = 0;
    fence_mbar_init();
  }
  if ((threadIdx.x >> 5) == 1) {
    tmem_alloc(smem_addr(&s.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
}

__device__ __forceinline__ void teardown(Bars& s) {
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if ((threadIdx.x >> 5) == 1) tmem_dealloc(s.tmem_base, kTmemCols);
}

// An SM's split between L1 and shared memory does not change while a CTA runs on
// it, so the small kernels around a stream share SMs with it only when they ask
// for its split.  (Once per device and kernel; `slot` tells kernels of one
// signature apart.)
template <class K>
inline cudaError_t shares_sm_once(K kernel, int dev, int slot) {
  static std::atomic<unsigned long long> done[16] = {};
  const unsigned long long bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0ull;
  if (bit && (done[slot].load(std::memory_order_acquire) & bit)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                             cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess && bit) done[slot].fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

__device__ __forceinline__ uint8_t* ring_of(uint8_t* raw) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
}

// Sums of columns [0, count) of one row of a unit: out(token, value).
template <class F>
__device__ __forceinline__ void each_column(uint32_t tmem, int count, F&& out) {
  for (int c0 = 0; c0 < count; c0 += 16) {
    uint32_t v[16];
    __syncwarp();
    tmem_ld_32x32b_x16(tmem + c0, v);
    tmem_ld_wait();
#pragma unroll
    for (int c = 0; c < 16; ++c)
      if (c0 + c < count) out(c0 + c, static_cast<int>(v[c]));
  }
}

}  // namespace stream
}  // namespace qk
