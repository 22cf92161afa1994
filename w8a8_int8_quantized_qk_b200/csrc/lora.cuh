// lora.cuh -- low-rank adapters of many requests beside the shared W8A8
// projection: out = epilogue(a b^T) + s B[id]^T, s = lora_scale[id] * x A[id]^T,
// where token i uses adapter id = ids[i] (none when outside [0, adapters)).
//
// s (rank values per token) is kept in binary32, and so is the sum of the two
// parts: the output is rounded once.
#pragma once

#include "qk_common.cuh"
#include "quant.cuh"

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
  float* s;                   // [m, rank] workspace
  const int32_t* c;           // [m, n] workspace: the int32 sums of the projection
  void* out;
  int out_bf16;
};

__device__ __forceinline__ int adapter_of(const Args& p, int row) {
  const int id = __ldg(p.ids + row);
  return (id >= 0 && id < p.adapters) ? id : -1;
}

// s[i][r]: one warp per (token, rank row).
template <bool BF16>
__global__ void __launch_bounds__(256) lora_shrink_kernel(Args p) {
  constexpr int E = BF16 ? 8 : 4;
  constexpr int ES = BF16 ? 2 : 4;
  griddep_wait();
  griddep_launch_dependents();
  const int row = blockIdx.x, r = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= p.rank) return;
  const int id = adapter_of(p, row);
  if (id < 0) return;
  const char* x = static_cast<const char*>(p.x) + static_cast<int64_t>(row) * p.k * ES;
  const __nv_bfloat16* a = p.la + (static_cast<int64_t>(id) * p.rank + r) * p.k;
  float sum = 0.0f;
  for (int v = lane; v < p.k / E; v += 32) {
    float f[E];
    quant::widen<BF16>(ld_nc_v4(x + static_cast<int64_t>(v) * 16), f);
#pragma unroll
    for (int e = 0; e < E; ++e) sum = fmaf(f[e], __bfloat162float(a[v * E + e]), sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (lane == 0)
    p.s[static_cast<int64_t>(row) * p.rank + r] = p.lscale ? sum * __ldg(p.lscale + id) : sum;
}

// out = ((acc * sa) * sw) * alpha + s B^T: one thread per output.
__global__ void __launch_bounds__(256) lora_expand_kernel(Args p) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t total = static_cast<int64_t>(p.m) * p.n;
  for (int64_t o = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; o < total;
       o += static_cast<int64_t>(gridDim.x) * 256) {
    const int row = static_cast<int>(o / p.n), col = static_cast<int>(o % p.n);
    float v = __int2float_rn(p.c[o]);
    v = __fmul_rn(__fmul_rn(__fmul_rn(v, p.sa[row]), p.sw[col]), p.alpha);
    const int id = adapter_of(p, row);
    if (id >= 0) {
      const __nv_bfloat16* b = p.lb + (static_cast<int64_t>(id) * p.n + col) * p.rank;
      const float* s = p.s + static_cast<int64_t>(row) * p.rank;
      float d = 0.0f;
      for (int r = 0; r < p.rank; ++r) d = fmaf(s[r], __bfloat162float(b[r]), d);
      v = __fadd_rn(v, d);
    }
    if (p.out_bf16)
      static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(v);
    else
      static_cast<float*>(p.out)[o] = v;
  }
}

inline cudaError_t launch_shrink(const Args& a, bool x_bf16, cudaStream_t stream) {
  const dim3 grid(a.m, (a.rank + 7) / 8);
  return x_bf16 ? launch_pdl(lora_shrink_kernel<true>, grid, dim3(256), 0, stream, 1, a)
                : launch_pdl(lora_shrink_kernel<false>, grid, dim3(256), 0, stream, 1, a);
}

inline cudaError_t launch_expand(const Args& a, int num_sms, cudaStream_t stream) {
  const int64_t want = (static_cast<int64_t>(a.m) * a.n + 255) / 256, cap = static_cast<int64_t>(num_sms) * 8;
  return launch_pdl(lora_expand_kernel, dim3(static_cast<unsigned>(want < cap ? want : cap)), dim3(256), 0,
                    stream, 1, a);
}

}  // namespace lora
}  // namespace qk
