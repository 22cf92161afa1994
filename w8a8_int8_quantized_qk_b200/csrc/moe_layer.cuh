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
#pragma once

#include "gemv.cuh"
#include "qk_common.cuh"
#include "quant.cuh"

namespace qk {
namespace moe {

struct Args {
  int m, hidden, inter, experts, topk;
  const int8_t* a;      // [m, hidden]
  const float* sa;      // [m]
  const int32_t* ids;   // [m, topk]
  const float* wt;      // [m, topk]
  const int8_t* w13;    // [experts, 2 inter, hidden]
  const float* s13;     // [experts, 2 inter]
  const int8_t* w2;     // [experts, hidden, inter]
  const float* s2;      // [experts, hidden]
  float* h;             // [pairs, inter] workspace
  int8_t* q;            // [pairs, inter] workspace
  float* sh;            // [pairs] workspace
  float* y;             // [pairs, hidden] workspace
  void* out;            // [m, hidden]
  int out_bf16;
};

__device__ __forceinline__ int expert_of(const Args& p, int pair) {
  const int e = __ldg(p.ids + pair);
  return (e >= 0 && e < p.experts) ? e : -1;
}

__device__ __forceinline__ int warp_dot(const int8_t* w, const int8_t* a, int k) {
  int acc = 0;
  for (int v = threadIdx.x & 31; v < k / 16; v += 32)
    acc = gemv::dot16(ld_stream_v4(w + v * 16), ld_nc_v4(a + v * 16), acc);
  return __reduce_add_sync(0xFFFFFFFFu, acc);
}

// h[pair][j]: one warp per gate / up row pair.
__global__ void __launch_bounds__(256) moe_gate_up_kernel(Args p) {
  griddep_wait();
  griddep_launch_dependents();
  const int pair = blockIdx.y, j = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (j >= p.inter) return;
  const int e = expert_of(p, pair), token = pair / p.topk;
  float* h = p.h + static_cast<int64_t>(pair) * p.inter + j;
  if (e < 0) {
    if (lane == 0) *h = 0.0f;
    return;
  }
  const int64_t row = static_cast<int64_t>(e) * 2 * p.inter + j;
  const int8_t* a = p.a + static_cast<int64_t>(token) * p.hidden;
  const int g = warp_dot(p.w13 + row * p.hidden, a, p.hidden);
  const int u = warp_dot(p.w13 + (row + p.inter) * p.hidden, a, p.hidden);
  if (lane == 0) {
    const float sa = p.sa[token];
    *h = quant::silu_mul(__fmul_rn(__fmul_rn(__int2float_rn(g), sa), p.s13[row]),
                         __fmul_rn(__fmul_rn(__int2float_rn(u), sa), p.s13[row + p.inter]));
  }
}

// out[i][j]: one warp per output, the slots in order.
__global__ void __launch_bounds__(256) moe_down_kernel(Args p) {
  griddep_wait();
  griddep_launch_dependents();
  const int i = blockIdx.y, j = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (j >= p.hidden) return;
  float f = 0.0f;
  for (int s = 0; s < p.topk; ++s) {
    const int pair = i * p.topk + s, e = expert_of(p, pair);
    if (e < 0) continue;
    const int64_t row = static_cast<int64_t>(e) * p.hidden + j;
    const int acc = warp_dot(p.w2 + row * p.inter, p.q + static_cast<int64_t>(pair) * p.inter, p.inter);
    const float y = __fmul_rn(__fmul_rn(__int2float_rn(acc), p.sh[pair]), p.s2[row]);
    f = __fmaf_rn(p.wt[pair], y, f);
  }
  if (lane == 0) {
    const int64_t o = static_cast<int64_t>(i) * p.hidden + j;
    if (p.out_bf16)
      static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(f);
    else
      static_cast<float*>(p.out)[o] = f;
  }
}

inline cudaError_t launch(const Args& a, int num_sms, cudaStream_t stream) {
  const int pairs = a.m * a.topk;
  cudaError_t e = launch_pdl(moe_gate_up_kernel, dim3((a.inter + 7) / 8, pairs), dim3(256), 0, stream, 1, a);
  if (e != cudaSuccess) return e;
  quant::Args q = {};
  q.m = pairs;
  q.k = a.inter;
  q.x = a.h;
  q.ld = a.inter;
  q.q = a.q;
  q.scale = a.sh;
  e = quant::launch<false>(q, false, num_sms, stream);
  if (e != cudaSuccess) return e;
  return launch_pdl(moe_down_kernel, dim3((a.hidden + 7) / 8, a.m), dim3(256), 0, stream, 1, a);
}

}  // namespace moe
}  // namespace qk
