// norm.cuh -- residual addition, root-mean-square norm and per-token 8-bit
// quantisation in one pass: the step of a decoder layer that makes the int8
// (or e4m3) tokens and scales its W8A8 products read.
//
// Per row, with r = x + residual rounded to x's type (r = x without one):
//     t = r * w                          (binary32, RN)
//     a = max |t|                        (exact)
//     rstd = 1 / sqrt(mean(r^2) + eps)
//     scale = max(a * rstd, 1e-12) / qmax, bounded by *ub (fp8)
//     q = round(t * inv),  inv = qmax * (1 / a)  (rstd / scale when the scale
//                                                 was clamped or bounded)
//     y = t * rstd                       (optional, rounded to x's type)
// The norm's factor rstd cancels between a value and its row's scale, so the
// codes need only t and a, and the maximum and the sum of squares are reduced
// together: one reduction per row, where norm-then-quantise has two, the
// second waiting for the first.  It also makes the codes independent of the
// order in which the squares are added.
#pragma once

#include "qk_common.cuh"
#include "quant.cuh"

namespace qk {
namespace norm {

struct Args {
  int m, k;
  const void* x;
  int64_t ldx;        // row strides in elements
  const void* res;    // or null
  int64_t ldr;
  void* res_out;      // or null; may be res or x
  int64_t ldo;
  const void* w;      // [k]
  float eps;
  void* y;            // [m, k] or null
  int8_t* q;          // [m, k]
  float* scale;       // [m]
  int fp8;
  const float* ub;    // fp8 only, optional
};

// (plain loads: residual_out may be one of the inputs)
__device__ __forceinline__ uint4 ld_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// E binary32 values -> a 16-byte vector of x's type.
template <bool BF16>
__device__ __forceinline__ uint4 narrow(const float (&f)[BF16 ? 8 : 4]) {
  if constexpr (BF16) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  } else {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
}

// r = x + residual, rounded to the stream's type (what residual_out holds).
template <bool BF16>
__device__ __forceinline__ uint4 add_rows(const uint4& x, const uint4& res) {
  constexpr int E = BF16 ? 8 : 4;
  float a[E], b[E];
  quant::widen<BF16>(x, a);
  quant::widen<BF16>(res, b);
#pragma unroll
  for (int e = 0; e < E; ++e) a[e] = __fadd_rn(a[e], b[e]);
  return narrow<BF16>(a);
}

struct RowFactors {
  float rstd, scale, inv;
};

__device__ __forceinline__ RowFactors row_factors(const Args& p, float amax, float ss) {
  RowFactors f;
  f.rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, static_cast<float>(p.k)), p.eps)));
  const float qmax = p.fp8 ? 448.0f : 127.0f;
  const float z = __fmul_rn(amax, f.rstd);
  const float whole = __fdiv_rn(fmaxf(z, 1e-12f), qmax);
  f.scale = p.ub != nullptr ? fminf(whole, __ldg(p.ub)) : whole;
  f.inv = (z >= 1e-12f && f.scale == whole) ? __fmul_rn(qmax, __fdiv_rn(1.0f, amax))
                                                : __fdiv_rn(f.rstd, f.scale);
  return f;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// One row per CTA, read twice (the second time from cache): any row length.
constexpr int kTwoPassThreads = 512;

template <bool BF16>
__global__ void __launch_bounds__(kTwoPassThreads) norm_quant_twopass_kernel(Args p) {
  constexpr int E = BF16 ? 8 : 4;
  constexpr int ES = BF16 ? 2 : 4;
  constexpr int NW = kTwoPassThreads / 32;
  __shared__ float red_a[NW], red_s[NW];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nvec = p.k / E;
  griddep_wait();  // the previous kernel in the stream is done with our buffers
  griddep_launch_dependents();
  const char* xr = static_cast<const char*>(p.x) + row * p.ldx * ES;
  const char* rr = p.res ? static_cast<const char*>(p.res) + row * p.ldr * ES : nullptr;
  char* ro = p.res_out ? static_cast<char*>(p.res_out) + row * p.ldo * ES : nullptr;
  const char* w = static_cast<const char*>(p.w);
  float a = 0.0f, ss = 0.0f;
  for (int v = tid; v < nvec; v += kTwoPassThreads) {
    const int64_t o = static_cast<int64_t>(v) * 16;
    uint4 r = ld_v4(xr + o);
    if (rr) r = add_rows<BF16>(r, ld_v4(rr + o));
    if (ro) *reinterpret_cast<uint4*>(ro + o) = r;
    float f[E], g[E];
    quant::widen<BF16>(r, f);
    quant::widen<BF16>(ld_nc_v4(w + o), g);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      ss = __fmaf_rn(f[e], f[e], ss);
      a = fmaxf(a, fabsf(__fmul_rn(f[e], g[e])));
    }
  }
  a = quant::warp_max(a);
  ss = warp_sum(ss);
  if (lane == 0) {
    red_a[warp] = a;
    red_s[warp] = ss;
  }
  __syncthreads();
  a = quant::warp_max(lane < NW ? red_a[lane] : 0.0f);
  ss = warp_sum(lane < NW ? red_s[lane] : 0.0f);
  const RowFactors fac = row_factors(p, a, ss);
  quant::Args qa = {};
  qa.fp8 = p.fp8;
  int8_t* qr = p.q + row * p.k;
  char* yr = p.y ? static_cast<char*>(p.y) + row * p.k * ES : nullptr;
  for (int v = tid; v < nvec; v += kTwoPassThreads) {
    const int64_t o = static_cast<int64_t>(v) * 16;
    uint4 r;
    if (ro) {
      r = ld_v4(ro + o);  // what this thread stored above (x or res may be gone)
    } else {
      r = ld_v4(xr + o);
      if (rr) r = add_rows<BF16>(r, ld_v4(rr + o));
    }
    float f[E], g[E];
    quant::widen<BF16>(r, f);
    quant::widen<BF16>(ld_nc_v4(w + o), g);
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = __fmul_rn(f[e], g[e]);
    quant::store_q<E>(qa, qr + static_cast<int64_t>(v) * E, f, fac.inv);
    if (yr) {
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = __fmul_rn(f[e], fac.rstd);
      *reinterpret_cast<uint4*>(yr + o) = narrow<BF16>(f);
    }
  }
  if (tid == 0) p.scale[row] = fac.scale;
}

inline cudaError_t launch(const Args& a, bool bf16, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  return bf16 ? launch_pdl(norm_quant_twopass_kernel<true>, dim3(a.m), dim3(kTwoPassThreads), 0, stream, 1, a)
              : launch_pdl(norm_quant_twopass_kernel<false>, dim3(a.m), dim3(kTwoPassThreads), 0, stream, 1, a);
}

}  // namespace norm
}  // namespace qk
