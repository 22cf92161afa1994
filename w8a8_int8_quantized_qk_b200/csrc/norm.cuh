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
//
// Bound by reading x and the residual and writing their sum and the codes, once.
// As in the plain quantiser, a row is held in registers between the two passes
// (as 16-byte vectors of the stream's type, which r is exact in), many rows are
// walked by persistent CTAs that load a row ahead, and a row is split over a
// cluster when rows are few.  4096 x 4096 bf16 with residual (117 MB): 29.2 us with
// the row read twice, 21.0 us here (5.6 TB/s, 0.86 of the copy rate), 16.0 us into
// outputs that are still in L2.
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
    return vec4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  } else {
    return vec4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
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

// t = r * w of a vector, and its share of the row's maximum and sum of squares.
template <bool BF16>
__device__ __forceinline__ void weigh(const uint4& r, const uint4& w, float (&t)[BF16 ? 8 : 4], float& a, float& ss) {
  constexpr int E = BF16 ? 8 : 4;
  float f[E], g[E];
  quant::widen<BF16>(r, f);
  quant::widen<BF16>(w, g);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    ss = __fmaf_rn(f[e], f[e], ss);
    t[e] = __fmul_rn(f[e], g[e]);
    a = fmaxf(a, fabsf(t[e]));
  }
}

// Codes (and the normalised values) of a vector.
template <bool BF16>
__device__ __forceinline__ void emit(const Args& p, const RowFactors& fac, const uint4& r, const uint4& w, int8_t* q,
                                     char* y) {
  constexpr int E = BF16 ? 8 : 4;
  float t[E], a = 0.0f, ss = 0.0f;
  weigh<BF16>(r, w, t, a, ss);
  quant::Args qa = {};
  qa.fp8 = p.fp8;
  quant::store_q<E>(qa, q, t, fac.inv);
  if (y) {
#pragma unroll
    for (int e = 0; e < E; ++e) t[e] = __fmul_rn(t[e], fac.rstd);
    *reinterpret_cast<uint4*>(y) = narrow<BF16>(t);
  }
}

// Maximum and sum over the CTA (and the cluster when CLUSTER), to every thread.
template <bool CLUSTER>
__device__ __forceinline__ void row_reduce(float& a, float& ss, float2* red /*[33]*/) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = (blockDim.x + 31) >> 5;
  a = quant::warp_max(a);
  ss = warp_sum(ss);
  if (lane == 0) red[warp] = make_float2(a, ss);
  __syncthreads();
  const float2 v = lane < nwarps ? red[lane] : make_float2(0.0f, 0.0f);
  a = quant::warp_max(v.x);
  ss = warp_sum(v.y);
  if constexpr (CLUSTER) {
    namespace cg = cooperative_groups;
    cg::cluster_group cl = cg::this_cluster();
    if (threadIdx.x == 0) red[32] = make_float2(a, ss);
    cl.sync();
    a = 0.0f;
    ss = 0.0f;
    const unsigned n = cl.num_blocks();
    for (unsigned r = 0; r < n; ++r) {
      const float2 o = *cl.map_shared_rank(&red[32], r);
      a = fmaxf(a, o.x);
      ss = __fadd_rn(ss, o.y);
    }
  }
}

// Few rows: one row per CTA, or per cluster; a thread holds up to kRowVec vectors.
constexpr int kRowVec = 4;

template <bool BF16, bool CLUSTER>
__global__ void __launch_bounds__(quant::kMaxThreads) norm_quant_rows_kernel(Args p) {
  constexpr int E = BF16 ? 8 : 4;
  constexpr int ES = BF16 ? 2 : 4;
  __shared__ float2 red[33];
  int ranks = 1, rank = 0;
  int64_t row = blockIdx.x;
  if constexpr (CLUSTER) {
    namespace cg = cooperative_groups;
    ranks = static_cast<int>(cg::this_cluster().num_blocks());
    rank = static_cast<int>(cg::this_cluster().block_rank());
    row = blockIdx.x / ranks;
  }
  const int nvec = p.k / E, stride = ranks * blockDim.x, t0 = rank * blockDim.x + threadIdx.x;
  griddep_wait();  // the previous kernel in the stream is done with our buffers
  griddep_launch_dependents();
  const char* xr = static_cast<const char*>(p.x) + row * p.ldx * ES;
  const char* rr = p.res ? static_cast<const char*>(p.res) + row * p.ldr * ES : nullptr;
  char* ro = p.res_out ? static_cast<char*>(p.res_out) + row * p.ldo * ES : nullptr;
  uint4 r[kRowVec], w[kRowVec];
#pragma unroll
  for (int j = 0; j < kRowVec; ++j) {
    const int v = t0 + j * stride;
    const int64_t o = static_cast<int64_t>(v) * 16;
    const uint4 zero = vec4(0, 0, 0, 0);
    r[j] = v < nvec ? ld_v4(xr + o) : zero;
    w[j] = v < nvec ? ld_nc_v4(static_cast<const char*>(p.w) + o) : zero;
  }
  if (rr) {
    uint4 d[kRowVec];
#pragma unroll
    for (int j = 0; j < kRowVec; ++j) {
      const int v = t0 + j * stride;
      d[j] = v < nvec ? ld_v4(rr + static_cast<int64_t>(v) * 16) : vec4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < kRowVec; ++j) r[j] = add_rows<BF16>(r[j], d[j]);
  }
  float a = 0.0f, ss = 0.0f;
#pragma unroll
  for (int j = 0; j < kRowVec; ++j) {
    const int v = t0 + j * stride;
    float t[E];
    if (ro && v < nvec) *reinterpret_cast<uint4*>(ro + static_cast<int64_t>(v) * 16) = r[j];
    weigh<BF16>(r[j], w[j], t, a, ss);
  }
  row_reduce<CLUSTER>(a, ss, red);
  const RowFactors fac = row_factors(p, a, ss);
  int8_t* qr = p.q + row * p.k;
  char* yr = p.y ? static_cast<char*>(p.y) + row * p.k * ES : nullptr;
#pragma unroll
  for (int j = 0; j < kRowVec; ++j) {
    const int v = t0 + j * stride;
    if (v < nvec)
      emit<BF16>(p, fac, r[j], w[j], qr + static_cast<int64_t>(v) * E, yr ? yr + static_cast<int64_t>(v) * 16 : nullptr);
  }
  if (t0 == 0) p.scale[row] = fac.scale;
  if constexpr (CLUSTER) quant::cluster_arrive_wait_relaxed();  // peers may still read red[32]
}

// Many rows: persistent CTAs of T threads with V vectors each, the next row's
// loads in flight.  The warps' sums alternate between two buffers, so a row costs
// one barrier.  Short rows get few threads with up to 4 vectors each, so that many
// rows are in flight on an SM and their reductions and barriers stay small (8192 x
// 512 bf16 with residual: 17.7 us with 256 threads a row, 6.8 with 32; 8192 x 1024:
// 18.3 and 11.8).  With 256 threads at most a thread's share of the weight stays in
// registers; longer rows (T = 512) read it again from cache, and skip the last of 3
// or 5 vectors where they end before it (1500 x 10240: 26.2 us with 5 vectors and no
// skip, 22.8 with 3; 2049 x 8208 fp32 without residual: 18.5 and 17.8).
template <bool BF16, bool RES, int V, int T>
__global__ void __launch_bounds__(T) norm_quant_persistent_kernel(Args p) {
  constexpr int E = BF16 ? 8 : 4;
  constexpr int ES = BF16 ? 2 : 4;
  constexpr int NW = T / 32;
  constexpr bool KEEP = T < 512;
  // the last vectors are skipped where the row has none there (not with so many
  // registers in use that the branch costs more: 1000 x 18000 with residual 25.3 us, 26.5)
  constexpr bool SHORT = !KEEP && (V == 3 || (V == 5 && !RES));
  __shared__ float2 red[2][NW];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nvec = p.k / E;
  griddep_wait();  // the previous kernel in the stream is done with our buffers
  griddep_launch_dependents();
  uint4 xc[V], dc[RES ? V : 1], w[KEEP ? V : 1];
  auto fetch = [&](uint4 (&x)[V], uint4 (&d)[RES ? V : 1], int64_t row) {
    const char* xr = static_cast<const char*>(p.x) + row * p.ldx * ES;
    const char* rr = RES ? static_cast<const char*>(p.res) + row * p.ldr * ES : nullptr;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = tid + j * T;
      const bool in = row < p.m && v < nvec;
      x[j] = in ? ld_v4(xr + static_cast<int64_t>(v) * 16) : vec4(0, 0, 0, 0);
      if constexpr (RES) d[j] = in ? ld_v4(rr + static_cast<int64_t>(v) * 16) : vec4(0, 0, 0, 0);
    }
  };
  auto weight = [&](int j) {
    const int v = tid + j * T;
    return v < nvec ? __ldg(static_cast<const uint4*>(p.w) + v) : vec4(0, 0, 0, 0);
  };
  fetch(xc, dc, blockIdx.x);
  if constexpr (KEEP) {
#pragma unroll
    for (int j = 0; j < V; ++j) w[j] = weight(j);
  }
  int par = 0;
  for (int64_t row = blockIdx.x; row < p.m; row += gridDim.x) {
    uint4 xn[V], dn[RES ? V : 1];
    fetch(xn, dn, row + gridDim.x);
    float a = 0.0f, ss = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = tid + j * T;
      if (SHORT && j + 1 == V && v >= nvec) break;
      float t[E], sj = 0.0f;  // (a vector's squares on their own: a short chain)
      if constexpr (RES) {
        xc[j] = add_rows<BF16>(xc[j], dc[j]);
        if (p.res_out != nullptr && v < nvec)
          *reinterpret_cast<uint4*>(static_cast<char*>(p.res_out) + row * p.ldo * ES + static_cast<int64_t>(v) * 16) =
              xc[j];
      }
      weigh<BF16>(xc[j], KEEP ? w[KEEP ? j : 0] : weight(j), t, a, sj);
      ss = __fadd_rn(ss, sj);
    }
    a = quant::warp_max(a);
    ss = warp_sum(ss);
    if (lane == 0) red[par][warp] = make_float2(a, ss);
    __syncthreads();
    const float2 o = red[par][lane & (NW - 1)];
    a = o.x;
    ss = o.y;
#pragma unroll
    for (int s = NW / 2; s > 0; s >>= 1) {
      a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, s));
      ss = __fadd_rn(ss, __shfl_xor_sync(0xFFFFFFFFu, ss, s));
    }
    const RowFactors fac = row_factors(p, a, ss);
    int8_t* qr = p.q + row * p.k;
    char* yr = p.y ? static_cast<char*>(p.y) + row * p.k * ES : nullptr;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int v = tid + j * T;
      if (v < nvec)
        emit<BF16>(p, fac, xc[j], KEEP ? w[KEEP ? j : 0] : weight(j), qr + static_cast<int64_t>(v) * E,
                   yr ? yr + static_cast<int64_t>(v) * 16 : nullptr);
    }
    if (tid == 0) p.scale[row] = fac.scale;
    par ^= 1;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      xc[j] = xn[j];
      if constexpr (RES) dc[j] = dn[j];
    }
  }
}

// Rows too long for a cluster's registers: one row per CTA, read twice (the second
// time from cache).
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

// Persistent grid: the CTAs that can be resident at once (queried once per kernel;
// every device this library runs on has the same answer).
template <bool BF16, bool RES, int V, int T>
inline cudaError_t launch_persistent(const Args& a, int num_sms, cudaStream_t stream) {
  static std::atomic<int> cached{0};
  int per = cached.load(std::memory_order_relaxed);
  if (per == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, norm_quant_persistent_kernel<BF16, RES, V, T>, T, 0) !=
            cudaSuccess ||
        per < 1) {
      cudaGetLastError();
      per = 1;
    }
    constexpr int most = T < 128 ? 1024 / T : 8;
    per = per < most ? per : most;
    cached.store(per, std::memory_order_relaxed);
  }
  const int cap = per * num_sms, grid = a.m < cap ? a.m : cap;
  return launch_pdl(norm_quant_persistent_kernel<BF16, RES, V, T>, dim3(grid), dim3(T), 0, stream, 1, a);
}

template <bool BF16, bool RES>
inline cudaError_t launch_many(const Args& a, int nvec, int num_sms, cudaStream_t stream) {
  if (nvec <= 32) return launch_persistent<BF16, RES, 1, 32>(a, num_sms, stream);
  if (nvec <= 64) return launch_persistent<BF16, RES, 2, 32>(a, num_sms, stream);
  if (nvec <= 128) return launch_persistent<BF16, RES, 4, 32>(a, num_sms, stream);
  if (nvec <= 256) return launch_persistent<BF16, RES, 4, 64>(a, num_sms, stream);
  if (nvec <= 512) return launch_persistent<BF16, RES, 4, 128>(a, num_sms, stream);
  if (nvec <= 1024) return launch_persistent<BF16, RES, 4, 256>(a, num_sms, stream);
  if (nvec <= 3 * 512) return launch_persistent<BF16, RES, 3, 512>(a, num_sms, stream);
  if (nvec <= 5 * 512) return launch_persistent<BF16, RES, 5, 512>(a, num_sms, stream);
  return launch_persistent<BF16, RES, 8, 512>(a, num_sms, stream);
}

// From two rows an SM on, rows of up to 64 KB: persistent.  Else a CTA per row, of
// as many threads as there are vectors (one row's latency is what counts then: a
// row of 4096 bf16 alone takes 2.4 us so, 3.4 us as a cluster of two CTAs), a
// cluster only where a CTA's registers do not hold the row, and two reads beyond a
// cluster's.
template <bool BF16>
inline cudaError_t launch_typed(const Args& a, int num_sms, cudaStream_t stream) {
  constexpr int most = quant::kMaxThreads;
  const int nvec = a.k / (BF16 ? 8 : 4);
  if (a.m >= 2 * num_sms && nvec <= 8 * 512)
    return a.res != nullptr ? launch_many<BF16, true>(a, nvec, num_sms, stream)
                            : launch_many<BF16, false>(a, nvec, num_sms, stream);
  int cl = 1;
  while (cl < 8 && nvec > cl * most * kRowVec) cl *= 2;
  if (nvec > cl * most * kRowVec)
    return launch_pdl(norm_quant_twopass_kernel<BF16>, dim3(a.m), dim3(kTwoPassThreads), 0, stream, 1, a);
  const int want = ((nvec + cl - 1) / cl + 31) / 32 * 32, threads = want < most ? want : most;
  if (cl == 1) return launch_pdl(norm_quant_rows_kernel<BF16, false>, dim3(a.m), dim3(threads), 0, stream, 1, a);
  return launch_pdl(norm_quant_rows_kernel<BF16, true>, dim3(static_cast<unsigned>(a.m) * cl), dim3(threads), 0, stream,
                    static_cast<unsigned>(cl), a);
}

inline cudaError_t launch(const Args& a, bool bf16, int num_sms, cudaStream_t stream) {
  return bf16 ? launch_typed<true>(a, num_sms, stream) : launch_typed<false>(a, num_sms, stream);
}

}  // namespace norm
}  // namespace qk
