// RMS norm with the residual's addition, an e4m3 output with scales, and the
// backward.
//
// With h = dtype(x + residual), the value the residual stream holds:
//   rstd = 1 / sqrt(mean_j h_j^2 + eps),  y_j = h_j rstd gamma_j,
//   s_g = max_{j in group g} |y_j| / 448,  q_j = e4m3(y_j / s_g).
// Sums and statistics are fp32; h is rounded before the statistics so that
// the backward, which reads the stored h, differentiates the same function;
// y is rounded once, and q is taken from the unrounded y.
// Backward, with xhat = h rstd and g = dy gamma:
//   dx = rstd (g - xhat mean_j(g_j xhat_j)) + dh,  dgamma = sum_rows dy xhat.
#include <cuda_fp8.h>

#include "launch.cuh"

namespace moe {
namespace {

constexpr float kE4m3Max = 448.0f;
// Smallest amax a scale is made of: 448 / amax stays finite.
constexpr float kAmaxFloor = 7.70372e-34f;   // 2^-110

__device__ __forceinline__ float block_max(float v, float *smem32) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (lane == 0) smem32[warp] = v;
  __syncthreads();
  const int nw = blockDim.x >> 5;
  float r = lane < nw ? smem32[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, o));
  return r;
}

// Scale of a group and the factor y is multiplied with.
__device__ __forceinline__ float2 scale_of(float amax) {
  if (amax == 0.0f) return make_float2(1.0f, 0.0f);
  const float a = fmaxf(amax, kAmaxFloor);
  return make_float2(__fdiv_rn(a, kE4m3Max), __fdiv_rn(kE4m3Max, a));
}

template <int N> struct Bytes;
template <> struct Bytes<8> { using type = uint2; };
template <> struct Bytes<4> { using type = uint32_t; };

// N floats to N e4m3 bytes, round to nearest even, saturating; NaN stays NaN.
template <int N>
__device__ __forceinline__ typename Bytes<N>::type to_e4m3(const float (&v)[N], float r) {
  typename Bytes<N>::type out;
  __nv_fp8x2_storage_t *o = reinterpret_cast<__nv_fp8x2_storage_t *>(&out);
#pragma unroll
  for (int i = 0; i < N / 2; ++i)
    o[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * r, v[2 * i + 1] * r), __NV_SATFINITE,
                                    __NV_E4M3);
  return out;
}

// One row per warp (WARP) or per CTA, held in registers as packed vectors:
// x and the residual are read once, and a thread writes only columns that it
// has read, so h and y may replace x or the residual in place.
template <typename T, int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 1024) rmsnorm_kernel(RmsNormArgs a) {
  constexpr int N = Vec<T>::N;
  __shared__ float red[32];
  const int W = WARP ? 32 : blockDim.x;
  const int id = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t row = WARP ? ((int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5))
                           : (int64_t)blockIdx.x;
  if (WARP && row >= a.rows) return;   // a whole warp
  const int nvec = a.d / N;
  const uint4 *x = reinterpret_cast<const uint4 *>(a.x) + row * nvec;
  const uint4 *res = reinterpret_cast<const uint4 *>(a.residual) + row * nvec;
  const uint4 *gam = reinterpret_cast<const uint4 *>(a.gamma);
  uint4 h[NV], g[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = id + i * W;
    h[i] = v < nvec ? x[v] : make_uint4(0, 0, 0, 0);
  }
  if (a.residual != nullptr) {
    uint4 r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = id + i * W;
      r[i] = v < nvec ? res[v] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float xv[N], rv[N];
      unpack16<T>(h[i], xv);
      unpack16<T>(r[i], rv);
#pragma unroll
      for (int k = 0; k < N; ++k) xv[k] = __fadd_rn(xv[k], rv[k]);
      store16<T>(reinterpret_cast<T *>(&h[i]), xv);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = id + i * W;
    g[i] = v < nvec ? gam[v] : make_uint4(0, 0, 0, 0);
  }
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = id + i * W;
    if (a.h != nullptr && v < nvec) reinterpret_cast<uint4 *>(a.h)[row * nvec + v] = h[i];
    float f[N];
    unpack16<T>(h[i], f);
#pragma unroll
    for (int k = 0; k < N; ++k) ss = fmaf(f[k], f[k], ss);
  }
  ss = WARP ? warp_sum(ss) : block_sum(ss, red);
  const float rstd = __frsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)a.d), a.eps));
  if (a.rstd != nullptr && id == 0) a.rstd[row] = rstd;
  if (a.y != nullptr) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = id + i * W;
      float f[N], gv[N];
      unpack16<T>(h[i], f);
      unpack16<T>(g[i], gv);
#pragma unroll
      for (int k = 0; k < N; ++k) f[k] = f[k] * rstd * gv[k];
      if (v < nvec) store16<T>(reinterpret_cast<T *>(a.y) + row * a.d + (int64_t)v * N, f);
    }
  }
  if (a.q == nullptr) return;
  using Q = typename Bytes<N>::type;
  Q *q = reinterpret_cast<Q *>(a.q) + row * nvec;
  if (a.group == 0) {   // one scale for the row
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[N], gv[N];
      unpack16<T>(h[i], f);
      unpack16<T>(g[i], gv);
#pragma unroll
      for (int k = 0; k < N; ++k) m = fmaxf(m, fabsf(f[k] * rstd * gv[k]));
    }
    if (WARP) {
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    } else {
      m = block_max(m, red);
    }
    const float2 sc = scale_of(m);
    if (id == 0) a.q_scale[row] = sc.x;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = id + i * W;
      float f[N], gv[N];
      unpack16<T>(h[i], f);
      unpack16<T>(g[i], gv);
#pragma unroll
      for (int k = 0; k < N; ++k) f[k] = f[k] * rstd * gv[k];
      if (v < nvec) q[v] = to_e4m3<N>(f, sc.y);
    }
    return;
  }
  // a group is group / N consecutive vectors, so consecutive lanes of a warp
  const int lanes = a.group / N;
  const int ng = (a.d + a.group - 1) / a.group;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = id + i * W;
    float f[N], gv[N], m = 0.0f;
    unpack16<T>(h[i], f);
    unpack16<T>(g[i], gv);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      f[k] = f[k] * rstd * gv[k];
      m = fmaxf(m, fabsf(f[k]));
    }
    for (int o = lanes >> 1; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float2 sc = scale_of(m);
    if (v < nvec) {
      if ((v & (lanes - 1)) == 0) a.q_scale[row * ng + v / lanes] = sc.x;
      q[v] = to_e4m3<N>(f, sc.y);
    }
  }
}

// ---------------------------------------------------------------------------
// Backward. A persistent grid: a CTA takes rows blockIdx.x, + gridDim.x, ...;
// a thread keeps the same columns for every row, so its share of dgamma stays
// in registers and leaves once, as a row of `partial`.

template <typename T> __device__ __forceinline__ void load_n(const T *p, float (&v)[8]) {
  if constexpr (Vec<T>::N == 8) {
    load16<T>(p, v);
  } else {
    const float4 a = *reinterpret_cast<const float4 *>(p);
    const float4 b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}
template <typename T> __device__ __forceinline__ void load_n(const T *p, float (&v)[4]) {
  load16<T>(p, v);
}
template <typename T> __device__ __forceinline__ void store_n(T *p, const float (&v)[8]) {
  if constexpr (Vec<T>::N == 8) {
    store16<T>(p, v);
  } else {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
}
template <typename T> __device__ __forceinline__ void store_n(T *p, const float (&v)[4]) {
  store16<T>(p, v);
}

template <typename T, typename TY, typename TX, int NV>
__global__ void __launch_bounds__(NV <= 2 ? 512 : 1024) rmsnorm_bwd_kernel(RmsNormBwdArgs a) {
  constexpr int N = Vec<T>::N;   // columns per thread and step
  __shared__ float red[32];
  const int nvec = a.d / N, W = blockDim.x;
  const T *h = reinterpret_cast<const T *>(a.h);
  const T *dh = reinterpret_cast<const T *>(a.dh);
  const T *gamma = reinterpret_cast<const T *>(a.gamma);
  const TY *dy = reinterpret_cast<const TY *>(a.dy);
  TX *dx = reinterpret_cast<TX *>(a.dx);
  float acc[NV][N];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < N; ++k) acc[i][k] = 0.0f;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float rstd = a.rstd[row];
    float xh[NV][N], gy[NV][N];
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * W;
      if (v < nvec) {
        const int64_t at = row * a.d + (int64_t)v * N;
        float gv[N];
        load_n<T>(h + at, xh[i]);
        load_n<TY>(dy + at, gy[i]);
        load_n<T>(gamma + v * N, gv);
#pragma unroll
        for (int k = 0; k < N; ++k) {
          xh[i][k] *= rstd;
          acc[i][k] = fmaf(gy[i][k], xh[i][k], acc[i][k]);
          gy[i][k] *= gv[k];
          dot = fmaf(gy[i][k], xh[i][k], dot);
        }
      }
    }
    const float m = __fdiv_rn(block_sum(dot, red), (float)a.d);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * W;
      if (v < nvec) {
        const int64_t at = row * a.d + (int64_t)v * N;
        float o[N];
#pragma unroll
        for (int k = 0; k < N; ++k) o[k] = rstd * fmaf(-xh[i][k], m, gy[i][k]);
        if (a.dh != nullptr) {
          float dv[N];
          load_n<T>(dh + at, dv);
#pragma unroll
          for (int k = 0; k < N; ++k) o[k] += dv[k];
        }
        store_n<TX>(dx + at, o);
      }
    }
  }
  float *part = a.partial + (int64_t)blockIdx.x * a.d;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = threadIdx.x + i * W;
    if (v < nvec) store_n<float>(part + v * N, acc[i]);
  }
}

// dgamma[j] = sum over the CTAs' partial rows, in a fixed order: 32 columns
// per CTA, 32 warps taking every 32nd partial row, then the warps in order.
__global__ void __launch_bounds__(1024) dgamma_kernel(const float *partial, int nparts, int d,
                                                      float *dgamma) {
  __shared__ float s[32][33];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j = blockIdx.x * 32 + lane;
  float v = 0.0f;
  if (j < d)
    for (int p = warp; p < nparts; p += 32) v += partial[(int64_t)p * d + j];
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && j < d) {
    float t = 0.0f;
    for (int w = 0; w < 32; ++w) t += s[w][lane];
    dgamma[j] = t;
  }
}

template <typename T, int NV, bool WARP>
cudaError_t fwd(const RmsNormArgs &a, int threads, cudaStream_t s) {
  const int64_t per = WARP ? threads / 32 : 1;
  rmsnorm_kernel<T, NV, WARP><<<(unsigned)((a.rows + per - 1) / per), threads, 0, s>>>(a);
  return cudaGetLastError();
}

constexpr int round32(int v) { return (v + 31) & ~31; }

template <typename T> cudaError_t fwd_t(const RmsNormArgs &a, cudaStream_t s) {
  const int nvec = a.d / Vec<T>::N;
  if (nvec <= 32) return fwd<T, 1, true>(a, 128, s);
  if (nvec <= 64) return fwd<T, 2, true>(a, 128, s);
  if (nvec <= 128) return fwd<T, 4, true>(a, 128, s);
  if (nvec <= 512) return fwd<T, 2, false>(a, round32((nvec + 1) / 2), s);
  return fwd<T, 4, false>(a, round32((nvec + 3) / 4), s);
}

template <typename T, typename TY, typename TX, int NV>
cudaError_t bwd(const RmsNormBwdArgs &a, int threads, cudaStream_t s) {
  int64_t grid = rmsnorm_bwd_max_partials(a.rows);
  const int64_t want = (int64_t)sm_count() * 2;
  if (grid > want) grid = want;
  rmsnorm_bwd_kernel<T, TY, TX, NV><<<(unsigned)grid, threads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_pdl(dgamma_kernel, dim3((a.d + 31) / 32), dim3(1024), 0, s, a.partial, (int)grid, a.d,
                    a.dgamma);
}

template <typename T, typename TY, typename TX>
cudaError_t bwd_t(const RmsNormBwdArgs &a, cudaStream_t s) {
  const int nvec = a.d / Vec<T>::N;
  if (nvec <= 256) return bwd<T, TY, TX, 1>(a, round32(nvec), s);
  if (nvec <= 1024) return bwd<T, TY, TX, 2>(a, round32((nvec + 1) / 2), s);
  return bwd<T, TY, TX, 4>(a, round32((nvec + 3) / 4), s);
}

}  // namespace

// Rows of `partial` that the workspace holds, whatever the device's SM count.
int64_t rmsnorm_bwd_max_partials(int64_t rows) { return rows < 1024 ? rows : 1024; }

cudaError_t launch_rmsnorm(const RmsNormArgs &a, cudaStream_t s) {
  return a.dtype == MOE_BF16 ? fwd_t<__nv_bfloat16>(a, s) : fwd_t<float>(a, s);
}

cudaError_t launch_rmsnorm_bwd(const RmsNormBwdArgs &a, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (a.dtype == MOE_F32) return bwd_t<float, float, float>(a, s);
  if (a.dy_dtype == MOE_F32)
    return a.dx_dtype == MOE_F32 ? bwd_t<B, float, float>(a, s) : bwd_t<B, float, B>(a, s);
  return a.dx_dtype == MOE_F32 ? bwd_t<B, B, float>(a, s) : bwd_t<B, B, B>(a, s);
}

}  // namespace moe
