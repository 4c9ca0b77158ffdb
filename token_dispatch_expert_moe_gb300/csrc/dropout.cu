// Dropout, out = residual + drop(x), and its backward, dx = drop(dy): one pass
// over the data, the mask made from a counter (philox.cuh).
#include "launch.cuh"
#include "philox.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;   // blocks of eight elements a thread has in flight

// eight elements as loaded: one 16-byte word of bf16, two of fp32
template <typename T> struct Eight {
  static constexpr int W = sizeof(T) / 2;
  uint4 w[W];
  __device__ __forceinline__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = reinterpret_cast<const uint4 *>(p)[i];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      float part[Vec<T>::N];
      unpack16<T>(w[i], part);
#pragma unroll
      for (int j = 0; j < Vec<T>::N; ++j) v[i * Vec<T>::N + j] = part[j];
    }
  }
};
template <typename T> __device__ __forceinline__ void store8(T *p, const float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += Vec<T>::N) {
    float part[Vec<T>::N];
#pragma unroll
    for (int j = 0; j < Vec<T>::N; ++j) part[j] = v[i + j];
    store16<T>(p + i, part);
  }
}

template <int J>
__device__ __forceinline__ void drop_one(const Philox &g, const uint4 &w, float scale, float (&v)[8],
                                         const float (&r)[8]) {
  v[J] = g.kept<J>(w) ? fmaf(v[J], scale, r[J]) : r[J];
}
__device__ __forceinline__ void drop8(const Philox &g, const uint4 &w, float scale, float (&v)[8],
                                      const float (&r)[8]) {
  drop_one<0>(g, w, scale, v, r); drop_one<1>(g, w, scale, v, r);
  drop_one<2>(g, w, scale, v, r); drop_one<3>(g, w, scale, v, r);
  drop_one<4>(g, w, scale, v, r); drop_one<5>(g, w, scale, v, r);
  drop_one<6>(g, w, scale, v, r); drop_one<7>(g, w, scale, v, r);
}

// TI: x and dy; TO: out, dx and the residual
template <typename TI, typename TO, bool RES>
__global__ void __launch_bounds__(kThreads) dropout_kernel(int64_t n, const TI *x, const TO *res,
                                                           uint32_t threshold, float scale,
                                                           const uint64_t *rng, TO *out) {
  pdl_wait();
  const int64_t blocks = n / 8;
  const int64_t first = (int64_t)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
  Eight<TI> a[kUnroll];
  Eight<TO> r[RES ? kUnroll : 1];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int64_t b = first + i * kThreads;
    if (b < blocks) {
      a[i].load(x + b * 8);
      if (RES) r[i].load(res + b * 8);
    }
  }
  const Philox g(rng, threshold);
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int64_t b = first + i * kThreads;
    if (b < blocks) {
      const uint4 w = g.block((uint64_t)b);
      float v[8], q[8] = {};
      a[i].get(v);
      if (RES) r[i].get(q);
      drop8(g, w, scale, v, q);
      store8<TO>(out + b * 8, v);
    } else if (b == blocks && (n & 7)) {   // the last, shorter block
      const uint4 w = g.block((uint64_t)b);
      float v[8] = {}, q[8] = {};
      const int m = (int)(n & 7);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < m) {
          v[j] = to_f32(x[b * 8 + j]);
          if (RES) q[j] = to_f32(res[b * 8 + j]);
        }
      drop8(g, w, scale, v, q);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < m) out[b * 8 + j] = from_f32<TO>(v[j]);
    }
  }
}

template <typename TI, typename TO>
cudaError_t run(const DropoutArgs &a, cudaStream_t s) {
  const int64_t per = (int64_t)kThreads * kUnroll;
  const int64_t grid = ((a.n + 7) / 8 + per - 1) / per;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  const TI *x = static_cast<const TI *>(a.x);
  const TO *r = static_cast<const TO *>(a.residual);
  TO *out = static_cast<TO *>(a.out);
  const float scale = drop_scale(a.threshold);
  if (r != nullptr)
    return launch_pdl(dropout_kernel<TI, TO, true>, dim3((unsigned)grid), dim3(kThreads), 0, s, a.n, x, r,
                      a.threshold, scale, a.rng, out);
  return launch_pdl(dropout_kernel<TI, TO, false>, dim3((unsigned)grid), dim3(kThreads), 0, s, a.n, x, r,
                    a.threshold, scale, a.rng, out);
}

}  // namespace

cudaError_t launch_dropout(const DropoutArgs &a, cudaStream_t s) {
  if (a.in_dtype == MOE_F32) {
    return a.out_dtype == MOE_F32 ? run<float, float>(a, s) : run<float, __nv_bfloat16>(a, s);
  }
  return a.out_dtype == MOE_F32 ? run<__nv_bfloat16, float>(a, s) : run<__nv_bfloat16, __nv_bfloat16>(a, s);
}

}  // namespace moe
