// The global norm of many gradient tensors, and clipping by it.
//
//   norm = sqrt(sum over tensors and elements of g^2)
//   coef = max_norm / norm if max_norm < norm < inf, else 1;  out = g coef
//
// Tensors are cut into chunks of kChunkBytes; a persistent grid takes chunk
// after chunk, so a few huge tensors and many tiny ones load it alike. The
// squares of a thread's share of a chunk are added in fp32 and carried on in
// fp64; where that fp32 sum leaves the safe range (gradients above 1e18 or all
// below 1e-15) the share is summed again in fp64, so the norm is right
// wherever it is an fp32 number. The order of the additions is fixed.
#include "launch.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 8;                               // 16-byte vectors per thread and chunk
constexpr int64_t kChunkVecs = kThreads * kUnroll;       // 32 KB
constexpr int kBatch = 96;                               // tensors per launch

// Tensors of one launch, passed by value: nothing of the caller's host arrays
// is read after the call. first_chunk[n] is the number of chunks.
struct Batch {
  const void *in[kBatch];
  void *out[kBatch];
  int64_t numel[kBatch];
  int64_t first_chunk[kBatch + 1];
  uint8_t bf16[kBatch];
  int n;
};

// A tensor's 16-byte vectors: those that its bytes touch, the first and the
// last perhaps in part.
__host__ __device__ inline int64_t vectors_of(const void *p, int64_t numel, int size) {
  if (numel == 0) return 0;
  const int64_t head = (int64_t)(reinterpret_cast<uintptr_t>(p) & 15u);
  return (head + numel * size + 15) / 16;
}

__device__ __forceinline__ int tensor_of(const Batch &b, int64_t chunk) {
  int lo = 0, hi = b.n - 1;   // the last tensor whose first chunk is <= chunk
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.first_chunk[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Vector v of a tensor, elements outside it zero.
template <typename T>
__device__ __forceinline__ uint4 load_vec(const T *p, int64_t numel, int64_t v) {
  constexpr int N = Vec<T>::N;
  const int64_t head = (int64_t)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
  const int64_t lo = v * N - head;   // element index of the vector's start
  if (lo >= 0 && lo + N <= numel) return *reinterpret_cast<const uint4 *>(p + lo);
  uint4 u = make_uint4(0, 0, 0, 0);
  T *e = reinterpret_cast<T *>(&u);
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (lo + i >= 0 && lo + i < numel) e[i] = p[lo + i];
  return u;
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T *p, int64_t numel, int64_t v0) {
  constexpr int N = Vec<T>::N;
  const int64_t nvec = vectors_of(p, numel, sizeof(T));
  uint4 u[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int64_t v = v0 + i * kThreads + threadIdx.x;
    u[i] = v < nvec ? load_vec<T>(p, numel, v) : make_uint4(0, 0, 0, 0);
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    float f[N];
    unpack16<T>(u[i], f);
#pragma unroll
    for (int k = 0; k < N; ++k) s = fmaf(f[k], f[k], s);
  }
  if (s < 1e37f && s > 1e-30f) return (double)s;
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) any |= u[i].x | u[i].y | u[i].z | u[i].w;
  if (any == 0) return 0.0;
  double d = 0.0;   // outside the range that fp32 squares hold, or not finite
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    float f[N];
    unpack16<T>(u[i], f);
#pragma unroll
    for (int k = 0; k < N; ++k) d = fma((double)f[k], (double)f[k], d);
  }
  return d;
}

// Sum of doubles over the CTA, in a fixed order; valid in thread 0.
__device__ __forceinline__ double block_sum_double(double v, double *smem32) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) smem32[warp] = v;
  __syncthreads();
  double r = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) r += smem32[w];
  return r;
}

__global__ void __launch_bounds__(kThreads) squares_kernel(const __grid_constant__ Batch b,
                                                           double *partial, int add) {
  __shared__ double red[32];
  pdl_wait();   // the gradients, and the call before that may still read `partial`
  pdl_trigger();
  double s = 0.0;
  const int64_t chunks = b.first_chunk[b.n];
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = tensor_of(b, c);
    const int64_t v0 = (c - b.first_chunk[i]) * kChunkVecs;
    s += b.bf16[i] ? chunk_squares(static_cast<const __nv_bfloat16 *>(b.in[i]), b.numel[i], v0)
                   : chunk_squares(static_cast<const float *>(b.in[i]), b.numel[i], v0);
  }
  s = block_sum_double(s, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = add ? partial[blockIdx.x] + s : s;
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const double *partial, int n, float *norm) {
  __shared__ double red[32];
  pdl_wait();
  pdl_trigger();
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) s += partial[i];
  s = block_sum_double(s, red);
  if (threadIdx.x == 0) norm[0] = (float)sqrt(s);
}

__device__ __forceinline__ float coef_of(float norm, float max_norm) {
  return norm > max_norm && norm < INFINITY ? __fdiv_rn(max_norm, norm) : 1.0f;
}

template <typename T>
__device__ __forceinline__ void scale_chunk(const T *in, T *out, int64_t numel, int64_t v0,
                                            float coef) {
  constexpr int N = Vec<T>::N;
  const int64_t head = (int64_t)((reinterpret_cast<uintptr_t>(in) & 15u) / sizeof(T));
  const int64_t nvec = vectors_of(in, numel, sizeof(T));
  // both sides at the same place within their 16 bytes: whole vectors move
  const bool same = ((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
  uint4 u[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int64_t v = v0 + i * kThreads + threadIdx.x;
    if (v < nvec) u[i] = load_vec<T>(in, numel, v);
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int64_t v = v0 + i * kThreads + threadIdx.x;
    if (v >= nvec) continue;
    float f[N];
    unpack16<T>(u[i], f);
#pragma unroll
    for (int k = 0; k < N; ++k) f[k] *= coef;
    const int64_t lo = v * N - head;
    if (same && lo >= 0 && lo + N <= numel) {
      store16<T>(out + lo, f);
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (lo + k >= 0 && lo + k < numel) out[lo + k] = from_f32<T>(f[k]);
    }
  }
}

__global__ void __launch_bounds__(kThreads) clip_kernel(const __grid_constant__ Batch b,
                                                        const float *norm, float max_norm,
                                                        float *coef_out) {
  pdl_wait();
  pdl_trigger();
  const float coef = coef_of(norm[0], max_norm);
  if (coef_out != nullptr && blockIdx.x == 0 && threadIdx.x == 0) coef_out[0] = coef;
  const int64_t chunks = b.first_chunk[b.n];
  // last chunk first: the norm's pass has left the tail in L2
  for (int64_t c = chunks - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
    const int i = tensor_of(b, c);
    const int64_t v0 = (c - b.first_chunk[i]) * kChunkVecs;
    if (coef == 1.0f && b.in[i] == b.out[i]) continue;
    if (b.bf16[i])
      scale_chunk(static_cast<const __nv_bfloat16 *>(b.in[i]), static_cast<__nv_bfloat16 *>(b.out[i]),
                  b.numel[i], v0, coef);
    else
      scale_chunk(static_cast<const float *>(b.in[i]), static_cast<float *>(b.out[i]), b.numel[i],
                  v0, coef);
  }
}

// Tensors [at, ...) of the list as a batch; returns the first that is left.
int fill(Batch &b, int at, int n, const moe_tensor_t *in, const moe_tensor_t *out) {
  b.n = 0;
  int64_t chunks = 0;
  for (; at < n && b.n < kBatch; ++at) {
    if (in[at].numel == 0) continue;
    const int i = b.n++;
    b.in[i] = in[at].data;
    b.out[i] = out != nullptr ? out[at].data : in[at].data;
    b.numel[i] = in[at].numel;
    b.bf16[i] = in[at].dtype == MOE_BF16;
    b.first_chunk[i] = chunks;
    const int64_t nvec = vectors_of(b.in[i], b.numel[i], b.bf16[i] ? 2 : 4);
    chunks += (nvec + kChunkVecs - 1) / kChunkVecs;
  }
  b.first_chunk[b.n] = chunks;
  return at;
}

int grid_of(const Batch &b, int ctas) {
  const int64_t chunks = b.first_chunk[b.n];
  return (int)(chunks < ctas ? (chunks > 0 ? chunks : 1) : ctas);
}

}  // namespace

cudaError_t launch_grad_norm(int n, const moe_tensor_t *grads, float *norm, double *partial,
                             cudaStream_t s) {
  int ctas = sm_count() * 8;
  if (ctas > kMaxNormPartials) ctas = kMaxNormPartials;
  int grid = 0;   // CTAs of every batch, so partials that hold a sum
  Batch b;
  for (int at = 0; at < n;) {
    at = fill(b, at, n, grads, nullptr);
    if (b.n == 0) break;
    const bool first = grid == 0;
    if (first) grid = at < n ? ctas : grid_of(b, ctas);
    cudaError_t e = launch_pdl(squares_kernel, dim3((unsigned)grid), dim3(kThreads), 0, s, b,
                               partial, first ? 0 : 1);   // later batches add theirs
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(norm_kernel, dim3(1), dim3(kThreads), 0, s, (const double *)partial, grid, norm);
}

cudaError_t launch_grad_clip(int n, const moe_tensor_t *grads, const moe_tensor_t *out,
                             const float *norm, float max_norm, float *coef, cudaStream_t s) {
  const int ctas = sm_count() * 8;
  Batch b;
  int at = 0;
  bool first = true;
  do {
    at = fill(b, at, n, grads, out);
    if (b.n == 0 && !first) break;
    cudaError_t e = launch_pdl(clip_kernel, dim3((unsigned)grid_of(b, ctas)), dim3(kThreads), 0, s, b,
                               norm, max_norm, first ? coef : (float *)nullptr);
    if (e != cudaSuccess) return e;
    first = false;
  } while (at < n);
  return cudaSuccess;
}

}  // namespace moe
