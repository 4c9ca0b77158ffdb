// The global norm of many gradient tensors, and clipping by it.
//
//   norm = sqrt(sum over tensors and elements of g^2)
//   coef = max_norm / norm if max_norm < norm < inf, else 1;  out = g coef
//
// Tensors are cut into chunks of 32 KB (norm) or 16 KB (clipping), so a few
// huge tensors and many tiny ones load the grid alike. The squares of a
// thread's share of a chunk are added in fp32 and carried on in fp64; where
// that fp32 sum leaves the safe range (gradients above 1e18 or all below
// 1e-15) the share is summed again in fp64, so the norm is right wherever it
// is an fp32 number. The order of the additions is fixed.
#include <cooperative_groups.h>

#include "launch.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kNormUnroll = 8;   // 16-byte vectors per thread and chunk: chunks of 32 KB
constexpr int kClipUnroll = 4;   // 16 KB
constexpr int kBatch = 96;       // tensors per launch

// Tensors of one launch, passed by value: nothing of the caller's host arrays
// is read after the call. first_chunk[n] is the number of chunks.
struct Batch {
  const void *in[kBatch];
  void *out[kBatch];
  int64_t numel[kBatch];
  int first_chunk[kBatch + 1];
  uint8_t bf16[kBatch];
  int n;
  bool in_place;   // out == in for all of them
};

// A tensor's 16-byte vectors: those that its bytes touch, the first and the
// last perhaps in part.
__host__ __device__ inline int64_t vectors_of(const void *p, int64_t numel, int size) {
  if (numel == 0) return 0;
  const int64_t head = (int64_t)(reinterpret_cast<uintptr_t>(p) & 15u);
  return (head + numel * size + 15) / 16;
}

// The last tensor whose first chunk is not after `chunk`.
__device__ __forceinline__ int tensor_of(const Batch &b, int chunk) {
  int lo = 0, hi = b.n - 1;
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
  constexpr int kUnroll = kNormUnroll;
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

// Sum of the squares of chunks first, first + step, ...; valid in thread 0.
__device__ __forceinline__ double squares_of(const Batch &b, int64_t first, int step, double *red) {
  double s = 0.0;
  const int64_t chunks = b.first_chunk[b.n];
  if (first < chunks) {
    int i = tensor_of(b, (int)first);
    for (int64_t c = first; c < chunks; c += step) {
      while (b.first_chunk[i + 1] <= c) ++i;
      const int64_t v0 = (c - b.first_chunk[i]) * (kThreads * kNormUnroll);
      s += b.bf16[i] ? chunk_squares(static_cast<const __nv_bfloat16 *>(b.in[i]), b.numel[i], v0)
                     : chunk_squares(static_cast<const float *>(b.in[i]), b.numel[i], v0);
    }
  }
  return block_sum_double(s, red);
}

__global__ void __launch_bounds__(kThreads) squares_kernel(const __grid_constant__ Batch b,
                                                           double *partial, int add) {
  __shared__ double red[32];
  pdl_wait();   // the gradients, and the call before that may still read `partial`
  const double s = squares_of(b, blockIdx.x, gridDim.x, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = add ? partial[blockIdx.x] + s : s;
}

// The whole norm of a short list in one launch: one cluster, whose CTAs hand
// their sums to the first through shared memory. Up to 16 chunks it takes the
// GPU no longer than the two kernels (3.2 to 4.4 us against 4.0 to 4.3) and the
// host one launch less (a stream of calls: 4.3 us each against 5.8); with 32
// chunks 6.1 us against 4.4.
constexpr int kSmallCtas = 8, kSmallChunks = 16;

__global__ void __cluster_dims__(kSmallCtas, 1, 1) __launch_bounds__(kThreads)
small_norm_kernel(const __grid_constant__ Batch b, float *norm) {
  cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
  __shared__ double red[32], all[kSmallCtas];
  pdl_wait();
  cluster.sync();   // all CTAs run: the first one's shared memory may be written
  const int rank = (int)cluster.block_rank();
  const double s = squares_of(b, rank, kSmallCtas, red);
  if (threadIdx.x == 0) *cluster.map_shared_rank(&all[rank], 0) = s;
  cluster.sync();
  if (rank == 0 && threadIdx.x == 0) {
    double t = 0.0;
    for (int r = 0; r < kSmallCtas; ++r) t += all[r];
    norm[0] = (float)sqrt(t);
  }
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const double *partial, int n, float *norm) {
  __shared__ double red[32];
  pdl_wait();
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
  constexpr int kUnroll = kClipUnroll;
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
                                                        float *coef_out, int per) {
  pdl_wait();
  const float coef = coef_of(norm[0], max_norm);
  if (coef_out != nullptr && blockIdx.x == 0 && threadIdx.x == 0) coef_out[0] = coef;
  if (coef == 1.0f && b.in_place) return;
  // last chunks first: the norm's pass has left the tail in L2
  const int hi = b.first_chunk[b.n] - 1 - (int)blockIdx.x * per;
  int i = tensor_of(b, hi);
  for (int c = hi; c >= 0 && c > hi - per; --c) {
    while (b.first_chunk[i] > c) --i;
    const int64_t v0 = (int64_t)(c - b.first_chunk[i]) * (kThreads * kClipUnroll);
    if (b.bf16[i])
      scale_chunk(static_cast<const __nv_bfloat16 *>(b.in[i]), static_cast<__nv_bfloat16 *>(b.out[i]),
                  b.numel[i], v0, coef);
    else
      scale_chunk(static_cast<const float *>(b.in[i]), static_cast<float *>(b.out[i]), b.numel[i],
                  v0, coef);
  }
}

// Tensors [at, ...) of the list as a batch; returns the first that is left. A
// batch ends before its chunks pass 2^30 (16 TB), so that 32 bits count them;
// list_check has seen to it that one tensor alone does not.
int fill(Batch &b, int at, int n, const moe_tensor_t *in, const moe_tensor_t *out, int chunk_vecs) {
  b.n = 0;
  b.in_place = true;
  int64_t chunks = 0;
  for (; at < n && b.n < kBatch; ++at) {
    if (in[at].numel == 0) continue;
    const bool bf16 = in[at].dtype == MOE_BF16;
    const int64_t nvec = vectors_of(in[at].data, in[at].numel, bf16 ? 2 : 4);
    const int64_t more = (nvec + chunk_vecs - 1) / chunk_vecs;
    if (b.n > 0 && chunks + more > (int64_t(1) << 30)) break;
    const int i = b.n++;
    b.in[i] = in[at].data;
    b.out[i] = out != nullptr ? out[at].data : in[at].data;
    if (b.out[i] != b.in[i]) b.in_place = false;
    b.numel[i] = in[at].numel;
    b.bf16[i] = bf16;
    b.first_chunk[i] = (int)chunks;
    chunks += more;
  }
  b.first_chunk[b.n] = (int)chunks;
  return at;
}

}  // namespace

cudaError_t launch_grad_norm(int n, const moe_tensor_t *grads, float *norm, double *partial,
                             cudaStream_t s) {
  // a persistent grid of what the registers let an SM hold (7.5 GB: 1015 us,
  // 7.41 TB/s; 4 CTAs an SM, so a second wave, 1240 us)
  int ctas = sm_count() * 3;
  if (ctas > kMaxNormPartials) ctas = kMaxNormPartials;
  int grid = 0;   // CTAs of every batch, so partials that hold a sum
  Batch b;
  for (int at = 0; at < n;) {
    at = fill(b, at, n, grads, nullptr, kThreads * kNormUnroll);
    if (b.n == 0) break;
    const bool first = grid == 0;
    if (first && at == n && b.first_chunk[b.n] <= kSmallChunks)
      return launch_pdl(small_norm_kernel, dim3(kSmallCtas), dim3(kThreads), 0, s, b, norm);
    if (first) grid = at == n && b.first_chunk[b.n] < ctas ? b.first_chunk[b.n] : ctas;
    cudaError_t e = launch_pdl(squares_kernel, dim3((unsigned)grid), dim3(kThreads), 0, s, b,
                               partial, first ? 0 : 1);   // later batches add theirs
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(norm_kernel, dim3(1), dim3(kThreads), 0, s, (const double *)partial, grid, norm);
}

cudaError_t launch_grad_clip(int n, const moe_tensor_t *grads, const moe_tensor_t *out,
                             const float *norm, float max_norm, float *coef, cudaStream_t s) {
  Batch b;
  int at = 0;
  bool first = true;
  do {
    at = fill(b, at, n, grads, out, kThreads * kClipUnroll);
    if (b.n == 0 && !first) break;
    // A CTA per chunk, like the norm's rows: DRAM rewards a narrow window (7.5
    // GB: 2100 us, 7.16 TB/s; a persistent grid 2200 us). In place the call
    // often has nothing to do, and then costs the launch of its CTAs (7.5 GB:
    // 465 us with a chunk each, 118 us with four, which clip in 2138 us): four
    // chunks a CTA once they outnumber the CTAs that the SMs hold.
    const int chunks = b.first_chunk[b.n];
    const int per = b.in_place && chunks > sm_count() * 8 ? 4 : 1;
    const int ctas = (chunks + per - 1) / per;
    cudaError_t e = launch_pdl(clip_kernel, dim3((unsigned)(ctas > 0 ? ctas : 1)), dim3(kThreads), 0, s,
                               b, norm, max_norm, first ? coef : (float *)nullptr, per);
    if (e != cudaSuccess) return e;
    first = false;
  } while (at < n);
  return cudaSuccess;
}

}  // namespace moe
