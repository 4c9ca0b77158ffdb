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
#include <atomic>

#include <cooperative_groups.h>
#include <cuda_fp8.h>

#include "launch.cuh"

namespace moe {
namespace {

constexpr float kE4m3Max = 448.0f;
// Smallest amax a scale is made of: the scale and its reciprocal stay normal numbers.
constexpr float kAmaxFloor = 7.70372e-34f;   // 2^-110

// Sum or maximum over the CTA with one barrier: every warp writes its value
// and reads them all. `red` alternates between two rows from call to call, so
// that a warp ahead by one call overwrites nothing that is still read.
template <bool MAX> __device__ __forceinline__ float reduce_op(float a, float b) {
  return MAX ? fmaxf(a, b) : a + b;
}
template <bool MAX>
__device__ __forceinline__ float warp_reduce(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v = reduce_op<MAX>(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <bool MAX>
__device__ __forceinline__ float cta_reduce(float v, float (&red)[2][32], int &turn) {
  v = warp_reduce<MAX>(v);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) red[turn][warp] = v;
  __syncthreads();
  v = lane < (int)(blockDim.x >> 5) ? red[turn][lane] : 0.0f;
  turn ^= 1;
  return warp_reduce<MAX>(v);
}

// Copies of 16 or 8 bytes to shared memory that complete in the background;
// a thread copies only what it reads itself, so waiting for its own groups is
// all the synchronisation that they need.
template <int BYTES> __device__ __forceinline__ void copy_async(void *smem, const void *gmem) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(gmem) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(d), "l"(gmem) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float reciprocal(float v) {   // within 1 ulp
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Scale of a group and the factor that y is multiplied with, its reciprocal.
// The largest |y| may come out a few ulp above 448: the conversion saturates.
__device__ __forceinline__ float2 scale_of(float amax) {
  if (amax == 0.0f) return make_float2(1.0f, 0.0f);
  const float s = fmaxf(amax, kAmaxFloor) * (1.0f / kE4m3Max);
  return make_float2(s, reciprocal(s));
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

// h = dtype(x + residual) of one vector
template <typename T> __device__ __forceinline__ uint4 add_residual(uint4 x, uint4 r) {
  constexpr int N = Vec<T>::N;
  float xv[N], rv[N];
  unpack16<T>(x, xv);
  unpack16<T>(r, rv);
#pragma unroll
  for (int k = 0; k < N; ++k) xv[k] = __fadd_rn(xv[k], rv[k]);
  uint4 h;
  store16<T>(reinterpret_cast<T *>(&h), xv);
  return h;
}

// The row's outputs from its h and gamma (in registers, W threads, vector
// id + i W in thread id): y, and q with its scales.
template <typename T, int NV, bool WARP>
__device__ __forceinline__ void write_row(const RmsNormArgs &a, int64_t row, int id, int W,
                                          const uint4 (&h)[NV], const uint4 (&g)[NV], float rstd,
                                          float (&red)[2][32], int &turn) {
  constexpr int N = Vec<T>::N;
  using Q = typename Bytes<N>::type;
  const int nvec = a.d / N;
  T *y = reinterpret_cast<T *>(a.y) + row * a.d;
  Q *q = reinterpret_cast<Q *>(a.q) + row * nvec;
  float2 sc = make_float2(0.0f, 0.0f);
  if (a.q != nullptr && a.group == 0) {   // one scale for the row
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[N], gv[N];
      unpack16<T>(h[i], f);
      unpack16<T>(g[i], gv);
#pragma unroll
      for (int k = 0; k < N; ++k) m = fmaxf(m, fabsf(f[k] * rstd * gv[k]));
    }
    m = WARP ? warp_reduce<true>(m) : cta_reduce<true>(m, red, turn);
    sc = scale_of(m);
    if (id == 0) a.q_scale[row] = sc.x;
  }
  // a group is 2^group_shift consecutive vectors, so consecutive lanes of a
  // warp: 4 to 32 of them
  const int last = (1 << a.group_shift) - 1;
  float *scales = a.q_scale + row * a.ng;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = id + i * W;
    const bool in = v < nvec;
    float f[N], gv[N];
    unpack16<T>(h[i], f);
    unpack16<T>(g[i], gv);
#pragma unroll
    for (int k = 0; k < N; ++k) f[k] = f[k] * rstd * gv[k];
    if (a.y != nullptr && in) store16<T>(y + v * N, f);
    if (a.q != nullptr) {
      if (a.group > 0) {
        float m = 0.0f;
#pragma unroll
        for (int k = 0; k < N; ++k) m = fmaxf(m, fabsf(f[k]));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
#pragma unroll
        for (int o = 4; o <= 16; o *= 2)
          if (o <= last) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        sc = scale_of(m);
        if (in && (v & last) == 0) scales[v >> a.group_shift] = sc.x;
      }
      if (in) q[v] = to_e4m3<N>(f, sc.y);
    }
  }
}

__device__ __forceinline__ float rstd_of(float ss, const RmsNormArgs &a) {
  return rsqrtf(fmaf(ss, a.inv_d, a.eps));   // within 2 ulp
}

// One row per warp (WARP) or per CTA, held in registers as packed vectors: x
// and the residual are read once, and a thread writes only columns that it has
// read, so h and y may replace x or the residual in place. HBM-bound. The
// grid is one CTA per row, not a persistent one: CTAs that start in order walk
// the matrices in a narrow window, which DRAM rewards (32768 x 8192 bf16 with
// residual and 8-bit rows: 359 us, 6.72 TB/s; persistent CTAs with the next
// rows fetched ahead through shared memory, in 2 to 4 stages: 404 to 414 us).
// Two vectors a thread: one takes 366 us, four 408 us (one row alone: 1.7 us on
// 6144 columns with two, 1.8 with one). 56 registers for two vectors: one fewer
// than the compiler takes by itself, and a third CTA of 384 threads fits
// (16384 x 6144: 150 -> 134 us; 32768 x 8192, CTAs of 512: 360 -> 362 us). The
// layout goes by d alone, so a row's results do not depend on the other rows.
template <typename T, int NV, bool WARP>
__global__ void __maxnreg__(WARP ? 80 : NV == 2 ? 56 : 64) rmsnorm_kernel(RmsNormArgs a) {
  constexpr int N = Vec<T>::N;
  __shared__ float red[2][32];
  int turn = 0;
  pdl_wait();
  const int W = WARP ? 32 : blockDim.x;
  const int id = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t row = WARP ? ((int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5))
                           : (int64_t)blockIdx.x;
  if (WARP && row >= a.rows) return;   // a whole warp
  const int nvec = a.d / N;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const uint4 *x = reinterpret_cast<const uint4 *>(a.x) + row * nvec;
  const uint4 *res = reinterpret_cast<const uint4 *>(a.residual) + row * nvec;
  const uint4 *gam = reinterpret_cast<const uint4 *>(a.gamma);
  uint4 h[NV], g[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = id + i * W;
    h[i] = v < nvec ? x[v] : zero;
    g[i] = v < nvec ? gam[v] : zero;
  }
  if (a.residual != nullptr) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = id + i * W;
      h[i] = add_residual<T>(h[i], v < nvec ? res[v] : zero);
    }
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
  ss = WARP ? warp_reduce<false>(ss) : cta_reduce<false>(ss, red, turn);
  const float rstd = rstd_of(ss, a);
  if (a.rstd != nullptr && id == 0) a.rstd[row] = rstd;
  write_row<T, NV, WARP>(a, row, id, W, h, g, rstd, red, turn);
}

// ---------------------------------------------------------------------------
// Backward. Persistent grids: a CTA (or a warp of it) takes row after row, and
// a thread keeps the same columns for every row, so its share of dgamma stays
// in registers and leaves once, in the CTA's row of `partial`. A thread's unit
// is 4 columns, 16 bytes of fp32 or 8 of bf16, so that every access of a warp
// is contiguous whatever mixture of types the call has.

template <typename T> struct Unit;
template <> struct Unit<float> { using type = float4; };
template <> struct Unit<__nv_bfloat16> { using type = uint2; };

__device__ __forceinline__ void unpack4(const float4 &u, float (&v)[4]) {
  v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
}
__device__ __forceinline__ void unpack4(const uint2 &u, float (&v)[4]) {
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.y));
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}
__device__ __forceinline__ void pack4(const float (&v)[4], float4 *out) {
  *out = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void pack4(const float (&v)[4], uint2 *out) {
  uint2 u;
  *reinterpret_cast<__nv_bfloat162 *>(&u.x) = __floats2bfloat162_rn(v[0], v[1]);
  *reinterpret_cast<__nv_bfloat162 *>(&u.y) = __floats2bfloat162_rn(v[2], v[3]);
  *out = u;
}

template <typename T, typename TY> constexpr int bwd_unit_bytes(bool dh) {
  return 4 * (int)(sizeof(TY) + sizeof(T) * (dh ? 2 : 1));
}

// Rows of up to 512 columns: one per warp, eight warps a CTA, whose shares of
// dgamma meet in shared memory at the end. Its many warps are what hides the
// loads' latency.
constexpr int kRowWarps = 8;

template <typename T, typename TY, typename TX, int NU, bool DH>
__global__ void __launch_bounds__(kRowWarps * 32) rmsnorm_bwd_warp_kernel(RmsNormBwdArgs a) {
  using UT = typename Unit<T>::type;
  using UY = typename Unit<TY>::type;
  using UX = typename Unit<TX>::type;
  __shared__ float sum[NU * 32 * 4];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nu = a.d / 4;
  const UY *dy = reinterpret_cast<const UY *>(a.dy);
  const UT *h = reinterpret_cast<const UT *>(a.h);
  const UT *dh = reinterpret_cast<const UT *>(a.dh);
  UX *dx = reinterpret_cast<UX *>(a.dx);
  UT g[NU];
  float acc[NU][4];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int u = lane + i * 32;
    g[i] = u < nu ? reinterpret_cast<const UT *>(a.gamma)[u] : UT{};
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[i][k] = 0.0f;
  }
  const int64_t step = (int64_t)gridDim.x * kRowWarps;
  for (int64_t row = (int64_t)blockIdx.x * kRowWarps + warp; row < a.rows; row += step) {
    UY yv[NU];
    UT hv[NU], dv[NU];
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int u = lane + i * 32;
      yv[i] = u < nu ? dy[row * nu + u] : UY{};
      hv[i] = u < nu ? h[row * nu + u] : UT{};
      if (DH) dv[i] = u < nu ? dh[row * nu + u] : UT{};
    }
    const float rstd = a.rstd[row];
    float xh[NU][4], gy[NU][4];   // xhat and dy gamma
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      float y4[4], gv[4];
      unpack4(yv[i], y4);
      unpack4(hv[i], xh[i]);
      unpack4(g[i], gv);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        xh[i][k] *= rstd;
        gy[i][k] = y4[k] * gv[k];
        acc[i][k] = fmaf(y4[k], xh[i][k], acc[i][k]);
        dot = fmaf(gy[i][k], xh[i][k], dot);
      }
    }
    const float m = warp_reduce<false>(dot) * a.inv_d;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int u = lane + i * 32;
      float o[4], d4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (DH) unpack4(dv[i], d4);
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = rstd * fmaf(-xh[i][k], m, gy[i][k]) + d4[k];
      if (u < nu) pack4(o, dx + row * nu + u);
    }
  }
  for (int w = 0; w < kRowWarps; ++w) {   // the warps add in order
    if (warp == w) {
#pragma unroll
      for (int i = 0; i < NU; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float *p = sum + (lane + i * 32) * 4 + k;
          *p = w == 0 ? acc[i][k] : *p + acc[i][k];
        }
    }
    __syncthreads();
  }
  for (int j = threadIdx.x; j < a.d; j += blockDim.x) a.partial[(int64_t)blockIdx.x * a.d + j] = sum[j];
}

// Wider rows: one per CTA, or per cluster of CTAs with a part of the columns
// each. A ring of STAGES rows in shared memory: the next rows' dy, h and dh are
// on their way while one row is reduced and written, so the loads run on across
// the reduction's barrier (32768 x 8192, dy and dx fp32, dh bf16: 480 us, 6.7
// TB/s; plain loads 821 us). Three rows where they fit and leave one CTA to an
// SM anyway (16384 x 6144: 177 us, with two 199 us), two where more CTAs fit
// then (65536 x 1024: 121 us, with three 129 us) and where three do not fit
// (16384 x 8192, all fp32: 308 us).
// WIDE: bf16 rows of more than 8192 columns, 1024 threads. dh goes to registers
// instead of the ring, and dy and h are read from the ring twice, before and
// after the row's sum, which leaves room for both (16384 x 16384: 481 us, 6.69
// TB/s; plain loads that read dy and h twice 800 us, two CTAs a row 613 us).
// CLUSTER: rows of more than 8192 (fp32) or 16384 (bf16) columns. The CTAs add
// up their sums through each other's shared memory; that barrier takes 1 us a
// row, so no narrower row is cut (8192 x 32768: 537 us, 6.0 TB/s).
constexpr int kMaxCluster = 2, kNarrow = 8192, kWide = 16384;

template <typename T, typename TY, typename TX, bool DH, int STAGES, bool WIDE, bool CLUSTER>
__global__ void __launch_bounds__(WIDE ? 1024 : 512) rmsnorm_bwd_kernel(RmsNormBwdArgs a) {
  using UT = typename Unit<T>::type;
  using UY = typename Unit<TY>::type;
  using UX = typename Unit<TX>::type;
  namespace cg = cooperative_groups;
  constexpr int NU = 4;             // units per thread
  extern __shared__ uint4 ring[];   // per stage: dy [NU][W], h [NU][W], dh [NU][W]
  __shared__ float red[2][32 * (CLUSTER ? kMaxCluster : 1)];
  int turn = 0;
  pdl_wait();
  const int W = blockDim.x, id = threadIdx.x, units = a.d / 4;
  int ctas = 1, rank = 0;
  if constexpr (CLUSTER) {
    ctas = (int)cg::this_cluster().num_blocks();
    rank = (int)cg::this_cluster().block_rank();
    cg::this_cluster().sync();   // all of them run: their shared memory may be written
  }
  // this CTA's units: [first, first + nu)
  const int share = (units + ctas - 1) / ctas, first = rank * share;
  const int nu = min(share, units - first);
  const UY *dy = reinterpret_cast<const UY *>(a.dy) + first;
  const UT *h = reinterpret_cast<const UT *>(a.h) + first;
  const UT *dh = reinterpret_cast<const UT *>(a.dh) + first;
  UX *dx = reinterpret_cast<UX *>(a.dx) + first;
  const int64_t row0 = blockIdx.x / ctas, step = gridDim.x / ctas;
  const size_t stage_bytes = (size_t)NU * W * bwd_unit_bytes<T, TY>(DH && !WIDE);
  auto dy_at = [&](int stage) {
    return reinterpret_cast<UY *>(reinterpret_cast<char *>(ring) + stage * stage_bytes) + id;
  };
  auto h_at = [&](int stage) {
    return reinterpret_cast<UT *>(reinterpret_cast<char *>(ring) + stage * stage_bytes +
                                  (size_t)NU * W * sizeof(UY)) + id;
  };
  auto fetch = [&](int64_t row, int stage) {
    if (row < a.rows) {
      UY *sy = dy_at(stage);
      UT *sh = h_at(stage);
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        const int u = id + i * W;
        if (u < nu) {
          copy_async<sizeof(UY)>(sy + i * W, dy + row * units + u);
          copy_async<sizeof(UT)>(sh + i * W, h + row * units + u);
          if (DH && !WIDE) copy_async<sizeof(UT)>(sh + (NU + i) * W, dh + row * units + u);
        }
      }
    }
    copy_commit();   // an empty group past the end keeps the count
  };
  // sum over the row's CTAs of a value per thread
  auto row_sum = [&](float v) {
    if constexpr (!CLUSTER) {
      return cta_reduce<false>(v, red, turn);
    } else {
      v = warp_reduce<false>(v);
      const int lane = id & 31, slot = rank * 32 + (id >> 5);
      if (lane < ctas) *cg::this_cluster().map_shared_rank(&red[turn][slot], lane) = v;
      cg::this_cluster().sync();
      const bool in = lane < (W >> 5);
      v = 0.0f;
      for (int r = 0; r < ctas; ++r) v += in ? red[turn][r * 32 + lane] : 0.0f;
      turn ^= 1;
      return warp_reduce<false>(v);
    }
  };
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) fetch(row0 + s * step, s);
  UT g[NU];
  float acc[NU][4];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int u = id + i * W;
    g[i] = u < nu ? (reinterpret_cast<const UT *>(a.gamma) + first)[u] : UT{};
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[i][k] = 0.0f;
  }
  int stage = 0;
  for (int64_t row = row0; row < a.rows; row += step) {
    const float rstd = a.rstd[row];
    // the stage read one row ago is free: its values have gone into that row's dx
    fetch(row + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
    copy_wait<STAGES - 1>();   // this row's group
    UT dv[NU];
    if (DH && WIDE) {
#pragma unroll
      for (int i = 0; i < NU; ++i)
        if (id + i * W < nu) dv[i] = dh[row * units + id + i * W];
    }
    float xh[NU][4], gy[NU][4];   // xhat and dy gamma
    auto read = [&](int i, float (&y4)[4]) {
      float gv[4];
      unpack4(dy_at(stage)[i * W], y4);
      unpack4(h_at(stage)[i * W], xh[i]);
      unpack4(g[i], gv);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        xh[i][k] *= rstd;
        gy[i][k] = y4[k] * gv[k];
      }
    };
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      if (id + i * W < nu) {
        float y4[4];
        read(i, y4);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          acc[i][k] = fmaf(y4[k], xh[i][k], acc[i][k]);
          dot = fmaf(gy[i][k], xh[i][k], dot);
        }
      }
    }
    const float m = row_sum(dot) * a.inv_d;
    if (DH && !WIDE) {
#pragma unroll
      for (int i = 0; i < NU; ++i) dv[i] = h_at(stage)[(NU + i) * W];
    }
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int u = id + i * W;
      if (u < nu) {
        if (WIDE) {   // not kept across the barrier
          float y4[4];
          read(i, y4);
        }
        float o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = rstd * fmaf(-xh[i][k], m, gy[i][k]);
        if (DH) {
          float d4[4];
          unpack4(dv[i], d4);
#pragma unroll
          for (int k = 0; k < 4; ++k) o[k] += d4[k];
        }
        pack4(o, dx + row * units + u);
      }
    }
    stage = stage == STAGES - 1 ? 0 : stage + 1;
  }
  copy_wait<0>();
  float4 *part = reinterpret_cast<float4 *>(a.partial + row0 * a.d) + first;
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int u = id + i * W;
    if (u < nu) pack4(acc[i], part + u);
  }
  if constexpr (CLUSTER) cg::this_cluster().sync();   // no CTA ends while another writes to it
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
#pragma unroll 8
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
  return launch_pdl(rmsnorm_kernel<T, NV, WARP>, dim3((unsigned)((a.rows + per - 1) / per)),
                    dim3(threads), 0, s, a);
}

constexpr int round32(int v) { return (v + 31) & ~31; }
constexpr size_t kSmem = 226 * 1024;   // of the 227 KB that a CTA may have; the rest for static arrays

// CTAs of a persistent grid: those that fit the device at once, at most
// `most`. The answer for the last device and size that a kernel was asked for
// is kept (one word, so that threads may race for it): the two calls behind it
// cost the host 1 us, half of what the launch does. The limit that is set here
// belongs to the kernel and the device: it holds in the device's other contexts
// and past a reset of the primary one (tests/test_gpu_norm_contexts.py).
template <typename K>
cudaError_t resident(K k, std::atomic<uint64_t> &kept, int threads, size_t smem, int64_t most,
                     int64_t *grid) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  // device (12 bits, + 1 so that no key is zero), threads (11), bytes (20), CTAs (21)
  const uint64_t key = (uint64_t)(dev + 1) << 52 | (uint64_t)threads << 41 | (uint64_t)smem << 21;
  uint64_t word = kept.load(std::memory_order_relaxed);
  if ((word >> 21) != (key >> 21)) {
    // 48 KB with the static arrays need no leave. The same limit in every
    // call: another thread's launch never finds less.
    if (smem > 40 * 1024) {
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
      if (e != cudaSuccess) return e;
    }
    int per_sm = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k, threads, smem);
    if (e != cudaSuccess) return e;
    word = key | (uint64_t)(sm_count() * (per_sm > 0 ? per_sm : 1));
    kept.store(word, std::memory_order_relaxed);
  }
  const int64_t fit = (int64_t)(word & ((1u << 21) - 1));
  *grid = most < fit ? most : fit;
  return cudaSuccess;
}

template <typename T> cudaError_t fwd_t(const RmsNormArgs &a, cudaStream_t s) {
  const int nvec = a.d / Vec<T>::N;
  if (nvec <= 32) return fwd<T, 1, true>(a, 128, s);
  if (nvec <= 64) return fwd<T, 2, true>(a, 128, s);
  if (nvec <= 128) return fwd<T, 4, true>(a, 128, s);
  if (nvec <= 2048) return fwd<T, 2, false>(a, round32((nvec + 1) / 2), s);
  return fwd<T, 4, false>(a, round32((nvec + 3) / 4), s);
}

// A backward kernel on as many clusters of CTAs as fit, and the sum of their
// partial rows.
template <typename K>
cudaError_t bwd(K k, std::atomic<uint64_t> &kept, const RmsNormBwdArgs &a, int threads, int cluster,
                size_t smem, int64_t most, cudaStream_t s) {
  int64_t grid = 0;
  cudaError_t e = resident(k, kept, threads, smem, most * cluster, &grid);
  grid /= cluster;
  if (e == cudaSuccess)
    e = launch_pdl_clusters(k, dim3((unsigned)(grid * cluster)), dim3(threads), cluster, smem, s, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(dgamma_kernel, dim3((a.d + 31) / 32), dim3(1024), 0, s, a.partial, (int)grid, a.d,
                    a.dgamma);
}

template <typename T, typename TY, typename TX, int NU, bool DH>
cudaError_t bwd_warp(const RmsNormBwdArgs &a, cudaStream_t s) {
  static std::atomic<uint64_t> kept{0};
  const int64_t most = rmsnorm_bwd_max_partials((a.rows + kRowWarps - 1) / kRowWarps);
  return bwd(rmsnorm_bwd_warp_kernel<T, TY, TX, NU, DH>, kept, a, kRowWarps * 32, 1, 0, most, s);
}

template <typename T, typename TY, typename TX, bool DH, int STAGES, bool WIDE, bool CLUSTER>
cudaError_t bwd_cta(const RmsNormBwdArgs &a, cudaStream_t s) {
  static std::atomic<uint64_t> kept{0};
  const int cluster = CLUSTER ? kMaxCluster : 1;
  const int threads = round32(((a.d / 4 + cluster - 1) / cluster + 3) / 4);
  const size_t smem = (size_t)STAGES * 4 * threads * bwd_unit_bytes<T, TY>(DH && !WIDE);
  return bwd(rmsnorm_bwd_kernel<T, TY, TX, DH, STAGES, WIDE, CLUSTER>, kept, a, threads, cluster, smem,
             rmsnorm_bwd_max_partials(a.rows), s);
}

template <typename T, typename TY, typename TX, bool DH>
cudaError_t bwd_t(const RmsNormBwdArgs &a, cudaStream_t s) {
  static_assert(2 * kNarrow * bwd_unit_bytes<float, float>(true) / 4 <= kSmem, "two narrow rows fit");
  static_assert(2 * kWide * bwd_unit_bytes<__nv_bfloat16, float>(false) / 4 <= kSmem, "two wide rows fit");
  if (a.d <= 128) return bwd_warp<T, TY, TX, 1, DH>(a, s);
  if (a.d <= 512) return bwd_warp<T, TY, TX, 4, DH>(a, s);
  if (a.d <= kNarrow) {
    const size_t row = (size_t)round32((a.d / 4 + 3) / 4) * 4 * bwd_unit_bytes<T, TY>(DH);
    return a.d > 2048 && 3 * row <= kSmem ? bwd_cta<T, TY, TX, DH, 3, false, false>(a, s)
                                          : bwd_cta<T, TY, TX, DH, 2, false, false>(a, s);
  }
  if constexpr (sizeof(T) == 4) {
    return bwd_cta<T, TY, TX, DH, 2, false, true>(a, s);
  } else {
    return a.d <= kWide ? bwd_cta<T, TY, TX, DH, 2, true, false>(a, s)
                        : bwd_cta<T, TY, TX, DH, 2, true, true>(a, s);
  }
}

template <typename T, typename TY, typename TX>
cudaError_t bwd_dh(const RmsNormBwdArgs &a, cudaStream_t s) {
  return a.dh != nullptr ? bwd_t<T, TY, TX, true>(a, s) : bwd_t<T, TY, TX, false>(a, s);
}

}  // namespace

// Rows of `partial` that the workspace holds, whatever the device's SM count.
int64_t rmsnorm_bwd_max_partials(int64_t rows) { return rows < 1024 ? rows : 1024; }

cudaError_t launch_rmsnorm(const RmsNormArgs &args, cudaStream_t s) {
  RmsNormArgs a = args;
  a.inv_d = 1.0f / (float)a.d;
  a.ng = a.group > 0 ? (a.d + a.group - 1) / a.group : 1;
  a.group_shift = 0;
  while ((a.dtype == MOE_BF16 ? 8 : 4) << a.group_shift < a.group) ++a.group_shift;
  return a.dtype == MOE_BF16 ? fwd_t<__nv_bfloat16>(a, s) : fwd_t<float>(a, s);
}

cudaError_t launch_rmsnorm_bwd(const RmsNormBwdArgs &args, cudaStream_t s) {
  using B = __nv_bfloat16;
  RmsNormBwdArgs a = args;
  a.inv_d = 1.0f / (float)a.d;
  if (a.dtype == MOE_F32) return bwd_dh<float, float, float>(a, s);
  if (a.dy_dtype == MOE_F32)
    return a.dx_dtype == MOE_F32 ? bwd_dh<B, float, float>(a, s) : bwd_dh<B, float, B>(a, s);
  return a.dx_dtype == MOE_F32 ? bwd_dh<B, B, float>(a, s) : bwd_dh<B, B, B>(a, s);
}

}  // namespace moe
