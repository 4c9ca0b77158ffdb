// The router's balance loss, the per-expert counts it is made of, and its
// gradient with respect to the logits.
//
// For every sub-sequence j (the blocks of S tokens in which drops are decided
// too) with n_j unmasked tokens, n = sum_j n_j:
//   c_je = number of unmasked (t, k) of the block with topk_idx = e,
//   P_je = mean over the unmasked tokens of p_te, p = softmax(logits),
//   loss = alpha sum_j (n_j / n) sum_e (E c_je / (K n_j)) P_je.
// The counts carry no gradient. A constant added to every expert's factor
// falls out of the softmax's gradient, so the backward uses the load's
// deviation from its mean,
//   a_je = alpha (E c_je - K n_j) / (K n_j)   (the integer part is exact),
//   dl_te = (dloss / n) p_te (a_je - sum_i p_ti a_ji):
// nothing cancels when the load is nearly even. Sums are fp32, counts are
// integers, every order is fixed.
#include "launch.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
// CTAs of the counting pass when sub-sequences are cut into chunks.
constexpr int64_t kTargetCtas = 304;

struct Split {
  int64_t chunks, len;   // chunks per sub-sequence and tokens per chunk
};
Split split_of(int64_t T, int64_t S, int lanes) {
  const int64_t n_sub = (T + S - 1) / S;
  const int64_t step = kThreads / lanes;   // tokens a CTA takes at once
  int64_t chunks = kTargetCtas / n_sub;
  const int64_t most = (S + step - 1) / step;
  if (chunks > most) chunks = most;
  if (chunks < 1) chunks = 1;
  Split r;
  r.len = (S + chunks - 1) / chunks;
  r.chunks = (S + r.len - 1) / r.len;
  return r;
}

// Lanes per token: each holds 4 consecutive experts.
int lanes_of(int E) {
  int l = 1;
  while (4 * l < E) l *= 2;
  return l;
}

// The softmax of a token's logits over its L lanes: p[i] of experts
// 4 * sub + i, zero past E and for a token whose logits are all -inf.
template <int L>
__device__ __forceinline__ void softmax4(const float *l, int sub, int E, bool live, float (&p)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = -INFINITY;
  if (live) {
    if ((E & 3) == 0) {
      if (4 * sub < E) {
        const float4 v = *reinterpret_cast<const float4 *>(l + 4 * sub);
        p[0] = v.x; p[1] = v.y; p[2] = v.z; p[3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * sub + i < E) p[i] = l[4 * sub + i];
    }
  }
  float m = fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3]));
#pragma unroll
  for (int o = L >> 1; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (m == -INFINITY) m = 0.0f;   // nothing left: every p becomes exp(-inf) = 0
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p[i] = expf(p[i] - m);
    s += p[i];
  }
#pragma unroll
  for (int o = L >> 1; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const float r = s == 0.0f ? 0.0f : __frcp_rn(s);
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] *= r;
}

// Partial sums of one chunk of tokens: P sums, counts and unmasked tokens.
struct Partials {
  float *prob;       // [blocks, E]
  int32_t *count;    // [blocks, E]
  int32_t *tokens;   // [blocks]
  float *term;       // [n_sub]: the loss's terms, when a block is a sub-sequence
};

// A block that holds a whole sub-sequence's sums writes its results; returns
// sum_e c_e P_e / n_j over the calling warp.
__device__ __forceinline__ float finish(const BalanceArgs &a, int64_t j, int e, float prob, int c,
                                        int n_j) {
  const float inv = n_j > 0 ? __frcp_rn((float)n_j) : 0.0f;
  const int64_t i = j * a.E + e;
  a.counts[i] = c;
  if (a.prob_mean != nullptr) a.prob_mean[i] = n_j > 0 ? __fdiv_rn(prob, (float)n_j) : 0.0f;
  const int64_t over = (int64_t)a.E * c - (int64_t)a.K * n_j;
  a.coef[i] = a.alpha * ((float)over / (float)a.K) * inv;
  return (float)c * (prob * inv);
}

template <int L>
__global__ void __launch_bounds__(kThreads) balance_count_kernel(BalanceArgs a, Partials w,
                                                                 int64_t chunks, int64_t len) {
  __shared__ int32_t cnt[64];
  __shared__ int32_t tok;
  __shared__ float red[kThreads / 32][64];
  constexpr int kPer = kThreads / L;
  const int64_t j = blockIdx.x / chunks, c = blockIdx.x - j * chunks;
  const int64_t lo = j * a.S + c * len;
  const int64_t hi = min(min(a.T, (j + 1) * a.S), lo + len);
  const int sub = threadIdx.x % L, slot = threadIdx.x / L;
  const int E = a.E, K = a.K;
  if (threadIdx.x < 64) cnt[threadIdx.x] = 0;
  if (threadIdx.x == 0) tok = 0;
  __syncthreads();
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  int mine = 0;
  for (int64_t t0 = lo; t0 < hi; t0 += kPer) {   // the same trips for every thread
    const int64_t t = t0 + slot;
    const bool live = t < hi && (a.mask == nullptr || a.mask[t] != 0);
    float p[4];
    softmax4<L>(a.logits + t * E, sub, E, live, p);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] += p[i];
    if (live) {
      if (sub == 0) ++mine;
      for (int k = sub; k < K; k += L) {
        const int e = a.topk_idx[t * K + k];
        if (e >= 0 && e < E) atomicAdd(&cnt[e], 1);
        else report(a.status, MOE_ERR_DEVICE, kInfoExpertRange);
      }
    }
  }
  if (mine > 0) atomicAdd(&tok, mine);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int o = 16; o >= L; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane < L)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[warp][4 * lane + i] = acc[i];
  __syncthreads();
  pdl_trigger();
  float s = 0.0f;
  if (threadIdx.x < E)
    for (int q = 0; q < kThreads / 32; ++q) s += red[q][threadIdx.x];
  if (chunks > 1) {
    if (threadIdx.x < E) {
      w.prob[(int64_t)blockIdx.x * E + threadIdx.x] = s;
      w.count[(int64_t)blockIdx.x * E + threadIdx.x] = cnt[threadIdx.x];
    }
    if (threadIdx.x == 0) w.tokens[blockIdx.x] = tok;
    return;
  }
  float term = 0.0f;
  if (threadIdx.x < E) term = finish(a, j, threadIdx.x, s, cnt[threadIdx.x], tok);
  term = block_sum(term, &red[0][0]);
  if (threadIdx.x == 0) {
    w.term[j] = term;
    w.tokens[j] = tok;
  }
}

// One CTA: joins the chunks of every sub-sequence in order (chunks > 1), and
// adds the sub-sequences' terms: loss and 1 / n.
__global__ void __launch_bounds__(1024) balance_join_kernel(BalanceArgs a, Partials w, int64_t chunks) {
  __shared__ float red[32];
  __shared__ unsigned long long total;
  if (threadIdx.x == 0) total = 0;
  pdl_wait();
  __syncthreads();
  const int E = a.E;
  float term = 0.0f;
  unsigned long long n = 0;
  if (chunks > 1) {
    for (int64_t i = threadIdx.x; i < a.n_sub * E; i += blockDim.x) {
      const int64_t j = i / E;
      const int e = (int)(i - j * E);
      float prob = 0.0f;
      int c = 0, n_j = 0;
      for (int64_t q = j * chunks; q < (j + 1) * chunks; ++q) {
        prob += w.prob[q * E + e];
        c += w.count[q * E + e];
        n_j += w.tokens[q];
      }
      term += finish(a, j, e, prob, c, n_j);
      if (e == 0) n += n_j;
    }
  } else {
    for (int64_t j = threadIdx.x; j < a.n_sub; j += blockDim.x) {
      term += w.term[j];
      n += w.tokens[j];
    }
  }
  if (n > 0) atomicAdd(&total, n);   // whole numbers: the order does not matter
  term = block_sum(term, red);
  if (threadIdx.x == 0) {
    const float inv = total > 0 ? (float)(1.0 / (double)total) : 0.0f;
    a.loss[0] = a.alpha * ((float)E / (float)a.K) * term * inv;
    a.coef[a.n_sub * E] = inv;
  }
}

template <int L>
__global__ void __launch_bounds__(kThreads) balance_bwd_kernel(BalanceArgs a) {
  constexpr int kPer = kThreads / L;
  const int sub = threadIdx.x % L;
  const int64_t t = (int64_t)blockIdx.x * kPer + threadIdx.x / L;
  const int E = a.E;
  const bool in = t < a.T;
  const bool live = in && (a.mask == nullptr || a.mask[t] != 0);
  float p[4], w[4], dot = 0.0f;
  softmax4<L>(a.logits + t * E, sub, E, live, p);
  const float *coef = a.coef + (in ? t / a.S : 0) * E;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = 4 * sub + i < E ? coef[4 * sub + i] : 0.0f;
    dot = fmaf(p[i], w[i], dot);
  }
#pragma unroll
  for (int o = L >> 1; o >= 1; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
  if (!in) return;
  const float g = (a.dloss != nullptr ? a.dloss[0] : 1.0f) * a.coef[a.n_sub * E];
  float *out = a.dlogits + t * E + 4 * sub;
  float o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = live ? g * (p[i] * (w[i] - dot)) : 0.0f;
  if ((E & 3) == 0) {
    if (4 * sub < E) *reinterpret_cast<float4 *>(out) = make_float4(o[0], o[1], o[2], o[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * sub + i < E) out[i] = o[i];
  }
}

constexpr size_t align256_(size_t v) { return (v + 255) & ~size_t(255); }

template <int L> cudaError_t fwd(const BalanceArgs &a, cudaStream_t s) {
  const Split sp = split_of(a.T, a.S, L);
  const int64_t blocks = sp.chunks * a.n_sub;
  Partials w{};
  char *p = static_cast<char *>(a.partial);
  w.tokens = reinterpret_cast<int32_t *>(p);
  p += align256_((size_t)blocks * 4);
  w.term = reinterpret_cast<float *>(p);
  w.prob = reinterpret_cast<float *>(p);
  w.count = reinterpret_cast<int32_t *>(p + align256_((size_t)blocks * a.E * 4));
  balance_count_kernel<L><<<(unsigned)blocks, kThreads, 0, s>>>(a, w, sp.chunks, sp.len);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_pdl(balance_join_kernel, dim3(1), dim3(1024), 0, s, a, w, sp.chunks);
}

template <int L> cudaError_t bwd(const BalanceArgs &a, cudaStream_t s) {
  const int64_t per = kThreads / L;
  balance_bwd_kernel<L><<<(unsigned)((a.T + per - 1) / per), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <bool BWD> cudaError_t by_lanes(const BalanceArgs &a, cudaStream_t s) {
  switch (lanes_of(a.E)) {
    case 1: return BWD ? bwd<1>(a, s) : fwd<1>(a, s);
    case 2: return BWD ? bwd<2>(a, s) : fwd<2>(a, s);
    case 4: return BWD ? bwd<4>(a, s) : fwd<4>(a, s);
    case 8: return BWD ? bwd<8>(a, s) : fwd<8>(a, s);
    default: return BWD ? bwd<16>(a, s) : fwd<16>(a, s);
  }
}

}  // namespace

size_t balance_workspace_bytes(int64_t T, int64_t S, int E) {
  const Split sp = split_of(T, S, lanes_of(E));
  const int64_t n_sub = (T + S - 1) / S, blocks = sp.chunks * n_sub;
  if (sp.chunks == 1) return align256_((size_t)blocks * 4) * 2;
  return align256_((size_t)blocks * 4) + align256_((size_t)blocks * E * 4) * 2;
}

cudaError_t launch_balance_loss(const BalanceArgs &a, cudaStream_t s) { return by_lanes<false>(a, s); }
cudaError_t launch_balance_loss_bwd(const BalanceArgs &a, cudaStream_t s) {
  return by_lanes<true>(a, s);
}

}  // namespace moe
