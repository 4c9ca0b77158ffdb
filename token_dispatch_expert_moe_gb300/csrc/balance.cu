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

constexpr int kThreads = 512;      // counting pass
constexpr int kJoinThreads = 256;
constexpr int kBwdThreads = 256;
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

// A token's experts lie over L lanes, V quads (4 consecutive experts) a lane:
// quad v of lane `sub` starts at expert 4 (sub + v L), so that the lanes read
// consecutive 16 bytes. At most 4 lanes: the row's maximum and sum take two
// shuffles each, and a lane's 16 exponentials overlap. (16 lanes with one quad
// each, four shuffles: 55.7 us for 262144 x 64 against the figure below.)
// The softmax of a token's logits: p[4 v + i] of expert 4 (sub + v L) + i,
// zero past E, for a token that is not live, and where all logits are -inf.
template <int L, int V>
__device__ __forceinline__ void softmax_quads(const float *l, int sub, int E, bool live,
                                              float (&p)[4 * V]) {
#pragma unroll
  for (int i = 0; i < 4 * V; ++i) p[i] = -INFINITY;
  if (live) {
    if ((E & 3) == 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = 4 * (sub + v * L);
        if (e < E) {
          const float4 q = *reinterpret_cast<const float4 *>(l + e);
          p[4 * v] = q.x; p[4 * v + 1] = q.y; p[4 * v + 2] = q.z; p[4 * v + 3] = q.w;
        }
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = 4 * (sub + v * L) + i;
          if (e < E) p[4 * v + i] = l[e];
        }
    }
  }
  float m = p[0];
#pragma unroll
  for (int i = 1; i < 4 * V; ++i) m = fmaxf(m, p[i]);
#pragma unroll
  for (int o = L >> 1; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (m == -INFINITY) m = 0.0f;   // nothing left: every p becomes exp(-inf) = 0
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 4 * V; ++i) {
    p[i] = expf(p[i] - m);
    s += p[i];
  }
#pragma unroll
  for (int o = L >> 1; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const float r = s == 0.0f ? 0.0f : __frcp_rn(s);
#pragma unroll
  for (int i = 0; i < 4 * V; ++i) p[i] *= r;
}

// The workspace: partial sums per chunk of tokens, the loss's terms, and the
// number of join CTAs that are done.
struct Partials {
  uint32_t *done;
  int32_t *tokens;   // [chunks in all]: unmasked tokens
  float *term;       // [terms]
  float *prob;       // [chunks in all, E]: sums of p
  int32_t *count;    // [chunks in all, E]
};

// Results of expert e of sub-sequence j; returns c_je P_je.
__device__ __forceinline__ float finish(const BalanceArgs &a, int64_t j, int e, float prob, int c,
                                        int n_j) {
  const float inv = n_j > 0 ? __frcp_rn((float)n_j) : 0.0f;
  const int64_t i = j * a.E + e;
  const float mean = prob * inv;
  a.counts[i] = c;
  if (a.prob_mean != nullptr) a.prob_mean[i] = mean;
  const int64_t over = (int64_t)a.E * c - (int64_t)a.K * n_j;
  a.coef[i] = a.alpha * ((float)over / (float)a.K) * inv;
  return (float)c * mean;
}

template <int L, int V>
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
  if (blockIdx.x == 0 && threadIdx.x == 0) *w.done = 0;
  __syncthreads();
  float acc[4 * V];
#pragma unroll
  for (int i = 0; i < 4 * V; ++i) acc[i] = 0.0f;
  int mine = 0;
  for (int64_t t0 = lo; t0 < hi; t0 += kPer) {   // the same trips for every thread
    const int64_t t = t0 + slot;
    const bool live = t < hi && (a.mask == nullptr || a.mask[t] != 0);
    int e[8 / L];
#pragma unroll
    for (int i = 0; i < 8 / L; ++i) {   // the lanes share out the token's K slots
      const int k = sub + i * L;
      e[i] = live && k < K ? a.topk_idx[t * K + k] : -2;
    }
    float p[4 * V];
    softmax_quads<L, V>(a.logits + t * E, sub, E, live, p);
#pragma unroll
    for (int i = 0; i < 4 * V; ++i) acc[i] += p[i];
    if (live && sub == 0) ++mine;
#pragma unroll
    for (int i = 0; i < 8 / L; ++i) {
      if (e[i] >= 0 && e[i] < E) atomicAdd(&cnt[e[i]], 1);
      else if (live && sub + i * L < K) report(a.status, MOE_ERR_DEVICE, kInfoExpertRange);
    }
  }
  mine = __reduce_add_sync(0xffffffffu, mine);
  if ((threadIdx.x & 31) == 0 && mine > 0) atomicAdd(&tok, mine);
#pragma unroll
  for (int i = 0; i < 4 * V; ++i)
#pragma unroll
    for (int o = 16; o >= L; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane < L)
#pragma unroll
    for (int i = 0; i < 4 * V; ++i) red[warp][4 * (lane + (i / 4) * L) + i % 4] = acc[i];
  __syncthreads();
  pdl_trigger();
  float s = 0.0f;
  if (threadIdx.x < E)
    for (int q = 0; q < kThreads / 32; ++q) s += red[q][threadIdx.x];
  if (threadIdx.x == 0) w.tokens[blockIdx.x] = tok;
  if (chunks > 1) {
    if (threadIdx.x < E) {
      w.prob[(int64_t)blockIdx.x * E + threadIdx.x] = s;
      w.count[(int64_t)blockIdx.x * E + threadIdx.x] = cnt[threadIdx.x];
    }
    return;
  }
  float term = 0.0f;
  if (threadIdx.x < E) term = finish(a, j, threadIdx.x, s, cnt[threadIdx.x], tok);
  term = block_sum(term, &red[0][0]);
  if (threadIdx.x == 0) w.term[j] = term;
}

// Joins the chunks of the sub-sequences (chunks > 1): a CTA takes 16 experts
// of one sub-sequence, 16 threads an expert, and adds their chunks in a fixed
// order. The CTA that finishes last (one CTA alone, when there is nothing to
// join) adds the terms and the token counts, in order again.
constexpr int kJoinExperts = 16, kJoinSlices = kJoinThreads / kJoinExperts;

__global__ void __launch_bounds__(kJoinThreads) balance_join_kernel(BalanceArgs a, Partials w,
                                                                    int64_t chunks, int64_t terms) {
  __shared__ float probs[kJoinSlices][kJoinExperts];
  __shared__ int32_t counts[kJoinSlices][kJoinExperts], tok[kJoinSlices][kJoinExperts];
  __shared__ float red[32];
  __shared__ uint32_t total, before;
  pdl_wait();
  const int E = a.E;
  const int64_t groups = (E + kJoinExperts - 1) / kJoinExperts;
  if (chunks > 1) {
    const int64_t j = blockIdx.x / groups;
    const int x = threadIdx.x % kJoinExperts, slice = threadIdx.x / kJoinExperts;
    const int e = (int)(blockIdx.x - j * groups) * kJoinExperts + x;
    float prob = 0.0f;
    int c = 0, n_j = 0;
    if (e < E) {
#pragma unroll 8
      for (int64_t q = j * chunks + slice; q < (j + 1) * chunks; q += kJoinSlices) {
        prob += w.prob[q * E + e];
        c += w.count[q * E + e];
        n_j += w.tokens[q];
      }
    }
    probs[slice][x] = prob;
    counts[slice][x] = c;
    tok[slice][x] = n_j;
    __syncthreads();
    float term = 0.0f;
    if (slice == 0) {
      for (int q = 1; q < kJoinSlices; ++q) {
        prob += probs[q][x];
        c += counts[q][x];
        n_j += tok[q][x];
      }
      if (e < E) term = finish(a, j, e, prob, c, n_j);
    }
    term = block_sum(term, red);
    if (threadIdx.x == 0) {
      w.term[blockIdx.x] = term;
      __threadfence();
      before = atomicAdd(w.done, 1u);
    }
    __syncthreads();
    if (before != gridDim.x - 1) return;   // the same in every thread
    __threadfence();
  }
  if (threadIdx.x == 0) total = 0;
  __syncthreads();
  float term = 0.0f;
  uint32_t n = 0;   // at most T < 2^31
  const int64_t all = chunks * a.n_sub;
  for (int64_t i = threadIdx.x; i < terms; i += kJoinThreads) term += __ldcg(w.term + i);
  for (int64_t i = threadIdx.x; i < all; i += kJoinThreads) n += w.tokens[i];
  n = __reduce_add_sync(0xffffffffu, n);
  if ((threadIdx.x & 31) == 0) atomicAdd(&total, n);   // whole numbers: the order does not matter
  term = block_sum(term, red);
  if (threadIdx.x == 0) {
    const float inv = total > 0 ? (float)(1.0 / (double)total) : 0.0f;
    a.loss[0] = a.alpha * ((float)E / (float)a.K) * term * inv;
    a.coef[a.n_sub * E] = inv;
  }
}

template <int L, int V>
__global__ void __launch_bounds__(kBwdThreads) balance_bwd_kernel(BalanceArgs a) {
  constexpr int kPer = kBwdThreads / L;
  const int sub = threadIdx.x % L;
  const int64_t t = (int64_t)blockIdx.x * kPer + threadIdx.x / L;
  const int E = a.E;
  const bool in = t < a.T;
  const bool live = in && (a.mask == nullptr || a.mask[t] != 0);
  const float *coef = a.coef + (in ? t / a.S : 0) * E;
  float p[4 * V], w[4 * V], dot = 0.0f;
#pragma unroll
  for (int i = 0; i < 4 * V; ++i) {
    const int e = 4 * (sub + (i / 4) * L) + i % 4;
    w[i] = e < E ? coef[e] : 0.0f;
  }
  softmax_quads<L, V>(a.logits + t * E, sub, E, live, p);
#pragma unroll
  for (int i = 0; i < 4 * V; ++i) dot = fmaf(p[i], w[i], dot);
#pragma unroll
  for (int o = L >> 1; o >= 1; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
  if (!in) return;
  const float g = (a.dloss != nullptr ? a.dloss[0] : 1.0f) * a.coef[a.n_sub * E];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = 4 * (sub + v * L);
    float *out = a.dlogits + t * E + e;
    float o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = live ? g * (p[4 * v + i] * (w[4 * v + i] - dot)) : 0.0f;
    if ((E & 3) == 0) {
      if (e < E) *reinterpret_cast<float4 *>(out) = make_float4(o[0], o[1], o[2], o[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e + i < E) out[i] = o[i];
    }
  }
}

constexpr size_t align256_(size_t v) { return (v + 255) & ~size_t(255); }

// Lanes per token and quads per lane, by the number of experts.
int lanes_of(int E) { return E <= 4 ? 1 : E <= 8 ? 2 : 4; }

struct Regions {
  size_t tokens, term, prob, count, total;
};
Regions regions_of(int64_t T, int64_t S, int E) {
  const Split sp = split_of(T, S, lanes_of(E));
  const int64_t n_sub = (T + S - 1) / S, all = sp.chunks * n_sub;
  const int64_t terms = sp.chunks > 1 ? n_sub * ((E + kJoinExperts - 1) / kJoinExperts) : n_sub;
  const size_t rows = sp.chunks > 1 ? align256_((size_t)all * E * 4) : 0;
  Regions r{};
  r.tokens = 256;
  r.term = r.tokens + align256_((size_t)all * 4);
  r.prob = r.term + align256_((size_t)terms * 4);
  r.count = r.prob + rows;
  r.total = r.count + rows;
  return r;
}

template <int L, int V> cudaError_t fwd(const BalanceArgs &a, cudaStream_t s) {
  const Split sp = split_of(a.T, a.S, L);
  const Regions r = regions_of(a.T, a.S, a.E);
  char *p = static_cast<char *>(a.partial);
  Partials w{};
  w.done = reinterpret_cast<uint32_t *>(p);
  w.tokens = reinterpret_cast<int32_t *>(p + r.tokens);
  w.term = reinterpret_cast<float *>(p + r.term);
  w.prob = reinterpret_cast<float *>(p + r.prob);
  w.count = reinterpret_cast<int32_t *>(p + r.count);
  balance_count_kernel<L, V><<<(unsigned)(sp.chunks * a.n_sub), kThreads, 0, s>>>(a, w, sp.chunks, sp.len);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t joins = sp.chunks > 1 ? a.n_sub * ((a.E + kJoinExperts - 1) / kJoinExperts) : 1;
  const int64_t terms = sp.chunks > 1 ? joins : a.n_sub;
  return launch_pdl(balance_join_kernel, dim3((unsigned)joins), dim3(kJoinThreads), 0, s, a, w,
                    sp.chunks, terms);
}

template <int L, int V> cudaError_t bwd(const BalanceArgs &a, cudaStream_t s) {
  const int64_t per = kBwdThreads / L;
  balance_bwd_kernel<L, V><<<(unsigned)((a.T + per - 1) / per), kBwdThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <bool BWD> cudaError_t by_experts(const BalanceArgs &a, cudaStream_t s) {
  if (a.E <= 4) return BWD ? bwd<1, 1>(a, s) : fwd<1, 1>(a, s);
  if (a.E <= 8) return BWD ? bwd<2, 1>(a, s) : fwd<2, 1>(a, s);
  if (a.E <= 16) return BWD ? bwd<4, 1>(a, s) : fwd<4, 1>(a, s);
  if (a.E <= 32) return BWD ? bwd<4, 2>(a, s) : fwd<4, 2>(a, s);
  return BWD ? bwd<4, 4>(a, s) : fwd<4, 4>(a, s);
}

}  // namespace

size_t balance_workspace_bytes(int64_t T, int64_t S, int E) { return regions_of(T, S, E).total; }

cudaError_t launch_balance_loss(const BalanceArgs &a, cudaStream_t s) { return by_experts<false>(a, s); }
cudaError_t launch_balance_loss_bwd(const BalanceArgs &a, cudaStream_t s) {
  return by_experts<true>(a, s);
}

}  // namespace moe
