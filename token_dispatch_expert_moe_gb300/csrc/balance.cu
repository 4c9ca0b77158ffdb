// The router's balance loss, the per-expert counts it is made of, and its
// gradient with respect to the logits. Small calls are launch latency (512 x
// 4: 3.0 us and 1.6 us), 16384 x 64 in 4 sub-sequences takes 7.4 and 2.7 us.
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
#include <cooperative_groups.h>

#include "launch.cuh"

namespace moe {
namespace {

constexpr int kJoinThreads = 512, kJoinCtas = 8;   // one cluster
constexpr int kBwdThreads = 128;

// How the counting pass cuts the tokens. A sub-sequence that one CTA gets
// through in a few tokens a thread stays whole and needs no joining (a join
// adds 3 to 4 us); others are cut into chunks, two CTAs for each of 152 SMs
// in all.
constexpr int kMaxThreads = 512;
constexpr int kFewTokens = 8;            // a thread, of a whole sub-sequence
constexpr int kChunkThreads = 256;
constexpr int64_t kTargetCtas = 304;

struct Split {
  int64_t chunks, len;   // chunks per sub-sequence and tokens per chunk
  int threads;
};
Split split_of(int64_t T, int64_t S, int lanes) {
  const int64_t n_sub = (T + S - 1) / S;
  Split r;
  if (S * lanes <= kMaxThreads * kFewTokens || n_sub >= kTargetCtas) {
    r.chunks = 1;
    r.len = S;
    // few CTAs: as many threads as have a token; many: fewer, longer ones
    const int64_t want = n_sub <= 152 ? S * lanes : (S * lanes + kFewTokens - 1) / kFewTokens;
    r.threads = want <= 128 ? 128 : want <= 256 ? 256 : kMaxThreads;
    return r;
  }
  const int64_t step = kChunkThreads / lanes;   // tokens a CTA takes at once
  int64_t chunks = kTargetCtas / n_sub;
  const int64_t most = (S + step - 1) / step;
  if (chunks > most) chunks = most;
  if (chunks < 1) chunks = 1;
  r.len = (S + chunks - 1) / chunks;
  r.chunks = (S + r.len - 1) / r.len;
  r.threads = kChunkThreads;
  return r;
}

// A token's experts lie over L lanes, V quads (4 consecutive experts) a lane:
// quad v of lane `sub` starts at expert 4 (sub + v L), so that the lanes read
// consecutive 16 bytes. At most 4 lanes: the row's maximum and sum take two
// shuffles each, and a lane's 16 exponentials overlap (262144 x 64, loss and
// gradient: 16.5 and 20.7 us; 8 lanes of two quads 20.6 and 23.4 us, 16 lanes
// of one 31.1 and 29.4 us). Their bytes take 11.1 and 19.8 us: the gradient is
// bound by HBM, the loss waits for latency, with 16 warps an SM (98 registers),
// half the issue slots and two thirds of the bandwidth in use; logits fetched
// two tokens ahead through shared memory took 10 % more.

// A row of E values, l[4 v + i] of expert 4 (sub + v L) + i: `none` past E, and
// throughout where `in` is false (nothing is read then).
template <int L, int V>
__device__ __forceinline__ void load_quads(const float *row, int sub, int E, bool in, float none,
                                           float (&l)[4 * V]) {
#pragma unroll
  for (int i = 0; i < 4 * V; ++i) l[i] = none;
  if (!in) return;
  if ((E & 3) == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = 4 * (sub + v * L);
      if (e < E) {
        const float4 q = *reinterpret_cast<const float4 *>(row + e);
        l[4 * v] = q.x; l[4 * v + 1] = q.y; l[4 * v + 2] = q.z; l[4 * v + 3] = q.w;
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = 4 * (sub + v * L) + i;
        if (e < E) l[4 * v + i] = row[e];
      }
  }
}

__device__ __forceinline__ float exp2_of(float v) {   // within 2 ulp; below 2^-126: 0
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// The softmax numerators in place of the token's logits; returns the factor
// that makes them probabilities. All zero where every logit is -inf.
template <int L, int V> __device__ __forceinline__ float softmax_quads(float (&p)[4 * V]) {
  float m = p[0];
#pragma unroll
  for (int i = 1; i < 4 * V; ++i) m = fmaxf(m, p[i]);
#pragma unroll
  for (int o = L >> 1; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (m == -INFINITY) m = 0.0f;   // nothing left: every p becomes exp(-inf) = 0
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 4 * V; ++i) {
    // the distance first: lowest values and far logits neither overflow nor
    // cancel; two more roundings of it put |l - m| 2^-23 on p
    p[i] = exp2_of((p[i] - m) * 1.4426950408889634f);
    s += p[i];
  }
#pragma unroll
  for (int o = L >> 1; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s == 0.0f ? 0.0f : __frcp_rn(s);
}

// The workspace: partial sums per chunk of tokens, and the loss's term of each
// sub-sequence that is not cut.
struct Partials {
  int32_t *tokens;   // [chunks in all]: unmasked tokens
  float *term;       // [n_sub]
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

__device__ __forceinline__ void finish_loss(const BalanceArgs &a, float terms, uint32_t n) {
  const float inv = n > 0 ? __frcp_rn((float)n) : 0.0f;
  a.loss[0] = a.alpha * ((float)a.E / (float)a.K) * terms * inv;
  a.coef[a.n_sub * a.E] = inv;
}

template <int L, int V>
__global__ void __launch_bounds__(kMaxThreads) balance_count_kernel(BalanceArgs a, Partials w,
                                                                 int64_t chunks, int64_t len) {
  __shared__ int32_t cnt[64];
  __shared__ int32_t tok;
  __shared__ float red[kMaxThreads / 32][64];
  const int kPer = blockDim.x / L;
  const int64_t j = blockIdx.x / chunks, c = blockIdx.x - j * chunks;
  const int64_t lo = j * a.S + c * len;
  const int64_t hi = min(min(a.T, (j + 1) * a.S), lo + len);
  const int sub = threadIdx.x % L, slot = threadIdx.x / L;
  const int E = a.E, K = a.K;
  if (threadIdx.x < 64) cnt[threadIdx.x] = 0;
  if (threadIdx.x == 0) tok = 0;
  pdl_wait();
  __syncthreads();
  float acc[4 * V], next[4 * V];
#pragma unroll
  for (int i = 0; i < 4 * V; ++i) acc[i] = 0.0f;
  int mine = 0;
  // The next token's logits, indices and mask are on their way while one is
  // worked on. A masked token's logits are read and thrown away.
  constexpr int kSlots = 8 / L;   // the lanes share out the token's K slots
  int idx[kSlots], keep = 0;
  auto fetch = [&](int64_t t) {
    const bool in = t < hi;
    load_quads<L, V>(a.logits + t * E, sub, E, in, -INFINITY, next);
    keep = in && (a.mask == nullptr || a.mask[t] != 0);
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const int k = sub + i * L;
      idx[i] = in && k < K ? a.topk_idx[t * K + k] : 0;
    }
  };
  fetch(lo + slot);
  for (int64_t t0 = lo; t0 < hi; t0 += kPer) {   // the same trips for every thread
    float p[4 * V];
    int e[kSlots];
    const bool live = keep != 0;
#pragma unroll
    for (int i = 0; i < 4 * V; ++i) p[i] = next[i];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) e[i] = idx[i];
    fetch(t0 + kPer + slot);
    const float r = softmax_quads<L, V>(p);
    if (live) {
#pragma unroll
      for (int i = 0; i < 4 * V; ++i) acc[i] = fmaf(p[i], r, acc[i]);
      if (sub == 0) ++mine;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        if (sub + i * L >= K) continue;
        if (e[i] >= 0 && e[i] < E) atomicAdd(&cnt[e[i]], 1);
        else report(a.status, MOE_ERR_DEVICE, kInfoExpertRange);
      }
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
  float s = 0.0f;
  if (threadIdx.x < E)
    for (int q = 0; q < (int)(blockDim.x >> 5); ++q) s += red[q][threadIdx.x];
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
  if (threadIdx.x != 0) return;
  if (a.n_sub == 1) finish_loss(a, term, (uint32_t)tok);   // this CTA saw every token
  else w.term[j] = term;
}

// Joins the chunks of the sub-sequences (chunks > 1), then the sub-sequences'
// terms and token counts. One cluster of CTAs, so that the last step is an
// exchange of shared memory and not another trip through global memory: every
// such trip is 0.8 us, and this kernel is nothing else. The (sub-sequence,
// expert) pairs lie over the cluster; `slices` threads share out the chunks of
// a pair. Everything is added in a fixed order.
__global__ void __cluster_dims__(kJoinCtas, 1, 1) __launch_bounds__(kJoinThreads)
balance_join_kernel(BalanceArgs a, Partials w, int64_t chunks, int slices) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ float probs[kJoinThreads];
  __shared__ int32_t counts[kJoinThreads], toks[kJoinThreads];
  __shared__ float red[32];
  __shared__ uint32_t total;
  __shared__ float all_terms[kJoinCtas];
  __shared__ uint32_t all_tokens[kJoinCtas];
  if (threadIdx.x == 0) total = 0;
  const int rank = (int)cluster.block_rank();
  const int E = a.E;
  pdl_wait();
  cluster.sync();   // all CTAs run: the first one's shared memory may be written
  uint32_t n = 0;   // at most T < 2^31
  for (int64_t i = rank * kJoinThreads + threadIdx.x; i < chunks * a.n_sub; i += kJoinCtas * kJoinThreads)
    n += w.tokens[i];
  float term = 0.0f;
  if (chunks > 1) {
    const int per = kJoinThreads / slices;   // pairs of a CTA at once
    const int x = threadIdx.x % per, slice = threadIdx.x / per;
    const int64_t pairs = a.n_sub * E;
    for (int64_t p0 = (int64_t)rank * per; p0 < pairs; p0 += kJoinCtas * per) {   // the same in every thread
      const int64_t pair = p0 + x;
      const int64_t j = pair / E;
      const int e = (int)(pair - j * E);
      float prob = 0.0f;
      int c = 0, n_j = 0;
      if (pair < pairs) {
#pragma unroll 8
        for (int q = slice; q < (int)chunks; q += slices) {
          const int64_t row = j * chunks + q;
          prob += w.prob[row * E + e];
          c += w.count[row * E + e];
          n_j += w.tokens[row];
        }
      }
      probs[threadIdx.x] = prob;
      counts[threadIdx.x] = c;
      toks[threadIdx.x] = n_j;
      __syncthreads();
      if (slice == 0 && pair < pairs) {
        for (int q = 1; q < slices; ++q) {
          prob += probs[q * per + x];
          c += counts[q * per + x];
          n_j += toks[q * per + x];
        }
        term += finish(a, j, e, prob, c, n_j);
      }
      __syncthreads();
    }
  } else {
    for (int64_t i = rank * kJoinThreads + threadIdx.x; i < a.n_sub; i += kJoinCtas * kJoinThreads)
      term += w.term[i];
  }
  n = __reduce_add_sync(0xffffffffu, n);
  if ((threadIdx.x & 31) == 0 && n > 0) atomicAdd(&total, n);   // whole numbers: the order does not matter
  term = block_sum(term, red);
  if (threadIdx.x == 0) {
    *cluster.map_shared_rank(&all_terms[rank], 0) = term;
    *cluster.map_shared_rank(&all_tokens[rank], 0) = total;
  }
  cluster.sync();
  if (rank == 0 && threadIdx.x == 0) {
    term = 0.0f;
    n = 0;
    for (int r = 0; r < kJoinCtas; ++r) {
      term += all_terms[r];
      n += all_tokens[r];
    }
    finish_loss(a, term, n);
  }
}

template <int L, int V>
__global__ void __launch_bounds__(kBwdThreads) balance_bwd_kernel(BalanceArgs a) {
  constexpr int kPer = kBwdThreads / L;
  pdl_wait();
  const int sub = threadIdx.x % L;
  const int64_t t = (int64_t)blockIdx.x * kPer + threadIdx.x / L;
  const int E = a.E;
  const bool in = t < a.T;
  const bool live = in && (a.mask == nullptr || a.mask[t] != 0);
  // T and S fit in 32 bits; coef has the alignment of logits, so its rows too
  const float *coef = a.coef + (int64_t)(in ? (uint32_t)t / (uint32_t)a.S : 0) * E;
  float p[4 * V], w[4 * V], dot = 0.0f;
  load_quads<L, V>(coef, sub, E, true, 0.0f, w);
  load_quads<L, V>(a.logits + t * E, sub, E, live, -INFINITY, p);
  const float r = softmax_quads<L, V>(p);
#pragma unroll
  for (int i = 0; i < 4 * V; ++i) {
    p[i] *= r;
    dot = fmaf(p[i], w[i], dot);
  }
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
  size_t term, prob, count, total;   // tokens come first
};
Regions regions_of(int64_t T, int64_t S, int E) {
  const Split sp = split_of(T, S, lanes_of(E));
  const int64_t n_sub = (T + S - 1) / S, all = sp.chunks * n_sub;
  const size_t rows = sp.chunks > 1 ? align256_((size_t)all * E * 4) : 0;
  Regions r{};
  r.term = align256_((size_t)all * 4);
  r.prob = r.term + align256_((size_t)n_sub * 4);
  r.count = r.prob + rows;
  r.total = r.count + rows;
  return r;
}

template <int L, int V> cudaError_t fwd(const BalanceArgs &a, cudaStream_t s) {
  const Split sp = split_of(a.T, a.S, L);
  const Regions r = regions_of(a.T, a.S, a.E);
  char *p = static_cast<char *>(a.partial);
  Partials w{};
  w.tokens = reinterpret_cast<int32_t *>(p);
  w.term = reinterpret_cast<float *>(p + r.term);
  w.prob = reinterpret_cast<float *>(p + r.prob);
  w.count = reinterpret_cast<int32_t *>(p + r.count);
  cudaError_t e = launch_pdl(balance_count_kernel<L, V>, dim3((unsigned)(sp.chunks * a.n_sub)),
                             dim3(sp.threads), 0, s, a, w, sp.chunks, sp.len);
  if (e != cudaSuccess || sp.chunks * a.n_sub == 1) return e;
  // threads a pair: as many as fill the cluster, no more than chunks
  int slices = 1;
  while (2 * slices * a.n_sub * a.E <= kJoinCtas * kJoinThreads && 2 * slices <= sp.chunks && slices < 32)
    slices *= 2;
  return launch_pdl(balance_join_kernel, dim3(kJoinCtas), dim3(kJoinThreads), 0, s, a, w, sp.chunks, slices);
}

template <int L, int V> cudaError_t bwd(const BalanceArgs &a, cudaStream_t s) {
  const int64_t per = kBwdThreads / L;
  return launch_pdl(balance_bwd_kernel<L, V>, dim3((unsigned)((a.T + per - 1) / per)),
                    dim3(kBwdThreads), 0, s, a);
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
