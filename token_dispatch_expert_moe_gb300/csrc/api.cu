// C ABI of libmoe.so: argument checks, workspace layout, kernel launches.
// The operations and their sources are documented in include/moe.h.
// Every call that launches work opens an NVTX range named after itself, so
// profilers that record NVTX show where each layer step starts and ends
// (without a profiler attached the range calls return at once).
#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>

#include <nvtx3/nvToolsExt.h>

#include "common.cuh"

using namespace moe;

namespace {

struct NvtxRange {
  explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange &) = delete;
  NvtxRange &operator=(const NvtxRange &) = delete;
};

constexpr size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool overlap(const void *p, size_t np, const void *q, size_t nq) {
  if (p == nullptr || q == nullptr) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + nq && b < a + np;
}

struct Span {
  const void *p;
  size_t n;
};

// Whether one of the buffers that a call writes shares memory with another of
// them or with one that it reads. NULL shares none.
template <size_t W, size_t R>
bool any_overlap(const Span (&written)[W], const Span (&read)[R]) {
  for (size_t i = 0; i < W; ++i) {
    for (size_t j = i + 1; j < W; ++j)
      if (overlap(written[i].p, written[i].n, written[j].p, written[j].n)) return true;
    for (size_t j = 0; j < R; ++j)
      if (overlap(written[i].p, written[i].n, read[j].p, read[j].n)) return true;
  }
  return false;
}

bool shape_ok(const moe_shape_t *s) {
  if (s == nullptr) return false;
  if (s->T < 1 || s->d < 1 || s->E < 1 || s->E > 64 || s->K < 1 || s->K > 8 || s->K > s->E)
    return false;
  if (s->F < 1 || (s->dtype != MOE_F32 && s->dtype != MOE_BF16)) return false;
  if (s->drop != 0 && s->drop != 1) return false;
  if (s->drop && !(s->capacity_factor > 0.0f)) return false;
  if (s->subseq_len < 0 || (s->renorm != 0 && s->renorm != 1) || s->Fs < 0) return false;
  if (s->T * (int64_t)s->K >= (int64_t(1) << 31)) return false;  // int32 row indices
  if (s->d % (s->dtype == MOE_BF16 ? 8 : 4) != 0) return false;
  return true;
}

int64_t subseq(const moe_shape_t *s) {
  return (s->subseq_len > 0 && s->subseq_len < s->T) ? s->subseq_len : s->T;
}

struct Layout {
  size_t status, map, cap, capn, rbwd, bal, total;
};

// the tensor-core router's logits path (bf16, d % 64 == 0)
bool router_on_tensor_cores(const moe_shape_t *s) {
  return s->dtype == MOE_BF16 && s->d % 64 == 0;
}

Layout layout(const moe_shape_t *s) {
  Layout L{};
  size_t off = kStatusBytes;
  L.status = 0;
  L.map = off;
  off += align256((size_t)((s->T + 255) / 256) * s->E * sizeof(int32_t));
  L.cap = off;
  L.capn = off;
  if (s->drop) {
    const int64_t S = subseq(s);
    const int64_t n_sub = (s->T + S - 1) / S;
    off += align256((size_t)n_sub * s->E * S * sizeof(unsigned long long));
    L.capn = off;
    off += align256((size_t)n_sub * s->E * sizeof(uint32_t));
  }
  L.rbwd = off;
  off += align256(route_bwd_workspace_bytes(s->T, s->d, s->E));
  L.bal = off;
  off += align256(balance_workspace_bytes(s->T, subseq(s), s->E));
  L.total = off > MOE_FFN_BWD_WORKSPACE_BYTES ? off : MOE_FFN_BWD_WORKSPACE_BYTES;
  return L;
}

moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

uint32_t *status_word(void *ws) { return reinterpret_cast<uint32_t *>(ws); }

RouteArgs route_args(const moe_shape_t *s, void *ws) {
  RouteArgs a{};
  const Layout L = layout(s);
  a.T = s->T; a.d = s->d; a.E = s->E; a.K = s->K; a.dtype = s->dtype;
  a.renorm = s->renorm; a.drop = s->drop; a.S = subseq(s); a.cf = s->capacity_factor;
  a.status = status_word(ws);
  a.cap_keys = reinterpret_cast<unsigned long long *>(static_cast<char *>(ws) + L.cap);
  a.cap_counts = reinterpret_cast<uint32_t *>(static_cast<char *>(ws) + L.capn);
  return a;
}

// capacity dropping: the candidate list lengths start at zero (a memset
// ahead of the call's kernels keeps the kernels' dependent-launch chain whole)
cudaError_t clear_capacity_counts(const moe_shape_t *s, const RouteArgs &a, cudaStream_t st) {
  if (!s->drop) return cudaSuccess;
  const int64_t S = subseq(s);
  const int64_t n_sub = (s->T + S - 1) / S;
  return cudaMemsetAsync(a.cap_counts, 0, (size_t)n_sub * s->E * sizeof(uint32_t), st);
}

}  // namespace

extern "C" {

const char *moe_version(void) { return "0.1.0"; }

const char *moe_status_string(moe_status_t s) {
  switch (s) {
    case MOE_OK: return "ok";
    case MOE_ERR_INVALID_ARG: return "invalid argument";
    case MOE_ERR_UNSUPPORTED: return "unsupported shape";
    case MOE_ERR_CUDA: return "CUDA error";
    case MOE_ERR_TIMEOUT: return "device wait timed out";
    case MOE_ERR_DEVICE: return "device-side check failed";
  }
  return "unknown status";
}

size_t moe_workspace_size(const moe_shape_t *shape) {
  if (!shape_ok(shape)) return 0;
  return layout(shape).total;
}

moe_status_t moe_clear_status(void *ws, moe_stream_t stream) {
  if (ws == nullptr || !aligned16(ws)) return MOE_ERR_INVALID_ARG;
  return cuda_status(cudaMemsetAsync(ws, 0, 2 * sizeof(uint32_t), (cudaStream_t)stream));
}

moe_status_t moe_get_status(void *ws, moe_stream_t stream, uint32_t *info) {
  if (ws == nullptr || !aligned16(ws)) return MOE_ERR_INVALID_ARG;
  uint32_t h[2] = {0, 0};
  if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return MOE_ERR_CUDA;
  if (cudaMemcpy(h, ws, sizeof(h), cudaMemcpyDeviceToHost) != cudaSuccess) return MOE_ERR_CUDA;
  if (info != nullptr) *info = h[1];
  return (moe_status_t)h[0];
}

moe_status_t moe_route(const moe_shape_t *shape, const void *x, const void *W_r, const float *b_r,
                       const void *w_sg, float *logits, float *gate_logit, int32_t *topk_idx,
                       float *topk_prob, float *topk_w, uint8_t *keep, void *ws,
                       moe_stream_t stream) {
  NvtxRange trace("moe_route");
  if (!shape_ok(shape)) return MOE_ERR_INVALID_ARG;
  if (!x || !W_r || !logits || !topk_idx || !topk_prob || !topk_w || !keep || !ws)
    return MOE_ERR_INVALID_ARG;
  if ((w_sg == nullptr) != (gate_logit == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(W_r) || !aligned16(ws) || !aligned4(logits)) return MOE_ERR_INVALID_ARG;
  if (shape->drop && subseq(shape) >= (int64_t(1) << 29)) return MOE_ERR_UNSUPPORTED;
  RouteArgs a = route_args(shape, ws);
  a.x = x; a.W_r = W_r; a.b_r = b_r; a.w_sg = w_sg; a.logits = logits; a.gate_logit = gate_logit;
  a.topk_idx = topk_idx; a.topk_prob = topk_prob; a.topk_w = topk_w; a.keep = keep;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = clear_capacity_counts(shape, a, s);
  if (e != cudaSuccess) return cuda_status(e);
  if (router_on_tensor_cores(shape) && (w_sg == nullptr || aligned16(w_sg))) {
    // logits on the tensor cores; softmax, Top-K and weights in its epilogue
    // (few experts) or in the Top-K kernel
    e = launch_router_tc(a, s);
    if (e == cudaSuccess && !router_routes_in_epilogue(shape->T, shape->d, shape->E, w_sg != nullptr))
      e = launch_topk_from_logits(a, s);
  } else {
    e = launch_router_fused(a, s);
  }
  if (e == cudaSuccess && shape->drop) e = launch_capacity(a, s);
  return cuda_status(e);
}

moe_status_t moe_route_topk(const moe_shape_t *shape, const float *logits, int32_t *topk_idx,
                            float *topk_prob, float *topk_w, uint8_t *keep, void *ws,
                            moe_stream_t stream) {
  NvtxRange trace("moe_route_topk");
  if (!shape_ok(shape)) return MOE_ERR_INVALID_ARG;
  if (!logits || !topk_idx || !topk_prob || !topk_w || !keep || !ws || !aligned16(ws))
    return MOE_ERR_INVALID_ARG;
  if (shape->drop && subseq(shape) >= (int64_t(1) << 29)) return MOE_ERR_UNSUPPORTED;
  RouteArgs a = route_args(shape, ws);
  a.logits = const_cast<float *>(logits);
  a.topk_idx = topk_idx; a.topk_prob = topk_prob; a.topk_w = topk_w; a.keep = keep;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = clear_capacity_counts(shape, a, s);
  if (e == cudaSuccess) e = launch_topk_from_logits(a, s);
  if (e == cudaSuccess && shape->drop) e = launch_capacity(a, s);
  return cuda_status(e);
}

moe_status_t moe_permute(const moe_shape_t *shape, const void *x, const int32_t *topk_idx,
                         const uint8_t *keep, void *Xp, int32_t *row_of, int32_t *src_of,
                         int32_t *counts, int32_t *offsets, void *ws, moe_stream_t stream) {
  NvtxRange trace("moe_permute");
  if (!shape_ok(shape)) return MOE_ERR_INVALID_ARG;
  if (!x || !topk_idx || !keep || !row_of || !src_of || !counts || !offsets || !ws)
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || (Xp && !aligned16(Xp)) || !aligned16(ws)) return MOE_ERR_INVALID_ARG;
  PermuteArgs a{};
  a.T = shape->T; a.d = shape->d; a.E = shape->E; a.K = shape->K; a.dtype = shape->dtype;
  a.x = x; a.topk_idx = topk_idx; a.keep = keep; a.Xp = Xp; a.row_of = row_of; a.src_of = src_of;
  a.counts = counts; a.offsets = offsets;
  a.blk_counts = reinterpret_cast<int32_t *>(static_cast<char *>(ws) + layout(shape).map);
  a.status = status_word(ws);
  return cuda_status(launch_permute(a, (cudaStream_t)stream));
}

int64_t moe_padded_capacity(const moe_shape_t *shape) {
  if (!shape_ok(shape) || !shape->drop) return 0;
  const int64_t C = padded_rows_per_expert(shape->T, subseq(shape), shape->K, shape->E,
                                           shape->capacity_factor);
  return C * shape->E < (int64_t(1) << 31) ? C : 0;
}

moe_status_t moe_permute_padded(const moe_shape_t *shape, const void *x, const int32_t *topk_idx,
                                const uint8_t *keep, void *Xp, int32_t *row_of, int32_t *src_of,
                                int32_t *counts, int32_t *offsets, void *ws, moe_stream_t stream) {
  NvtxRange trace("moe_permute_padded");
  if (!shape_ok(shape)) return MOE_ERR_INVALID_ARG;
  if (!shape->drop) return MOE_ERR_UNSUPPORTED;   // dropless routing has no fixed capacity
  if (!x || !topk_idx || !keep || !row_of || !src_of || !counts || !offsets || !ws)
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || (Xp && !aligned16(Xp)) || !aligned16(ws)) return MOE_ERR_INVALID_ARG;
  const int64_t C = moe_padded_capacity(shape);
  if (C <= 0) return MOE_ERR_UNSUPPORTED;
  PermuteArgs a{};
  a.T = shape->T; a.d = shape->d; a.E = shape->E; a.K = shape->K; a.dtype = shape->dtype;
  a.x = x; a.topk_idx = topk_idx; a.keep = keep; a.Xp = Xp; a.row_of = row_of; a.src_of = src_of;
  a.counts = counts; a.offsets = offsets; a.pad_rows = C;
  a.blk_counts = reinterpret_cast<int32_t *>(static_cast<char *>(ws) + layout(shape).map);
  a.status = status_word(ws);
  cudaError_t e = launch_permute(a, (cudaStream_t)stream);
  if (e == cudaSuccess) e = launch_pad_fill(a, (cudaStream_t)stream);
  return cuda_status(e);
}

moe_status_t moe_permute_noalloc(const moe_shape_t *shape, const void *x, const int32_t *topk_idx,
                                 const uint8_t *keep, void *Xp, int32_t *row_of, int32_t *src_of,
                                 int32_t *counts, int32_t *offsets, moe_stream_t stream) {
  NvtxRange trace("moe_permute_noalloc");
  if (!shape_ok(shape)) return MOE_ERR_INVALID_ARG;
  if (!x || !topk_idx || !keep || !Xp || !row_of || !src_of || !counts || !offsets)
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(Xp)) return MOE_ERR_INVALID_ARG;
  if (shape->T > MOE_PERMUTE_NOALLOC_MAX_TOKENS) return MOE_ERR_UNSUPPORTED;
  PermuteArgs a{};
  a.T = shape->T; a.d = shape->d; a.E = shape->E; a.K = shape->K; a.dtype = shape->dtype;
  a.x = x; a.topk_idx = topk_idx; a.keep = keep; a.Xp = Xp; a.row_of = row_of; a.src_of = src_of;
  a.counts = counts; a.offsets = offsets;
  return cuda_status(launch_permute_noalloc(a, (cudaStream_t)stream));
}

static moe_status_t ffn_check(int32_t dtype, int64_t max_rows, int32_t d, int32_t F,
                              int32_t n_groups, const int32_t *offsets, void *ws) {
  if ((dtype != MOE_F32 && dtype != MOE_BF16) || max_rows < 1 || d < 1 || F < 1 || n_groups < 1 ||
      n_groups > 64 || !offsets || !ws || !aligned16(ws))
    return MOE_ERR_INVALID_ARG;
  if (max_rows >= (int64_t(1) << 31)) return MOE_ERR_INVALID_ARG;
  if (dtype == MOE_BF16 && (d % 128 != 0 || F % 128 != 0)) return MOE_ERR_UNSUPPORTED;
  if (dtype == MOE_F32 && (d % 4 != 0)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status_t moe_expert_ffn(int32_t dtype, int64_t max_rows, int32_t d, int32_t F,
                            int32_t n_groups, const int32_t *offsets, const void *Xp,
                            const void *W_gu, const void *W_down, void *A_save, void *H_save,
                            void *Yp, void *ws, moe_stream_t stream) {
  NvtxRange trace("moe_expert_ffn");
  moe_status_t st = ffn_check(dtype, max_rows, d, F, n_groups, offsets, ws);
  if (st != MOE_OK) return st;
  if (!Xp || !W_gu || !W_down || !H_save || !Yp) return MOE_ERR_INVALID_ARG;
  if (!aligned16(Xp) || !aligned16(W_gu) || !aligned16(W_down) || !aligned16(H_save) ||
      !aligned16(Yp) || (A_save && !aligned16(A_save)))
    return MOE_ERR_INVALID_ARG;
  FfnArgs a{};
  a.dtype = dtype; a.max_rows = max_rows; a.d = d; a.F = F; a.n_groups = n_groups;
  a.offsets = offsets; a.Xp = Xp; a.W_gu = W_gu; a.W_down = W_down; a.A_save = A_save;
  a.H_save = H_save; a.Yp = Yp; a.status = status_word(ws);
  cudaStream_t s = (cudaStream_t)stream;
  return cuda_status(dtype == MOE_BF16 ? launch_ffn_fwd_bf16(a, s) : launch_ffn_fwd_f32(a, s));
}

moe_status_t moe_expert_ffn_gather(int64_t max_rows, int32_t d, int32_t F, int32_t n_groups,
                                   const int32_t *offsets, const void *x, int64_t T, int32_t K,
                                   const int32_t *src_of, const void *W_gu, const void *W_down,
                                   void *A_save, void *H_save, void *Yp, void *ws,
                                   moe_stream_t stream) {
  NvtxRange trace("moe_expert_ffn_gather");
  moe_status_t st = ffn_check(MOE_BF16, max_rows, d, F, n_groups, offsets, ws);
  if (st != MOE_OK) return st;
  if (T < 1 || K < 1 || K > 8 || T * (int64_t)K >= (int64_t(1) << 31)) return MOE_ERR_INVALID_ARG;
  if (!x || !src_of || !W_gu || !W_down || !H_save || !Yp) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(W_gu) || !aligned16(W_down) || !aligned16(H_save) ||
      !aligned16(Yp) || (A_save && !aligned16(A_save)))
    return MOE_ERR_INVALID_ARG;
  FfnArgs a{};
  a.dtype = MOE_BF16; a.max_rows = max_rows; a.d = d; a.F = F; a.n_groups = n_groups;
  a.offsets = offsets; a.W_gu = W_gu; a.W_down = W_down; a.A_save = A_save;
  a.H_save = H_save; a.Yp = Yp; a.status = status_word(ws);
  a.x = x; a.src_of = src_of; a.K = K; a.T = T;
  const cudaError_t e = launch_ffn_fwd_bf16(a, (cudaStream_t)stream);
  return e == cudaErrorNotSupported ? MOE_ERR_UNSUPPORTED : cuda_status(e);
}

moe_status_t moe_unpermute(const moe_shape_t *shape, const void *Yp, const int32_t *row_of,
                           const float *topk_w, const void *Ys, const float *gate_logit, void *out,
                           moe_stream_t stream) {
  NvtxRange trace("moe_unpermute");
  if (!shape_ok(shape)) return MOE_ERR_INVALID_ARG;
  if (!Yp || !row_of || !topk_w || !out) return MOE_ERR_INVALID_ARG;
  if ((Ys == nullptr) != (gate_logit == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(Yp) || !aligned16(out) || (Ys && !aligned16(Ys))) return MOE_ERR_INVALID_ARG;
  UnpermuteArgs a{};
  a.T = shape->T; a.d = shape->d; a.K = shape->K; a.dtype = shape->dtype;
  a.Yp = Yp; a.row_of = row_of; a.topk_w = topk_w; a.Ys = Ys; a.gate_logit = gate_logit; a.out = out;
  return cuda_status(launch_unpermute(a, (cudaStream_t)stream));
}

moe_status_t moe_unpermute_bwd(const moe_shape_t *shape, const void *dout, const void *Yp,
                               const int32_t *row_of, const float *topk_w, const void *Ys,
                               const float *gate_logit, void *dYp, float *dw, void *dYs, float *dz,
                               moe_stream_t stream) {
  NvtxRange trace("moe_unpermute_bwd");
  if (!shape_ok(shape)) return MOE_ERR_INVALID_ARG;
  if (!dout || !Yp || !row_of || !topk_w || !dYp || !dw) return MOE_ERR_INVALID_ARG;
  const bool sh = Ys != nullptr;
  if ((gate_logit != nullptr) != sh || (dYs != nullptr) != sh || (dz != nullptr) != sh)
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(dout) || !aligned16(Yp) || !aligned16(dYp) || (sh && (!aligned16(Ys) || !aligned16(dYs))))
    return MOE_ERR_INVALID_ARG;
  UnpermuteArgs a{};
  a.T = shape->T; a.d = shape->d; a.K = shape->K; a.dtype = shape->dtype;
  a.dout = dout; a.Yp = Yp; a.row_of = row_of; a.topk_w = topk_w; a.Ys = Ys;
  a.gate_logit = gate_logit; a.dYp = dYp; a.dw = dw; a.dYs = dYs; a.dz = dz;
  return cuda_status(launch_unpermute_bwd(a, (cudaStream_t)stream));
}

moe_status_t moe_expert_ffn_bwd(int32_t dtype, int64_t max_rows, int32_t d, int32_t F,
                                int32_t n_groups, const int32_t *offsets, const void *dYp,
                                const void *Xp, const void *A_save, const void *H_save,
                                const void *W_gu, const void *W_down, void *dA, float *dXp,
                                float *dW_gu, float *dW_down, void *ws, size_t ws_bytes,
                                moe_stream_t stream) {
  NvtxRange trace("moe_expert_ffn_bwd");
  moe_status_t st = ffn_check(dtype, max_rows, d, F, n_groups, offsets, ws);
  if (st != MOE_OK) return st;
  if (ws_bytes < MOE_FFN_BWD_WORKSPACE_BYTES) return MOE_ERR_INVALID_ARG;
  if (!dYp || !Xp || !A_save || !H_save || !W_gu || !W_down || !dA || !dXp || !dW_gu || !dW_down)
    return MOE_ERR_INVALID_ARG;
  const void *ptrs[] = {dYp, Xp, A_save, H_save, W_gu, W_down, dA, dXp, dW_gu, dW_down};
  for (const void *q : ptrs)
    if (!aligned16(q)) return MOE_ERR_INVALID_ARG;
  FfnArgs a{};
  a.dtype = dtype; a.max_rows = max_rows; a.d = d; a.F = F; a.n_groups = n_groups;
  a.offsets = offsets; a.dYp = dYp; a.Xp = Xp; a.A_save = const_cast<void *>(A_save);
  a.H_save = const_cast<void *>(H_save); a.W_gu = W_gu; a.W_down = W_down; a.dA = dA;
  a.dXp = dXp; a.dW_gu = dW_gu; a.dW_down = dW_down; a.status = status_word(ws);
  // group tensor maps after the status word, 128-byte aligned
  a.maps = reinterpret_cast<void *>((reinterpret_cast<uintptr_t>(ws) + kStatusBytes + 127) &
                                    ~uintptr_t(127));
  static_assert(kStatusBytes + 127 + kFfnMapBytes <= MOE_FFN_BWD_WORKSPACE_BYTES,
                "group maps exceed the documented workspace");
  cudaStream_t s = (cudaStream_t)stream;
  return cuda_status(dtype == MOE_BF16 ? launch_ffn_bwd_bf16(a, s) : launch_ffn_bwd_f32(a, s));
}

moe_status_t moe_permute_bwd(const moe_shape_t *shape, const float *dXp, const int32_t *row_of,
                             const float *dx_add, float *dx, moe_stream_t stream) {
  NvtxRange trace("moe_permute_bwd");
  if (!shape_ok(shape)) return MOE_ERR_INVALID_ARG;
  if (!dXp || !row_of || !dx || !aligned16(dXp) || !aligned16(dx) || (dx_add && !aligned16(dx_add)))
    return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_permute_bwd(shape->T, shape->d, shape->K, dXp, row_of, dx_add, dx,
                                        (cudaStream_t)stream));
}

moe_status_t moe_sum_partials(int32_t dtype, int32_t n_parts, int64_t rows, int32_t d,
                              const void *partials, void *out, moe_stream_t stream) {
  NvtxRange trace("moe_sum_partials");
  if (dtype != MOE_BF16 && dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  if (n_parts < 1 || n_parts > 16 || rows < 0 || d < 1) return MOE_ERR_INVALID_ARG;
  if (d % (dtype == MOE_BF16 ? 8 : 4) != 0) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!partials || !out || !aligned16(partials) || !aligned16(out)) return MOE_ERR_INVALID_ARG;
  const size_t b = dtype == MOE_BF16 ? 2 : 4;
  const char *p0 = static_cast<const char *>(partials), *o0 = static_cast<const char *>(out);
  const size_t part = (size_t)rows * d * b;
  if (o0 < p0 + part * n_parts && p0 < o0 + part) return MOE_ERR_INVALID_ARG;   // aliasing
  return cuda_status(launch_sum_partials(dtype, n_parts, rows, d, partials, out,
                                         (cudaStream_t)stream));
}

static moe_status_t route_bwd(const moe_shape_t *shape, const void *x, const void *W_r,
                              const void *w_sg, const float *logits, const int32_t *topk_idx,
                              const float *topk_prob, const float *topk_w, const float *dw,
                              const float *dz, const float *dl_add, const float *dx_in,
                              float *dW_r, float *db_r, float *dw_sg, float *dx_router, void *ws,
                              moe_stream_t stream) {
  if (!shape_ok(shape)) return MOE_ERR_INVALID_ARG;
  if (!x || !W_r || !logits || !topk_idx || !topk_prob || !topk_w || !dw || !dW_r || !dx_router || !ws)
    return MOE_ERR_INVALID_ARG;
  const bool sh = w_sg != nullptr;
  if ((dz != nullptr) != sh || (dw_sg != nullptr) != sh) return MOE_ERR_INVALID_ARG;
  if (!aligned16(ws) || !aligned16(x) || !aligned16(W_r) || (sh && !aligned16(w_sg)) ||
      !aligned16(dx_router) || (dx_in != nullptr && !aligned16(dx_in)))
    return MOE_ERR_INVALID_ARG;   // 16-byte vector accesses
  const Layout L = layout(shape);
  RouteBwdArgs a{};
  a.T = shape->T; a.d = shape->d; a.E = shape->E; a.K = shape->K; a.dtype = shape->dtype;
  a.renorm = shape->renorm; a.x = x; a.W_r = W_r; a.w_sg = w_sg; a.logits = logits;
  a.topk_idx = topk_idx; a.topk_prob = topk_prob; a.topk_w = topk_w; a.dw = dw; a.dz = dz;
  a.dx_in = dx_in; a.dW_r = dW_r; a.db_r = db_r; a.dw_sg = dw_sg; a.dx_router = dx_router;
  a.dl_add = dl_add;
  a.dl = reinterpret_cast<float *>(static_cast<char *>(ws) + L.rbwd);
  a.partial = a.dl + align256((size_t)shape->T * shape->E * sizeof(float)) / sizeof(float);
  a.status = status_word(ws);
  return cuda_status(launch_route_bwd(a, (cudaStream_t)stream));
}

moe_status_t moe_route_bwd(const moe_shape_t *shape, const void *x, const void *W_r,
                           const void *w_sg, const float *logits, const int32_t *topk_idx,
                           const float *topk_prob, const float *topk_w, const float *dw,
                           const float *dz, const float *dx_in, float *dW_r, float *db_r,
                           float *dw_sg, float *dx_router, void *ws, moe_stream_t stream) {
  NvtxRange trace("moe_route_bwd");
  return route_bwd(shape, x, W_r, w_sg, logits, topk_idx, topk_prob, topk_w, dw, dz, nullptr, dx_in,
                   dW_r, db_r, dw_sg, dx_router, ws, stream);
}

moe_status_t moe_route_bwd_add(const moe_shape_t *shape, const void *x, const void *W_r,
                               const void *w_sg, const float *logits, const int32_t *topk_idx,
                               const float *topk_prob, const float *topk_w, const float *dw,
                               const float *dz, const float *dlogits_add, const float *dx_in,
                               float *dW_r, float *db_r, float *dw_sg, float *dx_router, void *ws,
                               moe_stream_t stream) {
  NvtxRange trace("moe_route_bwd_add");
  if (!shape_ok(shape) || !dlogits_add || !aligned4(dlogits_add)) return MOE_ERR_INVALID_ARG;
  const size_t n = (size_t)shape->T * shape->E * sizeof(float);
  if (overlap(dlogits_add, n, logits, n)) return MOE_ERR_INVALID_ARG;   // both are read
  // dl is written there while dlogits_add is read
  if (overlap(dlogits_add, n, ws, layout(shape).total)) return MOE_ERR_INVALID_ARG;
  return route_bwd(shape, x, W_r, w_sg, logits, topk_idx, topk_prob, topk_w, dw, dz, dlogits_add,
                   dx_in, dW_r, db_r, dw_sg, dx_router, ws, stream);
}

// ---------------------------------------------------------------------------
// Around the layer

static bool dtype_ok(int32_t dtype) { return dtype == MOE_F32 || dtype == MOE_BF16; }
static size_t size_of(int32_t dtype) { return dtype == MOE_BF16 ? 2 : 4; }
static bool group_ok(int32_t group) { return group == 0 || group == 32 || group == 64 || group == 128; }

// MOE_OK for a [rows, d] matrix that the norm's kernels take
static moe_status_t norm_check(int32_t dtype, int64_t rows, int32_t d) {
  if (!dtype_ok(dtype) || rows < 0 || d < 1 || d % (dtype == MOE_BF16 ? 8 : 4) != 0)
    return MOE_ERR_INVALID_ARG;
  if (rows >= (int64_t(1) << 31) || d > (dtype == MOE_BF16 ? 32768 : 16384)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status_t moe_rmsnorm(int32_t dtype, int64_t rows, int32_t d, const void *x, const void *residual,
                         const void *gamma, float eps, void *h, void *y, void *q, float *q_scale,
                         int32_t group, float *rstd, moe_stream_t stream) {
  NvtxRange trace("moe_rmsnorm");
  moe_status_t st = norm_check(dtype, rows, d);
  if (st != MOE_OK) return st;
  if (!(eps > 0.0f) || !std::isfinite(eps) || (q == nullptr) != (q_scale == nullptr) || group < 0)
    return MOE_ERR_INVALID_ARG;
  if (!group_ok(group)) return MOE_ERR_UNSUPPORTED;
  if (!h && !y && !q) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!x || !gamma) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || (residual && !aligned16(residual)) || !aligned16(gamma) || (h && !aligned16(h)) ||
      (y && !aligned16(y)) || (q && !aligned16(q)) || (q_scale && !aligned4(q_scale)) ||
      (rstd && !aligned4(rstd)))
    return MOE_ERR_INVALID_ARG;
  const size_t n = (size_t)rows * d, bytes = n * size_of(dtype);
  const int ng = group > 0 ? (d + group - 1) / group : 1;
  struct Range { const void *p; size_t n; };
  const Range outs[] = {{h, bytes}, {y, bytes}, {q, n}, {q_scale, (size_t)rows * ng * 4},
                        {rstd, (size_t)rows * 4}};
  const Range ins[] = {{x, bytes}, {residual, bytes}, {gamma, d * size_of(dtype)}};
  for (int i = 0; i < 5; ++i) {
    for (int j = i + 1; j < 5; ++j)
      if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return MOE_ERR_INVALID_ARG;
    for (int j = 0; j < 3; ++j) {
      const bool in_place = i < 2 && j < 2 && outs[i].p == ins[j].p;
      if (!in_place && overlap(outs[i].p, outs[i].n, ins[j].p, ins[j].n)) return MOE_ERR_INVALID_ARG;
    }
  }
  RmsNormArgs a{};
  a.rows = rows; a.d = d; a.dtype = dtype; a.group = group; a.eps = eps; a.x = x;
  a.residual = residual; a.gamma = gamma; a.h = h; a.y = y; a.q = q; a.q_scale = q_scale;
  a.rstd = rstd;
  return cuda_status(launch_rmsnorm(a, (cudaStream_t)stream));
}

size_t moe_rmsnorm_bwd_workspace_size(int64_t rows, int32_t d) {
  if (rows < 0 || rows >= (int64_t(1) << 31) || d < 1 || d > 32768) return 0;
  const size_t n = (size_t)rmsnorm_bwd_max_partials(rows > 0 ? rows : 1) * d * sizeof(float);
  return align256(n);
}

moe_status_t moe_rmsnorm_bwd(int32_t dtype, int32_t dy_dtype, int32_t dx_dtype, int64_t rows,
                             int32_t d, const void *dy, const void *h, const void *gamma,
                             const float *rstd, const void *dh, void *dx, float *dgamma, void *ws,
                             size_t ws_bytes, moe_stream_t stream) {
  NvtxRange trace("moe_rmsnorm_bwd");
  moe_status_t st = norm_check(dtype, rows, d);
  if (st != MOE_OK) return st;
  if (!dtype_ok(dy_dtype) || !dtype_ok(dx_dtype) ||
      (dtype == MOE_F32 && (dy_dtype != MOE_F32 || dx_dtype != MOE_F32)))
    return MOE_ERR_INVALID_ARG;
  if (!dgamma || !aligned16(dgamma)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if (rows == 0) return cuda_status(cudaMemsetAsync(dgamma, 0, (size_t)d * sizeof(float), s));
  if (!dy || !h || !gamma || !rstd || !dx || !ws) return MOE_ERR_INVALID_ARG;
  if (!aligned16(dy) || !aligned16(h) || !aligned16(gamma) || !aligned4(rstd) ||
      (dh && !aligned16(dh)) || !aligned16(dx) || !aligned16(ws))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < moe_rmsnorm_bwd_workspace_size(rows, d)) return MOE_ERR_INVALID_ARG;
  const size_t n = (size_t)rows * d, b = size_of(dtype), bdx = n * size_of(dx_dtype);
  const size_t bws = moe_rmsnorm_bwd_workspace_size(rows, d), bg = (size_t)d * sizeof(float);
  const bool on_dy = dx == dy && dx_dtype == dy_dtype, on_dh = dx == dh && dx_dtype == dtype;
  if ((!on_dy && overlap(dx, bdx, dy, n * size_of(dy_dtype))) ||
      (!on_dh && overlap(dx, bdx, dh, n * b)) || overlap(dx, bdx, h, n * b) ||
      overlap(dx, bdx, gamma, d * b) || overlap(dx, bdx, rstd, (size_t)rows * 4) ||
      overlap(dx, bdx, ws, bws) || overlap(dx, bdx, dgamma, bg))
    return MOE_ERR_INVALID_ARG;
  const struct { const void *p; size_t n; } ins[] = {{dy, n * size_of(dy_dtype)}, {h, n * b},
                                                     {gamma, d * b}, {rstd, (size_t)rows * 4},
                                                     {dh, n * b}};
  for (const auto &in : ins)
    if (overlap(dgamma, bg, in.p, in.n) || overlap(ws, bws, in.p, in.n)) return MOE_ERR_INVALID_ARG;
  if (overlap(dgamma, bg, ws, bws)) return MOE_ERR_INVALID_ARG;
  RmsNormBwdArgs a{};
  a.rows = rows; a.d = d; a.dtype = dtype; a.dy_dtype = dy_dtype; a.dx_dtype = dx_dtype; a.dy = dy;
  a.h = h; a.gamma = gamma; a.rstd = rstd; a.dh = dh; a.dx = dx; a.dgamma = dgamma;
  a.partial = static_cast<float *>(ws);
  return cuda_status(launch_rmsnorm_bwd(a, s));
}

static BalanceArgs balance_args(const moe_shape_t *s) {
  BalanceArgs a{};
  a.T = s->T; a.S = subseq(s); a.n_sub = (a.T + a.S - 1) / a.S; a.E = s->E; a.K = s->K;
  return a;
}

moe_status_t moe_balance_loss(const moe_shape_t *shape, const float *logits, const int32_t *topk_idx,
                              const uint8_t *mask, float alpha, float *loss, int32_t *counts,
                              float *prob_mean, float *coef, void *ws, moe_stream_t stream) {
  NvtxRange trace("moe_balance_loss");
  if (!shape_ok(shape) || !std::isfinite(alpha)) return MOE_ERR_INVALID_ARG;
  if (!logits || !topk_idx || !loss || !counts || !coef || !ws) return MOE_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned4(topk_idx) || !aligned4(loss) || !aligned4(counts) ||
      !aligned4(prob_mean) || !aligned16(coef) || !aligned16(ws))
    return MOE_ERR_INVALID_ARG;
  BalanceArgs a = balance_args(shape);
  const size_t pairs = (size_t)a.n_sub * a.E * 4;
  char *partial = static_cast<char *>(ws) + layout(shape).bal;
  const Span written[] = {{loss, 4}, {counts, pairs}, {prob_mean, pairs}, {coef, pairs + 4},
                          {ws, kStatusBytes}, {partial, balance_workspace_bytes(a.T, a.S, a.E)}};
  const Span read[] = {{logits, (size_t)a.T * a.E * 4}, {topk_idx, (size_t)a.T * a.K * 4},
                       {mask, (size_t)a.T}};
  if (any_overlap(written, read)) return MOE_ERR_INVALID_ARG;
  a.logits = logits; a.topk_idx = topk_idx; a.mask = mask; a.alpha = alpha; a.loss = loss;
  a.counts = counts; a.prob_mean = prob_mean; a.coef = coef;
  a.partial = partial;
  a.status = status_word(ws);
  return cuda_status(launch_balance_loss(a, (cudaStream_t)stream));
}

moe_status_t moe_balance_loss_bwd(const moe_shape_t *shape, const float *logits, const uint8_t *mask,
                                  const float *coef, const float *dloss, float *dlogits,
                                  moe_stream_t stream) {
  NvtxRange trace("moe_balance_loss_bwd");
  if (!shape_ok(shape) || !logits || !coef || !dlogits) return MOE_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned16(coef) || !aligned4(dloss) || !aligned16(dlogits))
    return MOE_ERR_INVALID_ARG;
  BalanceArgs a = balance_args(shape);
  const size_t n = (size_t)a.T * a.E * sizeof(float);
  const Span written[] = {{dlogits, n}};
  const Span read[] = {{dlogits == logits ? nullptr : logits, n}, {mask, (size_t)a.T},
                       {coef, (size_t)(a.n_sub * a.E + 1) * 4}, {dloss, 4}};
  if (any_overlap(written, read)) return MOE_ERR_INVALID_ARG;
  a.logits = logits; a.mask = mask; a.coef = const_cast<float *>(coef); a.dloss = dloss;
  a.dlogits = dlogits;
  return cuda_status(launch_balance_loss_bwd(a, (cudaStream_t)stream));
}

moe_status_t moe_permute_e4m3(const moe_shape_t *shape, const void *q, const float *q_scale,
                              int32_t group, const int32_t *topk_idx, const uint8_t *keep, void *Xp,
                              int32_t *row_of, int32_t *src_of, int32_t *counts, int32_t *offsets,
                              void *ws, moe_stream_t stream) {
  NvtxRange trace("moe_permute_e4m3");
  if (!shape_ok(shape) || group < 0) return MOE_ERR_INVALID_ARG;
  if (!group_ok(group)) return MOE_ERR_UNSUPPORTED;
  if ((size_t)shape->d * size_of(shape->dtype) > kPermRowCap) return MOE_ERR_UNSUPPORTED;
  if (!q || !q_scale || !topk_idx || !keep || !Xp || !row_of || !src_of || !counts || !offsets || !ws)
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned4(q_scale) || !aligned16(Xp) || !aligned16(ws) || !aligned4(topk_idx) ||
      !aligned4(row_of) || !aligned4(src_of) || !aligned4(counts) || !aligned4(offsets))
    return MOE_ERR_INVALID_ARG;
  const Layout L = layout(shape);
  const size_t T = (size_t)shape->T, d = (size_t)shape->d, slots = T * shape->K;
  const size_t scales = group > 0 ? (d + group - 1) / group : 1;
  const Span written[] = {{Xp, slots * d * size_of(shape->dtype)}, {row_of, slots * 4}, {src_of, slots * 4},
                          {counts, (size_t)shape->E * 4}, {offsets, (size_t)(shape->E + 1) * 4},
                          {ws, kStatusBytes}, {static_cast<char *>(ws) + L.map, L.cap - L.map}};
  const Span read[] = {{q, T * d}, {q_scale, T * scales * 4}, {topk_idx, slots * 4}, {keep, slots}};
  if (any_overlap(written, read)) return MOE_ERR_INVALID_ARG;
  PermuteArgs a{};
  a.T = shape->T; a.d = shape->d; a.E = shape->E; a.K = shape->K; a.dtype = shape->dtype;
  a.topk_idx = topk_idx; a.keep = keep; a.row_of = row_of; a.src_of = src_of;
  a.counts = counts; a.offsets = offsets;
  a.blk_counts = reinterpret_cast<int32_t *>(static_cast<char *>(ws) + L.map);
  a.status = status_word(ws);
  cudaError_t e = launch_permute(a, (cudaStream_t)stream);   // Xp NULL: the map
  a.Xp = Xp;
  if (e == cudaSuccess) e = launch_permute_e4m3_rows(a, q, q_scale, group, (cudaStream_t)stream);
  return cuda_status(e);
}

// MOE_OK for a list of tensors
static moe_status_t list_check(int32_t n, const moe_tensor_t *list) {
  if (n < 0 || (n > 0 && !list)) return MOE_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n; ++i) {
    const moe_tensor_t &t = list[i];
    if (t.numel < 0 || t.numel >= (int64_t(1) << 42) || !dtype_ok(t.dtype)) return MOE_ERR_INVALID_ARG;
    if (t.numel > 0 && (!t.data || reinterpret_cast<uintptr_t>(t.data) % size_of(t.dtype) != 0))
      return MOE_ERR_INVALID_ARG;
  }
  return MOE_OK;
}

static size_t bytes_of(const moe_tensor_t &t) { return (size_t)t.numel * size_of(t.dtype); }

// Whether clipping would write to what it still reads, or twice to one place:
// two outputs, or an output and another gradient, or norm or coef and an
// output, or coef and a gradient. The outputs are sorted by address, so that
// long lists cost n log n; only without host memory for that is every pair
// looked at.
static bool clip_overlap(int32_t n, const moe_tensor_t *grads, const moe_tensor_t *out,
                         const float *norm, const float *coef) {
  const moe_tensor_t *w = out != nullptr ? out : grads;
  if (overlap(norm, 4, coef, 4)) return true;
  for (int32_t i = 0; i < n; ++i) {
    if (grads[i].numel == 0) continue;   // nowhere
    const size_t b = bytes_of(grads[i]);
    if (overlap(norm, 4, w[i].data, b) || overlap(coef, 4, w[i].data, b) ||
        overlap(coef, 4, grads[i].data, b) ||
        (w[i].data != grads[i].data && overlap(w[i].data, b, grads[i].data, b)))
      return true;
  }
  constexpr int32_t kFew = 64;
  int32_t few[kFew];
  int32_t *order = n <= kFew ? few : static_cast<int32_t *>(std::malloc((size_t)n * sizeof(int32_t)));
  bool found = false;
  if (order == nullptr) {
    for (int32_t i = 0; i < n && !found; ++i)
      for (int32_t j = 0; j < n && !found; ++j)
        if (i != j && grads[i].numel > 0 && grads[j].numel > 0)
          found = overlap(w[i].data, bytes_of(w[i]), w[j].data, bytes_of(w[j])) ||
                  overlap(w[i].data, bytes_of(w[i]), grads[j].data, bytes_of(grads[j]));
    return found;
  }
  int32_t m = 0;
  for (int32_t i = 0; i < n; ++i)
    if (grads[i].numel > 0) order[m++] = i;
  const auto start = [&](int32_t i) { return reinterpret_cast<uintptr_t>(w[i].data); };
  std::sort(order, order + m, [&](int32_t i, int32_t j) { return start(i) < start(j); });
  for (int32_t k = 1; k < m && !found; ++k) found = start(order[k]) < start(order[k - 1]) + bytes_of(w[order[k - 1]]);
  if (out != nullptr)
    for (int32_t j = 0; j < n && !found; ++j) {
      if (grads[j].numel == 0) continue;
      // the outputs that start before this gradient's end, from the last: they
      // do not overlap each other, so the first that ends before it ends the search
      const uintptr_t at = reinterpret_cast<uintptr_t>(grads[j].data), end = at + bytes_of(grads[j]);
      int32_t k = (int32_t)(std::lower_bound(order, order + m, end,
                                             [&](int32_t i, uintptr_t v) { return start(i) < v; }) - order);
      while (--k >= 0 && start(order[k]) + bytes_of(w[order[k]]) > at && !found) found = order[k] != j;
    }
  if (order != few) std::free(order);
  return found;
}

moe_status_t moe_grad_norm(int32_t n, const moe_tensor_t *grads, float *norm, void *ws,
                           size_t ws_bytes, moe_stream_t stream) {
  NvtxRange trace("moe_grad_norm");
  static_assert(kMaxNormPartials * sizeof(double) <= MOE_GRAD_NORM_WORKSPACE_BYTES,
                "partial sums exceed the documented workspace");
  moe_status_t st = list_check(n, grads);
  if (st != MOE_OK) return st;
  if (!norm || !aligned4(norm) || !ws || !aligned16(ws) || ws_bytes < MOE_GRAD_NORM_WORKSPACE_BYTES)
    return MOE_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n; ++i)
    if (grads[i].numel > 0 && overlap(ws, MOE_GRAD_NORM_WORKSPACE_BYTES, grads[i].data, bytes_of(grads[i])))
      return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_grad_norm(n, grads, norm, static_cast<double *>(ws), (cudaStream_t)stream));
}

moe_status_t moe_grad_clip(int32_t n, const moe_tensor_t *grads, const moe_tensor_t *out,
                           const float *norm, float max_norm, float *coef, moe_stream_t stream) {
  NvtxRange trace("moe_grad_clip");
  moe_status_t st = list_check(n, grads);
  if (st == MOE_OK && out != nullptr) st = list_check(n, out);
  if (st != MOE_OK) return st;
  if (!norm || !aligned4(norm) || !aligned4(coef) || !(max_norm >= 0.0f) || !std::isfinite(max_norm))
    return MOE_ERR_INVALID_ARG;
  if (out != nullptr)
    for (int32_t i = 0; i < n; ++i)
      if (out[i].numel != grads[i].numel || out[i].dtype != grads[i].dtype) return MOE_ERR_INVALID_ARG;
  if (clip_overlap(n, grads, out, norm, coef)) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_grad_clip(n, grads, out, norm, max_norm, coef, (cudaStream_t)stream));
}

}  // extern "C"
