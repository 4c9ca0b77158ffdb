"""MoELayer: the whole layer through the C ABI, buffers held in torch tensors.

Forward: [moe_rmsnorm ->] moe_route [-> moe_balance_loss] -> moe_permute or
moe_permute_e4m3 -> moe_expert_ffn (routed experts)
[-> moe_expert_ffn (shared expert: one group, offsets {0, T})] -> moe_unpermute.
Backward: moe_unpermute_bwd -> moe_expert_ffn_bwd (routed [, shared])
[-> moe_balance_loss_bwd] -> moe_route_bwd -> moe_permute_bwd
[-> moe_rmsnorm_bwd]; clip_grads: moe_grad_norm -> moe_grad_clip.
torch only allocates device memory and supplies the stream; every step runs
in libmoe.so.
"""
from __future__ import annotations

import numpy as np
import torch

from . import _lib as L

E4M3_GROUP = 128   # columns per scale of the 8-bit rows


def to_device(a: np.ndarray, device="cuda") -> torch.Tensor:
    """Host array -> device tensor; uint16 arrays are bf16 bit patterns."""
    if a.dtype == np.uint16:
        return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16).to(device)
    return torch.from_numpy(np.ascontiguousarray(a)).to(device)


class MoELayer:
    """One MoE layer of configuration `cfg` (a synthetic.MoEConfig-like object)
    with device weights W_r, W_gu, W_down (+ b_r, w_sg, Ws_gu, Ws_down).

    etp > 1 runs the routed experts F-split the way an expert-tensor-parallel
    group of `etp` ranks would (MoE Parallel Folding study notes, "method
    overview": the expert's FFN dimension is sharded and a ReduceScatter-V
    sums the partial outputs): shard s holds gate and up rows
    [s*F/etp, (s+1)*F/etp) and the matching W_down columns, each shard is one
    moe_expert_ffn call, and moe_sum_partials adds the partial Yp (and, in the
    backward, the partial dXp) in shard order. Weight gradients stay per shard.

    layout="padded" (token dropping only) uses the fixed GShard-style layout of
    moe_permute_padded: expert e owns rows [e*C, (e+1)*C), zero rows after its
    kept ones, and the grouped GEMMs run every padded row.

    gather=True (bf16, forward only, etp = 1) fuses the permutation into the
    routed experts' gate/up GEMM: moe_permute builds the map alone (Xp NULL)
    and moe_expert_ffn_gather reads each permuted row from x through src_of,
    so the permuted copy of the tokens is never written.

    With a weight "gamma" [d] (in the layer's dtype) the layer is pre-normed:
    forward(x, residual) first forms h = x + residual (kept in self.h, the
    residual stream that goes on beside the output; without a residual self.h
    is x, which the backward reads) and runs the MoE layer on its RMS norm;
    backward(dout, dh=...) takes the gradient that reaches h from elsewhere
    and gives "dx", the gradient of h (so of x and residual alike), and
    "dgamma". dx_dtype="act" gives dx in the layer's dtype instead of fp32,
    which is what the layer below takes as its dout and dh.

    dispatch="e4m3" (with gamma; compact layout, no gather) moves the routed
    experts' rows in 8 bits with one scale per 128 columns: the norm writes
    them and moe_permute_e4m3 reads them. Router and shared expert still read
    the norm's output, so on one GPU this saves no memory traffic: it computes
    what a dispatch of 8-bit rows between ranks would. The gradient passes the
    rounding as if it were not there.

    balance > 0 adds the router's balance loss with that factor: forward leaves
    it in self.loss ([1], on the device) and the pre-drop counts per
    sub-sequence and expert in self.load; forward's mask ([T] uint8, 0 =
    padding) takes tokens out of it; backward adds its gradient, times dloss
    ([1] on the device) if given, to the router's.

    x, residual, dout and dh are [T, d] (or [..., d]) in the layer's dtype,
    dense, on the layer's device; a tensor of another kind is refused with a
    ValueError before anything is launched."""

    def __init__(self, cfg, weights: dict, device="cuda", backward=None, etp: int = 1,
                 layout: str = "compact", gather: bool = False, norm_eps: float = 1e-6,
                 dispatch: str = "act", balance: float = 0.0, dx_dtype: str = "f32"):
        self.cfg = cfg
        self.etp = etp
        self.layout = layout
        self.gather = gather
        if gather and (etp != 1 or cfg.dtype != "bf16"
                       or (cfg.backward if backward is None else backward)):
            raise ValueError("gather=True serves the bf16 forward-only layer with etp = 1")
        self.shape = L.shape_of(cfg)
        self.backward_enabled = cfg.backward if backward is None else backward
        self.w = weights
        T, d, E, K, F = cfg.T, cfg.d, cfg.E, cfg.K, cfg.F
        dt = torch.bfloat16 if cfg.dtype == "bf16" else torch.float32
        self.dt = dt
        self.dtype_code = L.MOE_BF16 if cfg.dtype == "bf16" else L.MOE_F32
        if layout == "padded":
            C = L.moe_padded_capacity(L.shape_of(cfg))
            if C <= 0:
                raise ValueError("the padded layout needs token dropping (a fixed capacity)")
            N = E * C
        elif layout == "compact":
            N = T * K
        else:
            raise ValueError(f"unknown layout {layout!r}")
        self.rows = N   # rows of the permuted buffers
        self.norm, self.norm_eps, self.balance = "gamma" in weights, norm_eps, balance
        if dispatch not in ("act", "e4m3") or dx_dtype not in ("f32", "act"):
            raise ValueError(f"unknown dispatch {dispatch!r} or dx_dtype {dx_dtype!r}")
        if dispatch == "e4m3" and (not self.norm or layout != "compact" or gather):
            raise ValueError('dispatch="e4m3" needs gamma, the compact layout and gather=False')
        if dx_dtype == "act" and not self.norm:
            raise ValueError('dx_dtype="act" needs gamma')
        self.e4m3 = dispatch == "e4m3"
        z = lambda *s, dtype=dt: torch.empty(*s, dtype=dtype, device=device)  # noqa: E731
        self.ws = torch.zeros(L.moe_workspace_size(self.shape), dtype=torch.uint8, device=device)
        if self.norm:
            self._take("gamma", weights["gamma"], (dt,), d)
            self.h_own = z(T, d)   # x + residual; without a residual h is x
            self.y = z(T, d)
            self.rstd = z(T, dtype=torch.float32)
            self.q = self.q_scale = None
            if self.e4m3:
                self.q = z(T, d, dtype=torch.float8_e4m3fn)
                self.q_scale = z(T, -(-d // E4M3_GROUP), dtype=torch.float32)
        if balance:
            n_sub = -(-T // cfg.subseq)
            self.loss = z(1, dtype=torch.float32)
            self.load = z(n_sub, E, dtype=torch.int32)
            self.prob_mean = z(n_sub, E, dtype=torch.float32)
            self.balance_coef = z(n_sub * E + 1, dtype=torch.float32)
        self.logits = z(T, E, dtype=torch.float32)
        self.topk_idx = z(T, K, dtype=torch.int32)
        self.topk_prob = z(T, K, dtype=torch.float32)
        self.topk_w = z(T, K, dtype=torch.float32)
        self.keep = z(T, K, dtype=torch.uint8)
        self.Xp = None if gather else z(N, d)
        self.row_of = z(T, K, dtype=torch.int32)
        self.src_of = z(N, dtype=torch.int32)
        self.counts = z(E, dtype=torch.int32)
        self.offsets = z(E + 1, dtype=torch.int32)
        self.A_save = z(N, 2 * F) if self.backward_enabled and etp == 1 else None
        self.H = z(N, F) if etp == 1 else None
        self.Yp = z(N, d)
        if etp > 1:
            if F % etp != 0:
                raise ValueError(f"F={F} does not split into {etp} shards")
            Fl = F // etp
            self.Fl = Fl
            Wgu, Wdn = weights["W_gu"], weights["W_down"]
            self.W_gu_s = [torch.cat([Wgu[:, s * Fl:(s + 1) * Fl], Wgu[:, F + s * Fl:F + (s + 1) * Fl]],
                                     dim=1).contiguous() for s in range(etp)]
            self.W_down_s = [Wdn[:, :, s * Fl:(s + 1) * Fl].contiguous() for s in range(etp)]
            self.A_s = [z(N, 2 * Fl) if self.backward_enabled else None for _ in range(etp)]
            self.H_s = [z(N, Fl) for _ in range(etp)]
            self.Y_parts = z(etp, N, d)
        self.out = z(T, d)
        self.shared = cfg.Fs > 0
        if self.shared:
            Fs = cfg.Fs
            self.gate_logit = z(T, dtype=torch.float32)
            self.off1 = torch.tensor([0, T], dtype=torch.int32, device=device)
            self.As = z(T, 2 * Fs) if self.backward_enabled else None
            self.Hs = z(T, Fs)
            self.Ys = z(T, d)
        else:
            self.gate_logit = self.Ys = None
        if self.backward_enabled:
            # zeros: in the padded layout the padding rows of dYp are never
            # written, and the weight gradients read them (times zero activations)
            self.dYp = torch.zeros((N, d), dtype=dt, device=device)
            self.dw = z(T, K, dtype=torch.float32)
            self.dXp = z(N, d, dtype=torch.float32)
            if etp == 1:
                self.dA = z(N, 2 * F)
                self.dW_gu = z(E, 2 * F, d, dtype=torch.float32)
                self.dW_down = z(E, d, F, dtype=torch.float32)
            else:
                Fl = self.Fl
                self.dA_s = z(N, 2 * Fl)   # reused shard after shard
                self.dX_parts = z(etp, N, d, dtype=torch.float32)
                self.dW_gu = [z(E, 2 * Fl, d, dtype=torch.float32) for _ in range(etp)]
                self.dW_down = [z(E, d, Fl, dtype=torch.float32) for _ in range(etp)]
            self.dW_r = z(E, d, dtype=torch.float32)
            self.db_r = z(E, dtype=torch.float32)
            self.dx_router = z(T, d, dtype=torch.float32)
            self.dx = z(T, d, dtype=torch.float32)
            if balance:
                self.dlogits = z(T, E, dtype=torch.float32)
            if self.norm:
                self.dgamma = z(d, dtype=torch.float32)
                # None: dx itself, in place
                self.dx_h = z(T, d) if dx_dtype == "act" and dt != torch.float32 else None
                self.norm_ws = z(L.moe_rmsnorm_bwd_workspace_size(T, d), dtype=torch.uint8)
            self.grad_ws = z(L.MOE_GRAD_NORM_WORKSPACE_BYTES, dtype=torch.uint8)
            self.grad_norm = z(1, dtype=torch.float32)
            if self.shared:
                Fs = cfg.Fs
                self.dYs = z(T, d)
                self.dz = z(T, dtype=torch.float32)
                self.dAs = z(T, 2 * Fs)
                self.dXs = z(T, d, dtype=torch.float32)
                self.dWs_gu = z(2 * Fs, d, dtype=torch.float32)
                self.dWs_down = z(d, Fs, dtype=torch.float32)
                self.dw_sg = z(d, dtype=torch.float32)

        self.grads = None   # the weight gradients' list, made by the first clip_grads

    def _take(self, name, t, dtypes, numel, last=None, more=False, hint=""):
        """Refuses a tensor that the kernels would misread: another type, size (`more`: a longer one serves, its front
        is read), last dimension (of more than one), layout or device. None and raw pointers pass."""
        if not isinstance(t, torch.Tensor):
            return
        if t.dtype not in dtypes:
            raise ValueError(f"{name} is {t.dtype}, not {' or '.join(map(str, dtypes))}{hint}")
        if t.numel() < numel or (t.numel() > numel and not more) or (last and t.dim() > 1 and t.shape[-1] != last):
            raise ValueError(f"{name} has shape {tuple(t.shape)}: {numel} elements"
                             + (f" in rows of {last}" if last else "") + " are wanted")
        if not t.is_contiguous():
            raise ValueError(f"{name} of shape {tuple(t.shape)} and strides {t.stride()} is not contiguous")
        if t.device != self.ws.device:
            raise ValueError(f"{name} is on {t.device}, the layer on {self.ws.device}")

    def forward(self, x: torch.Tensor, stream=None, residual=None, mask=None) -> torch.Tensor:
        c, s, w = self.cfg, self.shape, self.w
        if residual is not None and not self.norm:
            raise ValueError("a residual needs the norm (weight gamma)")
        if mask is not None and not self.balance:
            raise ValueError("a mask needs the balance loss")
        self._take("x", x, (self.dt,), c.T * c.d, more=True)
        self._take("residual", residual, (self.dt,), c.T * c.d, last=c.d)
        self._take("mask", mask, (torch.uint8, torch.bool, torch.int8), c.T)
        if self.norm:
            self.h = x if residual is None else self.h_own
            L.moe_rmsnorm(self.dtype_code, c.T, c.d, x, residual, w["gamma"], self.norm_eps,
                          None if residual is None else self.h, self.y, self.q, self.q_scale,
                          E4M3_GROUP if self.e4m3 else 0, self.rstd, stream)
            x = self.y
        self.x, self.mask = x, mask
        L.moe_route(s, x, w["W_r"], w.get("b_r"), w.get("w_sg"), self.logits, self.gate_logit,
                    self.topk_idx, self.topk_prob, self.topk_w, self.keep, self.ws, stream)
        if self.balance:
            L.moe_balance_loss(s, self.logits, self.topk_idx, mask, self.balance, self.loss,
                               self.load, self.prob_mean, self.balance_coef, self.ws, stream)
        if self.e4m3:
            L.moe_permute_e4m3(s, self.q, self.q_scale, E4M3_GROUP, self.topk_idx, self.keep,
                               self.Xp, self.row_of, self.src_of, self.counts, self.offsets,
                               self.ws, stream)
        else:
            permute = L.moe_permute_padded if self.layout == "padded" else L.moe_permute
            permute(s, x, self.topk_idx, self.keep, self.Xp, self.row_of, self.src_of,
                    self.counts, self.offsets, self.ws, stream)
        self.routed_ffn(stream)
        if self.shared:
            L.moe_expert_ffn(self.dtype_code, c.T, c.d, c.Fs, 1, self.off1, x, w["Ws_gu"],
                             w["Ws_down"], self.As, self.Hs, self.Ys, self.ws, stream)
        L.moe_unpermute(s, self.Yp, self.row_of, self.topk_w, self.Ys, self.gate_logit, self.out,
                        stream)
        return self.out

    def routed_ffn(self, stream=None):
        c, w = self.cfg, self.w
        if self.gather:
            L.moe_expert_ffn_gather(self.rows, c.d, c.F, c.E, self.offsets, self.x, c.T, c.K,
                                    self.src_of, w["W_gu"], w["W_down"], self.A_save, self.H,
                                    self.Yp, self.ws, stream)
            return
        if self.etp == 1:
            L.moe_expert_ffn(self.dtype_code, self.rows, c.d, c.F, c.E, self.offsets, self.Xp,
                             w["W_gu"], w["W_down"], self.A_save, self.H, self.Yp, self.ws, stream)
            return
        for s in range(self.etp):
            L.moe_expert_ffn(self.dtype_code, self.rows, c.d, self.Fl, c.E, self.offsets, self.Xp,
                             self.W_gu_s[s], self.W_down_s[s], self.A_s[s], self.H_s[s],
                             self.Y_parts[s], self.ws, stream)
        L.moe_sum_partials(self.dtype_code, self.etp, self.rows, c.d, self.Y_parts, self.Yp, stream)

    def routed_ffn_bwd(self, stream=None):
        c, w = self.cfg, self.w
        if self.etp == 1:
            L.moe_expert_ffn_bwd(self.dtype_code, self.rows, c.d, c.F, c.E, self.offsets, self.dYp,
                                 self.Xp, self.A_save, self.H, w["W_gu"], w["W_down"], self.dA,
                                 self.dXp, self.dW_gu, self.dW_down, self.ws, stream)
            return
        for s in range(self.etp):
            L.moe_expert_ffn_bwd(self.dtype_code, self.rows, c.d, self.Fl, c.E, self.offsets,
                                 self.dYp, self.Xp, self.A_s[s], self.H_s[s], self.W_gu_s[s],
                                 self.W_down_s[s], self.dA_s, self.dX_parts[s], self.dW_gu[s],
                                 self.dW_down[s], self.ws, stream)
        L.moe_sum_partials(L.MOE_F32, self.etp, self.rows, c.d, self.dX_parts, self.dXp, stream)

    def backward(self, dout: torch.Tensor, stream=None, marks=None, dh=None, dloss=None) -> dict:
        """marks: optional dict of (start, end) CUDA event pairs, keyed by
        "unpermute_bwd", "ffn_bwd" (routed experts), "shared_ffn_bwd",
        "route_bwd" (the balance loss's gradient included), "permute_bwd" and
        "norm_bwd"; each present pair is recorded on the current stream around
        that call."""
        c, s, w = self.cfg, self.shape, self.w
        marks = marks or {}
        if dh is not None and not self.norm:
            raise ValueError("dh needs the norm (weight gamma)")
        if dloss is not None and not self.balance:
            raise ValueError("dloss needs the balance loss")
        hint = ' (a layer gives its dx in that type with dx_dtype="act")' if self.dt != torch.float32 else ""
        self._take("dout", dout, (self.dt,), c.T * c.d, more=True, hint=hint)
        self._take("dh", dh, (self.dt,), c.T * c.d, last=c.d, hint=hint)
        self._take("dloss", dloss, (torch.float32,), 1)

        def mark(name, i):
            if name in marks:
                marks[name][i].record()

        mark("unpermute_bwd", 0)
        L.moe_unpermute_bwd(s, dout, self.Yp, self.row_of, self.topk_w, self.Ys, self.gate_logit,
                            self.dYp, self.dw, self.dYs if self.shared else None,
                            self.dz if self.shared else None, stream)
        mark("unpermute_bwd", 1)
        mark("ffn_bwd", 0)
        self.routed_ffn_bwd(stream)
        mark("ffn_bwd", 1)
        dx_in = None
        if self.shared:
            mark("shared_ffn_bwd", 0)
            L.moe_expert_ffn_bwd(self.dtype_code, c.T, c.d, c.Fs, 1, self.off1, self.dYs, self.x,
                                 self.As, self.Hs, w["Ws_gu"], w["Ws_down"], self.dAs, self.dXs,
                                 self.dWs_gu, self.dWs_down, self.ws, stream)
            mark("shared_ffn_bwd", 1)
            dx_in = self.dXs
        mark("route_bwd", 0)
        args = [s, self.x, w["W_r"], w.get("w_sg"), self.logits, self.topk_idx, self.topk_prob,
                self.topk_w, self.dw, self.dz if self.shared else None]
        outs = [dx_in, self.dW_r, self.db_r if "b_r" in w else None,
                self.dw_sg if self.shared else None, self.dx_router, self.ws, stream]
        if self.balance:
            L.moe_balance_loss_bwd(s, self.logits, self.mask, self.balance_coef, dloss,
                                   self.dlogits, stream)
            L.moe_route_bwd_add(*args, self.dlogits, *outs)
        else:
            L.moe_route_bwd(*args, *outs)
        mark("route_bwd", 1)
        mark("permute_bwd", 0)
        L.moe_permute_bwd(s, self.dXp, self.row_of, self.dx_router, self.dx, stream)
        mark("permute_bwd", 1)
        dx = self.dx
        if self.norm:
            mark("norm_bwd", 0)
            code = L.MOE_F32
            if self.dx_h is not None:   # dx leaves in the layer's dtype
                dx, code = self.dx_h, self.dtype_code
            L.moe_rmsnorm_bwd(self.dtype_code, L.MOE_F32, code,
                              c.T, c.d, self.dx, self.h, w["gamma"], self.rstd, dh, dx, self.dgamma,
                              self.norm_ws, stream)
            mark("norm_bwd", 1)
        g = {"dx": dx, "dW_r": self.dW_r, "dW_gu": self.dW_gu, "dW_down": self.dW_down}
        if self.norm:
            g["dgamma"] = self.dgamma
        if "b_r" in w:
            g["db_r"] = self.db_r
        if self.shared:
            g.update(dWs_gu=self.dWs_gu, dWs_down=self.dWs_down, dw_sg=self.dw_sg)
        return g

    def weight_grads(self) -> list:
        """The weight gradients that backward writes, as one flat list (for a
        TensorList over several layers)."""
        g = [self.dW_r]
        for t in (self.dW_gu, self.dW_down):
            g += t if isinstance(t, list) else [t]
        if "b_r" in self.w:
            g.append(self.db_r)
        if self.shared:
            g += [self.dWs_gu, self.dWs_down, self.dw_sg]
        if self.norm:
            g.append(self.dgamma)
        return g

    def clip_grads(self, max_norm: float, stream=None) -> torch.Tensor:
        """Clips the weight gradients in place to a global norm of max_norm and
        returns their norm before it, [1] on the device; a norm that is not
        finite leaves them as they are."""
        now = self.weight_grads()
        old = [] if self.grads is None else self.grads.tensors
        if len(now) != len(old) or any(a is not b for a, b in zip(now, old)):
            self.grads = L.TensorList(now)   # the first call, or a buffer was replaced
        L.moe_grad_norm(self.grads, self.grad_norm, self.grad_ws, stream)
        L.moe_grad_clip(self.grads, None, self.grad_norm, max_norm, None, stream)
        return self.grad_norm
