"""The pre-normed layer with its balance loss, 8-bit rows and gradient
clipping, as a training step runs them: fp32 layers against 64-bit autograd of
the whole step (routing decisions and 8-bit values taken from the layer; the
fp32 tolerance of the layer tests), bf16 layers bit for bit against the same
calls made one by one."""
import dataclasses

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from synthetic import get_config, make_inputs  # noqa: E402
from tests.gpu_util import assert_close, dev, host, lib  # noqa: E402

ALPHA, EPS = 0.05, 1e-6


def _weights(cfg, inp):
    rng = np.random.default_rng(7)
    w = {k: dev(v) for k, v in inp.items() if k not in ("x", "dout")}
    dt = torch.bfloat16 if cfg.dtype == "bf16" else torch.float32
    w["gamma"] = torch.from_numpy(1 + 0.2 * rng.standard_normal(cfg.d)).to(dt).cuda()
    r = torch.from_numpy(rng.standard_normal((cfg.T, cfg.d))).to(dt).cuda()
    dh = torch.from_numpy(rng.standard_normal((cfg.T, cfg.d))).to(dt).cuda()
    mask = torch.from_numpy((rng.random(cfg.T) < 0.8).astype(np.uint8)).cuda()
    return w, r, dh, mask


def _autograd_step(cfg, layer, w, x, r, dout, dh, mask, dloss):
    """The step's outputs and gradients in 64 bits, on the CPU."""
    P = {k: v.detach().cpu().double().requires_grad_() for k, v in w.items()}
    h = (x.cpu() + r.cpu()).double().requires_grad_()
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * P["gamma"]
    logits = y @ P["W_r"].T + (P["b_r"] if "b_r" in P else 0.0)
    p = torch.softmax(logits, 1)
    idx, keep = layer.topk_idx.cpu().long(), layer.keep.cpu().bool()
    pk = p.gather(1, idx)
    wk = pk / pk.sum(1, keepdim=True) if cfg.renorm else pk
    xe = y
    if layer.e4m3:   # the values that the bytes stand for, the gradient straight through
        q = layer.q.float().cpu().double() * layer.q_scale.cpu().double().repeat_interleave(128, 1)[:, :cfg.d]
        xe = y + (q - y).detach()

    def ffn(a, gu, down):
        g, u = (a @ gu.T).chunk(2, dim=1)
        return (torch.nn.functional.silu(g) * u) @ down.T

    out = torch.zeros_like(y)
    for e in range(cfg.E):
        t, k = torch.nonzero((idx == e) & keep, as_tuple=True)
        if len(t):
            out = out.index_add(0, t, wk[t, k][:, None] * ffn(xe[t], P["W_gu"][e], P["W_down"][e]))
    if cfg.Fs:
        out = out + torch.sigmoid(y @ P["w_sg"])[:, None] * ffn(y, P["Ws_gu"], P["Ws_down"])
    live = mask.cpu().bool()
    loss, n = 0.0, int(live.sum())
    for lo in range(0, cfg.T, cfg.subseq):
        at = torch.arange(lo, min(cfg.T, lo + cfg.subseq))
        at = at[live[at]]
        c = torch.bincount(idx[at].reshape(-1), minlength=cfg.E).double()
        loss = loss + ALPHA * cfg.E / (cfg.K * n) * (c * p[at].mean(0)).sum()
    total = (out * dout.cpu().double()).sum() + (h * dh.cpu().double()).sum() + dloss * loss
    names = [k for k in P]
    grads = torch.autograd.grad(total, [h] + [P[k] for k in names])
    return out.detach(), loss.item(), grads[0], dict(zip(names, grads[1:]))


GRAD = {"gamma": "dgamma", "W_r": "dW_r", "W_gu": "dW_gu", "W_down": "dW_down", "b_r": "db_r", "w_sg": "dw_sg",
        "Ws_gu": "dWs_gu", "Ws_down": "dWs_down"}


@pytest.mark.gpu
@pytest.mark.parametrize("dispatch", ["act", "e4m3"])
@pytest.mark.parametrize("kw", [dict(), dict(T=300, E=8, K=3, S=64, drop=True, cf=0.8),
                                dict(T=257, d=136, E=6, K=2, F=72, bias=True, Fs=64, S=100)], ids=["tiny", "drop", "shared"])
def test_f32_training_step(kw, dispatch):
    L = lib()
    from token_dispatch_expert_moe_gb300.layer import MoELayer
    cfg = dataclasses.replace(get_config("tiny_f32"), backward=True, **kw)
    inp = make_inputs(cfg, need_backward=True)
    w, r, dh, mask = _weights(cfg, inp)
    layer = MoELayer(cfg, w, backward=True, balance=ALPHA, dispatch=dispatch, norm_eps=EPS)
    x, dout = dev(inp["x"]), dev(inp["dout"])
    dloss = torch.tensor([3.0], device="cuda")
    out = layer.forward(x, residual=r, mask=mask)
    g = layer.backward(dout, dh=dh, dloss=dloss)
    assert L.moe_get_status(layer.ws)[0] == 0
    ref, loss, dx, grads = _autograd_step(cfg, layer, w, x, r, dout, dh, mask, 3.0)
    assert torch.equal(layer.h, x + r)
    assert_close("out", host(out), ref.numpy(), "f32")
    assert abs(float(layer.loss) - loss) <= 1e-5 * loss
    assert int(layer.load.sum()) == int(mask.sum()) * cfg.K
    assert_close("dx", host(g["dx"]), dx.numpy(), "f32")
    for k, v in grads.items():
        assert_close(GRAD[k], host(g[GRAD[k]]), v.numpy(), "f32")
    # clipping: the norm of exactly these gradients, every one scaled
    before = {k: v.clone() for k, v in g.items() if k != "dx"}
    want = float(torch.sqrt(sum((v.double() ** 2).sum() for v in before.values())))
    norm = layer.clip_grads(0.25 * want)
    torch.cuda.synchronize()
    assert abs(float(norm) - want) <= 1e-5 * want
    coef = float(np.float32(0.25 * want) / np.float32(float(norm)))
    for k, v in before.items():
        assert torch.equal(g[k], v * coef), k
    assert abs(float(layer.clip_grads(1e9)) - 0.25 * want) <= 1e-5 * want


BF16 = [("mixtral_8x22b@small", {}), ("qwen2_57b_a14b@small", {}), ("mixtral_8x22b_g8t8@small", dict(layout="padded")),
        ("mixtral_8x22b_g8t8@small", dict(etp=2)), ("llama3_8x70b@small", dict(dx_dtype="act"))]


@pytest.mark.gpu
@pytest.mark.parametrize("name,kw", BF16, ids=lambda v: v if isinstance(v, str) else "-".join(map(str, v.values())) or "plain")
def test_bf16_step_is_the_calls_one_by_one(name, kw):
    L = lib()
    from token_dispatch_expert_moe_gb300.layer import MoELayer
    cfg = get_config(name)
    inp = make_inputs(cfg, need_backward=True)
    w, r, dh, mask = _weights(cfg, inp)
    x, dout = dev(inp["x"]), dev(inp["dout"])
    layer = MoELayer(cfg, w, backward=True, balance=ALPHA, norm_eps=EPS, **kw)
    out = layer.forward(x, residual=r, mask=mask)
    g = layer.backward(dout, dh=dh)
    T, d = cfg.T, cfg.d
    h, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device="cuda")
    L.moe_rmsnorm(L.MOE_BF16, T, d, x, r, w["gamma"], EPS, h, y, None, None, 0, rstd)
    plain = {k: v for k, v in kw.items() if k != "dx_dtype"}
    inner = MoELayer(cfg, {k: v for k, v in w.items() if k != "gamma"}, backward=True, balance=ALPHA, **plain)
    out2 = inner.forward(y, mask=mask)
    g2 = inner.backward(dout)
    assert torch.equal(out, out2) and torch.equal(layer.h, h) and torch.equal(layer.loss, inner.loss)
    act = kw.get("dx_dtype") == "act"
    dx = torch.empty(T, d, dtype=torch.bfloat16 if act else torch.float32, device="cuda")
    dgamma = torch.empty(d, device="cuda")
    ws = torch.empty(L.moe_rmsnorm_bwd_workspace_size(T, d), dtype=torch.uint8, device="cuda")
    L.moe_rmsnorm_bwd(L.MOE_BF16, L.MOE_F32, L.MOE_BF16 if act else L.MOE_F32, T, d, g2["dx"], h, w["gamma"], rstd, dh, dx,
                      dgamma, ws)
    torch.cuda.synchronize()
    assert torch.equal(g["dx"], dx) and torch.equal(g["dgamma"], dgamma)
    for k in g2:
        if k != "dx":
            a, b = (v if isinstance(v, list) else [v] for v in (g[k], g2[k]))
            assert all(torch.equal(s, t) for s, t in zip(a, b)), k
    # the balance loss moves the router's gradient, and nothing else of the weights'
    bare = MoELayer(cfg, {k: v for k, v in w.items() if k != "gamma"}, backward=True, **plain)
    bare.forward(y)
    g3 = bare.backward(dout)
    assert not torch.equal(g3["dW_r"], g2["dW_r"])
    assert torch.equal(*(torch.stack(v[k]) if isinstance(v[k], list) else v[k] for v in (g3, g2) for k in ("dW_gu",)))
    assert len(layer.weight_grads()) == sum(len(v) if isinstance(v, list) else 1 for k, v in g.items() if k != "dx")


@pytest.mark.gpu
def test_bf16_rows_in_8_bits():
    """dispatch="e4m3": Xp holds the values of the 8-bit rows; without a
    residual h is x; two stacked layers pass bf16 gradients down."""
    L = lib()
    from token_dispatch_expert_moe_gb300.layer import MoELayer
    cfg = get_config("mixtral_8x22b_g8t8@small")
    inp = make_inputs(cfg, need_backward=True)
    w, r, dh, _ = _weights(cfg, inp)
    x, dout = dev(inp["x"]), dev(inp["dout"])
    low = MoELayer(cfg, w, backward=True, dispatch="e4m3", dx_dtype="act")
    top = MoELayer(cfg, w, backward=True, dispatch="e4m3", dx_dtype="act")
    o1 = low.forward(x)
    assert low.h is x
    top.forward(o1, residual=low.h)
    n = int(top.offsets[cfg.E])
    rows = (top.q.float() * top.q_scale.repeat_interleave(128, 1)).to(torch.bfloat16)
    assert torch.equal(top.Xp[:n], rows[(top.src_of[:n] // cfg.K).long()])
    # 8 bits are near the rows they stand for: half a step of 2^-4
    assert (rows.float() - top.y.float()).norm() <= 2.0 ** -4 * top.y.float().norm()
    g = top.backward(dout, dh=dh)
    g1 = low.backward(g["dx"], dh=g["dx"])
    assert g1["dx"].dtype == torch.bfloat16 and all(torch.isfinite(v.float()).all() for v in g1.values())
    assert L.moe_get_status(low.ws)[0] == 0 and L.moe_get_status(top.ws)[0] == 0
    grads = L.TensorList(low.weight_grads() + top.weight_grads())   # one norm over both layers
    norm = torch.empty(1, device="cuda")
    L.moe_grad_norm(grads, norm, low.grad_ws)
    want = torch.sqrt(sum((t.double() ** 2).sum() for t in grads.tensors))
    assert abs(float(norm) - float(want)) <= 1e-5 * float(want)


@pytest.mark.gpu
def test_captured_step():
    """A whole step in one graph, replayed on new inputs."""
    lib()
    from token_dispatch_expert_moe_gb300.layer import MoELayer
    cfg = get_config("qwen2_57b_a14b@small")
    inp = make_inputs(cfg, need_backward=True)
    w, r, dh, mask = _weights(cfg, inp)
    x, dout = dev(inp["x"]), dev(inp["dout"])
    layer = MoELayer(cfg, w, backward=True, balance=ALPHA, dispatch="e4m3")

    def step():
        out = layer.forward(x, residual=r, mask=mask)
        g = layer.backward(dout, dh=dh)
        return out, g, layer.clip_grads(1.0)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, g, norm = step()
    x.copy_(x.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (out, norm, layer.loss, *g.values())]
    out, g, norm = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (out, norm, layer.loss, *g.values())))


@pytest.mark.gpu
def test_options_that_do_not_go_together():
    lib()
    from token_dispatch_expert_moe_gb300.layer import MoELayer
    cfg = get_config("mixtral_8x22b@small")
    inp = make_inputs(cfg, need_backward=False)
    w, r, _, mask = _weights(cfg, inp)
    bare = {k: v for k, v in w.items() if k != "gamma"}
    for weights, kw in ((bare, dict(dispatch="e4m3")), (w, dict(dispatch="e4m3", layout="padded")),
                        (w, dict(dispatch="e4m3", gather=True)), (w, dict(dispatch="int8")), (bare, dict(dx_dtype="act")),
                        (w, dict(dx_dtype="bf16"))):
        with pytest.raises(ValueError):
            MoELayer(cfg, weights, backward=False, **kw)
    layer = MoELayer(cfg, bare, backward=False)
    x = dev(inp["x"])
    with pytest.raises(ValueError):
        layer.forward(x, residual=r)
    with pytest.raises(ValueError):
        layer.forward(x, mask=mask)
    normed = MoELayer(cfg, w, backward=False, gather=True)   # the fused permutation reads the norm's output
    plain = MoELayer(cfg, w, backward=False)
    assert torch.equal(normed.forward(x), plain.forward(x))
