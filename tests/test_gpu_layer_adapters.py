"""The layer with residual dropout and per-token adapters, as a fine-tuning
step and a serving step run them: fp32 layers against 64-bit autograd of the
whole step (routing decisions taken from the layer; the fp32 tolerance of the
layer tests), bf16 layers bit for bit against the same calls made one by one."""
import dataclasses

import pytest

torch = pytest.importorskip("torch")

from synthetic import get_config, make_inputs  # noqa: E402
from tests.adapter_util import dropped  # noqa: E402
from tests.gpu_util import assert_close, dev, host, lib  # noqa: E402
from tests.test_gpu_layer_around import EPS, GRAD, _weights  # noqa: E402

SEEDS = [[12345, 2 ** 40], [2 ** 62 + 1, 7]]   # of the residual's dropout and of the adapters'


def _adapters(cfg, w, n, rank):
    g = torch.Generator().manual_seed(n)
    dt = torch.bfloat16 if cfg.dtype == "bf16" else torch.float32
    w["lora_A"] = (torch.randn(n, rank, cfg.d, generator=g) / cfg.d ** 0.5).to(dt).cuda()
    w["lora_B"] = (torch.randn(n, cfg.d, rank, generator=g) / rank ** 0.5).to(dt).cuda()
    w["lora_scale"] = (torch.rand(n, generator=g) + 0.5).cuda()
    return torch.randint(-1, n, (cfg.T,), generator=g).int().cuda(), torch.tensor(SEEDS, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(), dict(T=257, d=136, E=6, K=2, F=72, bias=True, Fs=64)], ids=["tiny", "shared"])
@pytest.mark.parametrize("train", [True, False])
def test_f32_step(kw, train):
    L = lib()
    from token_dispatch_expert_moe_gb300.layer import MoELayer
    cfg = dataclasses.replace(get_config("tiny_f32"), backward=True, **kw)
    inp = make_inputs(cfg, need_backward=True)
    w, r, dh, _ = _weights(cfg, inp)
    ids, rng = _adapters(cfg, w, 3, 12)
    p, q = 0.2, 0.3
    layer = MoELayer(cfg, w, backward=True, norm_eps=EPS, dropout=p, adapter_dropout=q)
    x, dout = dev(inp["x"]), dev(inp["dout"])
    out = layer.forward(x, residual=r, adapter=ids, rng=rng if train else None)
    g = layer.backward(dout, dh=dh)
    assert L.moe_get_status(layer.ws)[0] == 0 and L.moe_get_status(layer.adapter_ws)[0] == 0

    P = {k: v.detach().cpu().double().requires_grad_() for k, v in w.items() if k != "lora_scale"}
    one = torch.ones(cfg.T, cfg.d)
    keep, keep_a = (dropped(one, pr, *s) if train else one.double() for pr, s in zip((p, q), SEEDS))
    xd, rd = x.cpu().double().requires_grad_(), r.cpu().double().requires_grad_()
    h = rd + xd * keep
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * P["gamma"]
    prob = torch.softmax(y @ P["W_r"].T + (P["b_r"] if "b_r" in P else 0.0), 1)
    idx = layer.topk_idx.cpu().long()
    pk = prob.gather(1, idx)
    wk = pk / pk.sum(1, keepdim=True) if cfg.renorm else pk

    def ffn(a, gu, down):
        gate, up = (a @ gu.T).chunk(2, dim=1)
        return (torch.nn.functional.silu(gate) * up) @ down.T

    ref = torch.zeros_like(y)
    for e in range(cfg.E):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        ref = ref.index_add(0, t, wk[t, k][:, None] * ffn(y[t], P["W_gu"][e], P["W_down"][e]))
    if cfg.Fs:
        ref = ref + torch.sigmoid(y @ P["w_sg"])[:, None] * ffn(y, P["Ws_gu"], P["Ws_down"])
    a = ids.cpu().long()
    for i in range(3):
        t = torch.nonzero(a == i)[:, 0]
        ref = ref.index_add(0, t, float(w["lora_scale"][i]) * ((y * keep_a)[t] @ P["lora_A"][i].T) @ P["lora_B"][i].T)
    names = list(P)
    grads = torch.autograd.grad((ref * dout.cpu().double()).sum() + (h * dh.cpu().double()).sum(), [rd, xd] + [P[k] for k in names])
    assert_close("out", host(out), ref.detach().numpy(), "f32")
    assert_close("dx", host(g["dx"]), grads[0].numpy(), "f32")
    assert_close("dx_drop", host(g["dx_drop"]), grads[1].numpy(), "f32")
    for k, v in zip(names, grads[2:]):
        key = GRAD.get(k, "d" + k)
        assert_close(key, host(g[key]), v.numpy(), "f32")
    norm = layer.clip_grads(1e9)
    want = torch.sqrt(sum((t.double() ** 2).sum() for t in layer.weight_grads()))
    assert len(layer.weight_grads()) == len(names) and abs(float(norm) - float(want)) <= 1e-5 * float(want)


@pytest.mark.gpu
@pytest.mark.parametrize("name,kw", [("mixtral_8x22b@small", {}), ("qwen2_57b_a14b@small", dict(dispatch="e4m3")),
                                     ("llama3_8x70b@small", dict(dx_dtype="act"))])
def test_bf16_step_is_the_calls_one_by_one(name, kw):
    L = lib()
    from token_dispatch_expert_moe_gb300.layer import MoELayer
    cfg = get_config(name)
    inp = make_inputs(cfg, need_backward=True)
    w, r, dh, _ = _weights(cfg, inp)
    ids, rng = _adapters(cfg, w, 5, 16)
    x, dout = dev(inp["x"]), dev(inp["dout"])
    layer = MoELayer(cfg, w, backward=True, norm_eps=EPS, dropout=0.1, adapter_dropout=0.2, **kw)
    out = layer.forward(x, residual=r, adapter=ids, rng=rng)
    g = layer.backward(dout, dh=dh)
    T, d = cfg.T, cfg.d
    # the dropout and the residual, then the layer without adapters, then these
    h = torch.empty_like(x)
    L.moe_dropout(L.MOE_BF16, T * d, x, r, 0.1, rng[0], h)
    inner = MoELayer(cfg, {k: v for k, v in w.items() if not k.startswith("lora")}, backward=True, norm_eps=EPS, **kw)
    o = inner.forward(h)
    s = L.MoEAdapterShape(T=T, d_in=d, d_out=d, n=5, rank=16, dtype=L.MOE_BF16, dropout=0.2)
    ws = torch.zeros(L.moe_adapter_workspace_size(s), dtype=torch.uint8, device="cuda")
    m = torch.empty(L.moe_adapter_map_size(s), dtype=torch.uint8, device="cuda")
    u, y = torch.empty(T, 16, device="cuda"), torch.empty_like(o)
    L.moe_adapter_map(s, ids, m, ws)
    L.moe_adapter(s, inner.y, w["lora_A"], w["lora_B"], w["lora_scale"], None, m, rng[1], o, y, u, ws)
    assert torch.equal(layer.h, h) and torch.equal(out, y) and torch.equal(layer.u, u)
    inner.backward(dout, dh=dh)
    dA, dB = torch.empty(5, 16, d, device="cuda"), torch.empty(5, d, 16, device="cuda")
    dx = torch.empty(T, d, device="cuda")
    L.moe_adapter_bwd(s, L.MOE_F32, dout, inner.y, w["lora_A"], w["lora_B"], w["lora_scale"], m, rng[1], u,
                      inner.dXs if cfg.Fs else None, dx, dA, dB, ws)
    assert torch.equal(g["dlora_A"], dA) and torch.equal(g["dlora_B"], dB)
    if not cfg.Fs:
        assert torch.equal(layer.dx_adapter, dx)
    for k in ("dW_gu", "dW_down", "dW_r"):
        assert torch.equal(g[k], getattr(inner, k)), k
    drop = torch.empty_like(g["dx"])
    code = L.MOE_BF16 if g["dx"].dtype == torch.bfloat16 else L.MOE_F32
    L.moe_dropout_bwd(code, code, T * d, g["dx"], 0.1, rng[0], drop)
    assert torch.equal(g["dx_drop"], drop)


@pytest.mark.gpu
def test_serving_few_and_many_tokens():
    """Forward only, row by row and by tiles, and one adapter for all of them; tokens without one get the layer's output."""
    lib()
    from token_dispatch_expert_moe_gb300 import _lib as L
    from token_dispatch_expert_moe_gb300.layer import MoELayer
    for T in (3, 64, 1024):
        cfg = dataclasses.replace(get_config("mixtral_8x22b@small"), T=T, S=0, backward=False, drop=False)
        inp = make_inputs(cfg, need_backward=False)
        w, r, _, _ = _weights(cfg, {**inp})
        ids, _ = _adapters(cfg, w, 6, 8)
        x = dev(inp["x"])
        layer = MoELayer(cfg, w, backward=False)
        plain = MoELayer(cfg, {k: v for k, v in w.items() if not k.startswith("lora")}, backward=False)
        o, p = layer.forward(x, residual=r, adapter=ids), plain.forward(x, residual=r)
        assert torch.equal(o[ids < 0], p[ids < 0]) and not torch.equal(o, p)
        want = p.float()
        for a in range(6):
            t = ids == a
            want[t] += w["lora_scale"][a] * (plain.y[t].float() @ w["lora_A"][a].float().T) @ w["lora_B"][a].float().T
        assert_close("out", host(o), host(want), "bf16")
        one = layer.forward(x, residual=r)
        every = layer.forward(x, residual=r, adapter=torch.zeros_like(ids))
        assert_close("out", host(one), host(every), "bf16")
        assert L.moe_get_status(layer.adapter_ws)[0] == 0


@pytest.mark.gpu
def test_captured_step_draws_new_masks():
    lib()
    from token_dispatch_expert_moe_gb300.layer import MoELayer
    cfg = get_config("qwen2_57b_a14b@small")
    inp = make_inputs(cfg, need_backward=True)
    w, r, dh, _ = _weights(cfg, inp)
    ids, rng = _adapters(cfg, w, 4, 24)
    x, dout = dev(inp["x"]), dev(inp["dout"])
    layer = MoELayer(cfg, w, backward=True, dropout=0.1, adapter_dropout=0.1)

    def step():
        out = layer.forward(x, residual=r, adapter=ids, rng=rng)
        g = layer.backward(dout, dh=dh)
        layer.clip_grads(1.0)
        return [out, *g.values()]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
        rng[:, 1].add_(1)
    seen = []
    for i in range(2):
        graph.replay()
        torch.cuda.synchronize()
        seen.append([t.clone() for t in outs])
    assert not torch.equal(seen[0][0], seen[1][0])
    rng.copy_(torch.tensor(SEEDS, device="cuda"))
    for i in range(2):
        got = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, seen[i]))
        rng[:, 1].add_(1)
