"""moe_balance_loss, moe_balance_loss_bwd and moe_route_bwd_add against their
formulas in 64 bits.

With u = 2^-24 and R the largest distance of a logit from its row's maximum:
the distance is rounded once (R u on exp's argument, so on p), exp is within 2
ulp, the row's sum, reciprocal and product add at most 9 u: (16 + R) 2 u on p.
prob_mean adds a chain of tokens per thread and at most 13 + 304 joins; loss is
a positive sum of the same; dlogits sums p a over the experts: (32 + 2 R) 2 u of
|a_e| + sum p |a|. Counts are exact."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.gpu_util import lib  # noqa: E402

U = 2.0 ** -24
ALPHA = 0.02


def _inputs(T, E, K, seed=0, skew=1.0):
    g = torch.Generator().manual_seed(seed)
    logits = 2 * torch.randn(T, E, generator=g) + skew * torch.randn(E, generator=g)
    return logits, logits.topk(K, dim=1).indices.int()


def _reference(logits, idx, mask, S, dloss):
    """loss, counts, prob_mean, dlogits in numpy, sub-sequence by sub-sequence, uncentred."""
    l, idx = logits.double().numpy(), idx.numpy()
    T, E = l.shape
    K = idx.shape[1]
    live = np.ones(T, bool) if mask is None else mask.numpy() != 0
    n_sub = -(-T // S)
    with np.errstate(invalid="ignore"):
        m = l.max(1, keepdims=True)
        p = np.exp(l - np.where(np.isfinite(m), m, 0))
        z = p.sum(1, keepdims=True)
        p = np.divide(p, z, out=np.zeros_like(p), where=z != 0)
    counts, prob, coef = np.zeros((n_sub, E), np.int64), np.zeros((n_sub, E)), np.zeros((T, E))
    loss, n = 0.0, live.sum()
    for j in range(n_sub):
        at = np.arange(j * S, min(T, (j + 1) * S))
        at = at[live[at]]
        if len(at) == 0:
            continue
        e = idx[at].ravel()
        counts[j] = np.bincount(e[(e >= 0) & (e < E)], minlength=E)
        prob[j] = p[at].mean(0)
        loss += ALPHA * E / K * (counts[j] * prob[j]).sum() / n
        coef[at] = ALPHA * E / K * counts[j] / (n * len(at))
    dl = np.where(live[:, None], dloss * p * (coef - (p * coef).sum(1, keepdims=True)), 0.0)
    # what the uncentred difference itself loses in 64 bits (an even load: everything but this)
    lost = 2.0 ** -50 * abs(dloss) * p * (coef + (p * coef).sum(1, keepdims=True))
    return loss, counts, prob, dl, p, live, lost


def _run(L, logits, idx, mask, S, dloss=None, stream=None, in_place=False):
    T, E = logits.shape
    K = idx.shape[1]
    shape = L.MoEShape(T=T, d=64, E=E, K=K, F=64, dtype=L.MOE_BF16, subseq_len=S)
    n_sub = -(-T // S) if S else 1
    f = lambda *n: torch.full(n, 7.0, device="cuda")  # noqa: E731
    o = dict(loss=f(2), counts=torch.full((n_sub + 1, E), 7, dtype=torch.int32, device="cuda"), prob=f(n_sub + 1, E),
             coef=f(n_sub * E + 2), dl=f(T + 1, E))
    ws = torch.full((L.moe_workspace_size(shape) + 256,), 255, dtype=torch.uint8, device="cuda")
    L.moe_clear_status(ws)
    l, i = logits.cuda(), idx.cuda()
    m = None if mask is None else mask.cuda()
    d = None if dloss is None else torch.tensor([dloss], device="cuda")
    torch.cuda.synchronize()
    L.moe_balance_loss(shape, l, i, m, ALPHA, o["loss"], o["counts"], o["prob"], o["coef"], ws, stream)
    L.moe_balance_loss_bwd(shape, l, m, o["coef"], d, l if in_place else o["dl"], stream)
    torch.cuda.synchronize()
    assert float(o["loss"][1]) == 7 and (o["counts"][-1] == 7).all() and (o["prob"][-1] == 7).all()
    assert float(o["coef"][-1]) == 7 and (o["dl"][-1] == 7).all() and (ws[-256:] == 255).all()
    rc, _ = L.moe_get_status(ws)
    return dict(loss=float(o["loss"][0]), counts=o["counts"][:-1].cpu().numpy(), prob=o["prob"][:-1].cpu().numpy(),
                dl=(l if in_place else o["dl"][:-1]).cpu().numpy(), rc=rc, n_sub=n_sub)


def _check(got, logits, idx, mask, S, dloss=1.0):
    T, E = logits.shape
    loss, counts, prob, dl, p, live, lost = _reference(logits, idx, mask, S or T, dloss)
    l = logits.double().numpy()
    fin = np.isfinite(l)
    top = np.where(fin, l, -np.inf).max(1, keepdims=True)
    R = float(np.max(np.where(fin & np.isfinite(top), top - np.where(fin, l, 0), 0), initial=0.0))
    rel_p = (16 + R) * 2 * U
    chain = min(T, S or T) + 320
    assert np.array_equal(got["counts"], counts)
    assert np.all(np.abs(got["prob"] - prob) <= (rel_p + chain * U) * prob + 1e-38)
    assert abs(got["loss"] - loss) <= (rel_p + (chain + 1100) * U) * abs(loss)
    # the centred factors: |a| of each sub-sequence
    K = idx.shape[1]
    Sx = S or T
    n = max(int(live.sum()), 1)
    a = np.zeros((T, E))
    for j in range(-(-T // Sx)):
        s = slice(j * Sx, min(T, (j + 1) * Sx))
        n_j = max(int(live[s].sum()), 1)
        a[s] = np.abs(ALPHA * (E * counts[j] - K * int(live[s].sum())) / (K * n_j * n))
    bound = 2 * (rel_p + 32 * U) * abs(dloss) * p * (a + (p * a).sum(1, keepdims=True))
    # a row whose p does not add up to one (all masked out) has p = 0 throughout
    assert np.all(np.abs(got["dl"] - dl) <= bound + lost + 1e-38)
    assert np.all(got["dl"][~live] == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("E,K", [(1, 1), (2, 1), (3, 2), (4, 2), (5, 5), (8, 2), (9, 3), (16, 8), (30, 6), (60, 4), (63, 8),
                                 (64, 8)])
@pytest.mark.parametrize("T,S", [(1, 0), (2, 1), (37, 0), (512, 0), (1000, 256), (2049, 100), (3000, 7)])
def test_loss_counts_gradients(T, S, E, K):
    L = lib()
    logits, idx = _inputs(T, E, K)
    got = _run(L, logits, idx, None, S, 1.5)
    assert got["rc"] == 0
    _check(got, logits, idx, None, S, 1.5)


@pytest.mark.gpu
@pytest.mark.parametrize("E,K", [(4, 2), (7, 3), (64, 8)])
def test_padding_is_not_read(E, K):
    """Masked tokens hold NaN logits and wild indices; a sub-sequence and the
    last token's block may be padding altogether."""
    L = lib()
    T, S = 1000, 128
    logits, idx = _inputs(T, E, K)
    mask = (torch.rand(T, generator=torch.Generator().manual_seed(3)) < 0.7).to(torch.uint8)
    mask[128:256] = 0
    mask[896:] = 0
    mask[5] = 255
    clean = _run(L, logits, idx, mask, S)
    dead = mask == 0
    logits[dead] = float("nan")
    logits[300:310][dead[300:310]] = float("inf")
    idx[dead] = 1 << 30
    got = _run(L, logits, idx, mask, S)
    assert got["rc"] == 0 and got["loss"] == clean["loss"]
    for k in ("counts", "prob", "dl"):
        assert np.array_equal(got[k], clean[k]), k
    logits[dead] = 0.0
    _check(got, logits, idx, mask, S)
    none = _run(L, logits, idx, torch.zeros(T, dtype=torch.uint8), S)
    assert none["loss"] == 0 and not none["counts"].any() and not none["prob"].any() and not none["dl"].any()


@pytest.mark.gpu
def test_masked_experts_and_extreme_logits():
    """Logits of -inf, of the type's lowest value, and rows of nothing else."""
    L = lib()
    T, E, K = 300, 12, 2
    logits, idx = _inputs(T, E, K)
    logits[:, 3] = float("-inf")
    logits[7] = torch.finfo(torch.float32).min
    logits[9] = float("-inf")
    logits[11] = 80.0
    logits[13, 2] = torch.finfo(torch.float32).max
    got = _run(L, logits, idx, None, 64)
    loss, counts, prob, dl, p, _, _ = _reference(logits, idx, None, 64, 1.0)
    assert np.array_equal(got["counts"], counts)
    assert np.allclose(got["prob"], prob, rtol=1e-5, atol=1e-30) and np.isfinite(got["dl"]).all()
    assert abs(got["loss"] - loss) <= 1e-5 * loss
    assert not got["dl"][9].any() and not got["dl"][torch.isneginf(logits).numpy()].any()
    # one NaN logit spoils its own row's gradient and the loss, not the other rows' gradients
    logits[20, 1] = float("nan")
    bad = _run(L, logits, idx, None, 64)
    assert np.isnan(bad["loss"]) and np.isnan(bad["dl"][20]).all()
    keep = np.arange(T) != 20
    assert np.array_equal(bad["dl"][keep], got["dl"][keep])


@pytest.mark.gpu
def test_index_out_of_range_is_reported():
    L = lib()
    logits, idx = _inputs(100, 8, 2)
    idx[4, 1] = 8
    idx[5, 0] = -1
    got = _run(L, logits, idx, None, 0)
    _, counts, _, _, _, _, _ = _reference(logits, idx, None, 100, 1.0)
    assert got["rc"] == 5 and np.array_equal(got["counts"], counts) and counts.sum() == 198


@pytest.mark.gpu
def test_in_place_repeatable_stream_and_graph():
    L = lib()
    T, E, K, S = 5000, 64, 8, 512
    logits, idx = _inputs(T, E, K)
    a, b = _run(L, logits, idx, None, S), _run(L, logits, idx, None, S, in_place=True)
    c = _run(L, logits, idx, None, S, stream=torch.cuda.Stream())
    for o in (b, c):
        assert o["loss"] == a["loss"] and np.array_equal(o["dl"], a["dl"]) and np.array_equal(o["prob"], a["prob"])
    shape = L.MoEShape(T=T, d=64, E=E, K=K, F=64, dtype=L.MOE_BF16, subseq_len=S)
    ws = torch.zeros(L.moe_workspace_size(shape), dtype=torch.uint8, device="cuda")
    l, i = logits.cuda(), idx.cuda()
    n_sub = -(-T // S)
    loss, counts = torch.zeros(1, device="cuda"), torch.zeros(n_sub, E, dtype=torch.int32, device="cuda")
    coef, dl = torch.zeros(n_sub * E + 1, device="cuda"), torch.zeros(T, E, device="cuda")

    def step():
        L.moe_balance_loss(shape, l, i, None, ALPHA, loss, counts, None, coef, ws)   # no prob_mean asked for
        L.moe_balance_loss_bwd(shape, l, None, coef, None, dl)

    step()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]   # they share the workspace, and run in turn
    for g in graphs:
        with torch.cuda.graph(g):
            step()
    l2, i2 = _inputs(T, E, K, seed=8)
    l.copy_(l2), i.copy_(i2)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    want = _run(L, l2, i2, None, S)
    assert float(loss) == want["loss"] and np.array_equal(dl.cpu().numpy(), want["dl"])


@pytest.mark.gpu
def test_gradient_against_differences():
    L = lib()
    T, E, K, S = 40, 6, 2, 16
    logits, idx = _inputs(T, E, K)
    got = _run(L, logits, idx, None, S, 2.0)
    step = 1e-4
    for t, e in ((0, 0), (15, 3), (39, 5)):
        lo, hi = logits.double().clone(), logits.double().clone()
        lo[t, e] -= step
        hi[t, e] += step
        num = 2.0 * (_reference(hi, idx, None, S, 1.0)[0] - _reference(lo, idx, None, S, 1.0)[0]) / (2 * step)
        assert abs(num - got["dl"][t, e]) <= 1e-7


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [("bf16", 512), ("bf16", 192), ("f32", 64)])
def test_route_bwd_add(dtype, d):
    """route_bwd_add(g) - route_bwd = the router's products with g: dx_router
    gains g W_r, dW_r gains g^T x, db_r gains the column sums; with g = 0 it is
    route_bwd bit for bit."""
    L = lib()
    T, E, K = 333, 8, 2
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, W = r(T, d).to(dt), (r(E, d) / d ** 0.5).to(dt)
    logits = (x.float() @ W.float().T)
    p, idx = torch.softmax(logits, 1).topk(K, dim=1)
    w = p / p.sum(1, keepdim=True)
    dw, g = r(T, K), 0.1 * r(T, E)
    shape = L.MoEShape(T=T, d=d, E=E, K=K, F=64, dtype=L.MOE_BF16 if dtype == "bf16" else L.MOE_F32, renorm=1)
    ws = torch.zeros(L.moe_workspace_size(shape), dtype=torch.uint8, device="cuda")
    dv = [t.cuda() for t in (x, W, logits, idx.int(), p, w, dw)]

    def run(add):
        o = [torch.empty(E, d, device="cuda"), torch.empty(E, device="cuda"), torch.empty(T, d, device="cuda")]
        args = (shape, dv[0], dv[1], None, dv[2], dv[3], dv[4], dv[5], dv[6], None)
        if add is None:
            L.moe_route_bwd(*args, None, o[0], o[1], None, o[2], ws)
        else:
            L.moe_route_bwd_add(*args, add.cuda(), None, o[0], o[1], None, o[2], ws)
        torch.cuda.synchronize()
        return [t.cpu().double() for t in o]

    base, zero, full = run(None), run(torch.zeros(T, E)), run(g)
    assert all(torch.equal(a, b) for a, b in zip(base, zero))
    xd, Wd, gd = x.double(), W.double(), g.double()
    for got, b, add in zip(full, base, (gd.T @ xd, gd.sum(0), gd @ Wd)):
        # fp32 sums over at most T + E terms on either side
        assert (got - b - add).norm() <= 1e-5 * (add.norm() + b.norm())
