"""The operators around the layer where element offsets pass 32 bits, and in
calls that run at the same time: the far rows equal the same rows of a small
call, bit for bit."""
import pytest

torch = pytest.importorskip("torch")

from tests.gpu_util import lib  # noqa: E402

B16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _seeded():
    torch.manual_seed(0)
    yield
    torch.cuda.empty_cache()


def _norm(L, x, r, gamma):
    rows, d = x.shape
    o = dict(h=torch.empty_like(x), y=torch.empty_like(x), q=torch.empty(rows, d, dtype=torch.float8_e4m3fn, device="cuda"),
             s=torch.empty(rows, -(-d // 128), device="cuda"), rstd=torch.empty(rows, device="cuda"))
    L.moe_rmsnorm(L.MOE_BF16, rows, d, x, r, gamma, 1e-6, o["h"], o["y"], o["q"], o["s"], 128, o["rstd"])
    return o


@pytest.mark.gpu
@pytest.mark.parametrize("d", [256, 8192])
def test_norm_and_its_backward_beyond_32_bits(d):
    L = lib()
    rows = 2 ** 31 // d + 300
    x, gamma = torch.randn(rows, d, device="cuda", dtype=B16), torch.randn(d, device="cuda").to(B16)
    far = torch.tensor([0, 1, rows // 2, rows - 300, rows - 2, rows - 1], device="cuda")
    o = _norm(L, x, x, gamma)
    small = _norm(L, x[far], x[far], gamma)
    for k in o:
        assert torch.equal(o[k].view(torch.uint8)[far], small[k].view(torch.uint8)) if k != "rstd" else torch.equal(
            o[k][far], small[k]), k
    dx, dg = torch.empty_like(x), torch.empty(d, device="cuda")
    ws = torch.empty(L.moe_rmsnorm_bwd_workspace_size(rows, d), dtype=torch.uint8, device="cuda")
    L.moe_rmsnorm_bwd(1, 1, 1, rows, d, o["y"], o["h"], gamma, o["rstd"], x, dx, dg, ws)
    dxs, dgs = torch.empty_like(x[far]), torch.empty(d, device="cuda")
    L.moe_rmsnorm_bwd(1, 1, 1, len(far), d, small["y"], small["h"], gamma, small["rstd"], x[far], dxs, dgs, ws)
    assert torch.equal(dx[far], dxs)
    # dgamma over all rows: 64-bit sums block by block; a thread adds up to rows / 456 products in a chain
    ref, mag = torch.zeros(d, dtype=torch.float64, device="cuda"), torch.zeros(d, dtype=torch.float64, device="cuda")
    for lo in range(0, rows, 1 << 16):
        t = o["y"][lo:lo + (1 << 16)].double() * (o["h"][lo:lo + (1 << 16)].double() * o["rstd"][lo:lo + (1 << 16), None].double())
        ref += t.sum(0)
        mag += t.abs().sum(0)
    assert ((dg.double() - ref).abs() <= 2.0 ** -24 * (rows / 100 + 80) * mag).all()


@pytest.mark.gpu
def test_permute_e4m3_beyond_32_bits():
    L = lib()
    T, d, E, K = 34000, 8192, 8, 8   # 2.2e9 elements of Xp
    q = torch.randn(T, d, device="cuda").to(torch.float8_e4m3fn)
    s = torch.rand(T, d // 128, device="cuda")
    idx = torch.rand(T, E, device="cuda").argsort(1).int().contiguous()
    keep = torch.ones(T, K, dtype=torch.uint8, device="cuda")
    shape = L.MoEShape(T=T, d=d, E=E, K=K, F=64, dtype=L.MOE_BF16)
    ws = torch.zeros(L.moe_workspace_size(shape), dtype=torch.uint8, device="cuda")
    i = lambda *n: torch.empty(*n, dtype=torch.int32, device="cuda")  # noqa: E731
    Xp, row_of, src_of, counts, offsets = torch.empty(T * K, d, dtype=B16, device="cuda"), i(T, K), i(T * K), i(E), i(E + 1)
    L.moe_permute_e4m3(shape, q, s, 128, idx, keep, Xp, row_of, src_of, counts, offsets, ws)
    assert L.moe_get_status(ws)[0] == 0 and (counts == T).all()
    rows = torch.tensor([0, T * K // 2, T * K - T, T * K - 1], device="cuda")
    t = (src_of[rows] // K).long()
    want = (q[t].float() * s[t].repeat_interleave(128, 1)).to(B16)
    assert torch.equal(Xp[rows], want) and torch.equal(row_of.view(-1)[src_of[rows].long()].long(), rows)


@pytest.mark.gpu
def test_balance_beyond_32_bits():
    L = lib()
    T, E, K, S = 2 ** 25 + 100, 64, 1, 4096
    logits = torch.randn(T, E, device="cuda")
    idx = logits.argmax(1, keepdim=True).int()
    shape = L.MoEShape(T=T, d=8, E=E, K=K, F=64, dtype=L.MOE_BF16, subseq_len=S)
    n_sub = -(-T // S)
    ws = torch.zeros(L.moe_workspace_size(shape), dtype=torch.uint8, device="cuda")
    loss, counts = torch.empty(1, device="cuda"), torch.empty(n_sub, E, dtype=torch.int32, device="cuda")
    prob, coef, dl = torch.empty(n_sub, E, device="cuda"), torch.empty(n_sub * E + 1, device="cuda"), torch.empty_like(logits)
    L.moe_balance_loss(shape, logits, idx, None, 1.0, loss, counts, prob, coef, ws)
    L.moe_balance_loss_bwd(shape, logits, None, coef, None, dl)
    assert L.moe_get_status(ws)[0] == 0 and int(counts.sum()) == T
    # u = 2^-24, logits within R = 12 of their row's largest: p is (16 + R) 2 u off; a thread adds 32 tokens and 20
    # more joins follow: below 110 u on prob, and the loss adds 20 more. dlogits: (32 + 2 R) 2 u of |a| + sum p |a|.
    u = 2.0 ** -24
    assert float((logits.max(1).values - logits.min(1).values).max()) < 12
    for j in (0, n_sub // 2, n_sub - 1):   # the last one has 100 tokens
        at = slice(j * S, min(T, (j + 1) * S))
        p = torch.softmax(logits[at].double(), 1)
        n = p.shape[0]
        c = torch.bincount(idx[at].view(-1).long(), minlength=E)
        assert torch.equal(counts[j].long(), c)
        assert ((prob[j].double() - p.mean(0)).abs() <= 110 * u * p.mean(0)).all()
        a = (E * c - K * n).double() / (K * n)
        ref = p * (a - (p * a).sum(1, keepdim=True)) / T
        assert ((dl[at].double() - ref).abs() <= 112 * u * p * (a.abs() + (p * a.abs()).sum(1, keepdim=True)) / T).all()
    want = (counts.double() * prob.double()).sum() * E / (K * T)
    assert abs(float(loss) - float(want)) <= 130 * u * float(want)


@pytest.mark.gpu
def test_calls_at_the_same_time():
    """Two streams, each with its own workspace and outputs, many calls in
    flight: as one after the other."""
    L = lib()
    rows, d, T, E, K = 3000, 4104, 16384, 64, 8
    gen = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda *s, dt=torch.float32: torch.randn(*s, device="cuda", generator=gen).to(dt)  # noqa: E731
    sides = []
    for _ in range(2):
        x, gamma, dy, dh = randn(rows, d, dt=B16), randn(d, dt=B16), randn(rows, d), randn(rows, d, dt=B16)
        logits = randn(T, E)
        idx = logits.topk(K, dim=1).indices.int()
        grads = [randn(n) for n in (5_000_000, 333, 77_777)]
        sides.append(dict(x=x, gamma=gamma, dy=dy, dh=dh, logits=logits, idx=idx, grads=L.TensorList(grads)))
    shape = L.MoEShape(T=T, d=64, E=E, K=K, F=64, dtype=L.MOE_BF16, subseq_len=2048)

    def outputs():
        f = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        return dict(y=f(rows, d, dt=B16), rstd=f(rows), dx=f(rows, d), dg=f(d), loss=f(1), counts=f(8, E, dt=torch.int32),
                    coef=f(8 * E + 1), dl=f(T, E), norm=f(1),
                    ws=f(L.moe_rmsnorm_bwd_workspace_size(rows, d), dt=torch.uint8),
                    ws2=f(L.moe_workspace_size(shape), dt=torch.uint8), ws3=f(L.MOE_GRAD_NORM_WORKSPACE_BYTES, dt=torch.uint8))

    def calls(s, o, stream):
        L.moe_rmsnorm(1, rows, d, s["x"], None, s["gamma"], 1e-6, None, o["y"], None, None, 0, o["rstd"], stream)
        L.moe_balance_loss(shape, s["logits"], s["idx"], None, 0.1, o["loss"], o["counts"], None, o["coef"], o["ws2"], stream)
        L.moe_rmsnorm_bwd(1, 0, 0, rows, d, s["dy"], s["x"], s["gamma"], o["rstd"], s["dh"], o["dx"], o["dg"], o["ws"], stream)
        L.moe_grad_norm(s["grads"], o["norm"], o["ws3"], stream)
        L.moe_balance_loss_bwd(shape, s["logits"], None, o["coef"], None, o["dl"], stream)

    alone, both = [outputs() for _ in range(2)], [outputs() for _ in range(2)]
    for s, o in zip(sides, alone):
        calls(s, o, None)
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for s, o, st in zip(sides, both, streams):
            calls(s, o, st)
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        for k in ("y", "rstd", "dx", "dg", "loss", "counts", "coef", "dl", "norm"):
            assert torch.equal(a[k], b[k]), k
