"""moe_rmsnorm and moe_rmsnorm_bwd against their formulas in 64 bits.

Bounds, derived from the arithmetic (u = 2^-24, one fp32 rounding):
  rstd   the squares are positive, a thread adds at most 32 of them in a chain
         and a tree of at most 10 + 5 levels joins the threads: 48 u on the
         sum, with the mean, eps and the root's own rounding 52 u on rstd;
  y      two more products and one rounding to the type (2^-8 bf16, u fp32);
  scale  the largest |y|, and a division: 60 u;
  q s    half an e4m3 step of y: 2^-4 |y|, below the normal range 2^-10 s;
  dx     the same depths on sums of either sign: 64 u of the sum of magnitudes;
  dgamma rows added in a chain per CTA, then at most 1024 partial sums in
         chains of 32: u (rows / CTAs + 80) of the sum of magnitudes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.gpu_util import lib  # noqa: E402

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
EPS = 1e-5


def _rows(rows, d, dt, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, d, generator=g) * scale).to(dt)


def _guarded(rows, d, dt, fill=7.0):
    """A [rows, d] view with a row of sentinels on both sides."""
    b = torch.full((rows + 2, d), fill, device="cuda").to(dt)
    return b, b[1:rows + 1]


def _intact(b, fill=7.0):
    want = torch.full_like(b[0].float(), fill).to(b.dtype).float()
    return torch.equal(b[0].float(), want) and torch.equal(b[-1].float(), want)


def _code(L, dt):
    return L.MOE_BF16 if dt == torch.bfloat16 else L.MOE_F32


def _forward(L, x, r, gamma, group=None, y=True, h=True, stream=None):
    rows, d = x.shape
    dt = x.dtype
    out = {"rstd": torch.full((rows,), -1.0, device="cuda")}
    raw = {}
    if h:
        raw["h"], out["h"] = _guarded(rows, d, dt)
    if y:
        raw["y"], out["y"] = _guarded(rows, d, dt)
    if group is not None:
        ng = 1 if group == 0 else -(-d // group)
        raw["q"], out["q"] = _guarded(rows, d, torch.float8_e4m3fn)
        raw["s"], out["s"] = _guarded(rows, ng, torch.float32)
        if out["q"].data_ptr() % 16:   # rows of 8 (mod 16) bytes: no sentinels in front
            del raw["q"]
            out["q"] = torch.zeros(rows, d, dtype=torch.float8_e4m3fn, device="cuda")
    L.moe_rmsnorm(_code(L, dt), rows, d, x, r, gamma, EPS, out.get("h"), out.get("y"), out.get("q"),
                  out.get("s"), group or 0, out["rstd"], stream)
    torch.cuda.synchronize()
    for k, b in raw.items():
        assert _intact(b), k
    return out


def _check_forward(x, r, gamma, out, group, eps=EPS):
    dt, d = x.dtype, x.shape[1]
    h = x if r is None else (x.float() + r.float()).to(dt)
    if "h" in out:
        assert torch.equal(out["h"].cpu(), h)
    h = h.double()
    rstd = 1.0 / torch.sqrt(h.square().mean(1) + eps)
    assert ((out["rstd"].cpu().double() - rstd).abs() <= 52 * U * rstd).all()
    y = h * rstd[:, None] * gamma.double()
    tiny = 2.0 ** -126
    if "y" in out:
        assert ((out["y"].cpu().double() - y).abs() <= (HALF[dt] + 56 * U) * y.abs() + tiny).all()
    if group is None:
        return
    g = group or d
    ng = -(-d // g)
    q, s = out["q"].float().cpu().double(), out["s"].cpu().double()
    yg = torch.nn.functional.pad(y, (0, ng * g - d)).view(-1, ng, g)
    amax = yg.abs().amax(2)
    want = torch.where(amax > 0, amax.clamp_min(2.0 ** -110) / 448, torch.ones_like(amax))
    assert ((s - want).abs() <= 60 * U * want).all()
    se = s.repeat_interleave(g, 1)[:, :d]
    bound = torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * se) * (1 + 1e-5)
    assert ((q * se - y).abs() <= bound).all()


# rows x d: one token to several, every register layout's edges, rows that fill no warp
SHAPES = [(1, 8), (3, 64), (5, 256), (7, 264), (2, 512), (33, 520), (4, 1024), (3, 1032), (9, 2048), (5, 3584),
          (2, 4096), (3, 4104), (2, 6144), (17, 8192), (1, 16384), (2, 32768), (1000, 72)]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_forward(rows, d, dt):
    L = lib()
    if dt == torch.float32:
        if d == 32768:
            d = 16384
        d += 4 if d in (8, 264, 1032) else 0   # a multiple of 4 alone
    x, r = _rows(rows, d, dt, 1, 3.0), _rows(rows, d, dt, 2)
    gamma = (1 + 0.3 * _rows(1, d, torch.float32, 3)[0]).to(dt)
    xd, rd, gd = x.cuda(), r.cuda(), gamma.cuda()
    for res, rr in ((rd, r), (None, None)):
        for group in (None, 0, 32, 64, 128):
            out = _forward(L, xd, res, gd, group)
            _check_forward(x, rr, gamma, out, group)


@pytest.mark.gpu
def test_outputs_alone_and_in_place():
    L = lib()
    dt = torch.bfloat16
    x, r, gamma = _rows(37, 1032, dt, 1), _rows(37, 1032, dt, 2), _rows(1, 1032, dt, 3)[0]
    full = _forward(L, x.cuda(), r.cuda(), gamma.cuda(), 64)
    only_q = _forward(L, x.cuda(), r.cuda(), gamma.cuda(), 64, y=False, h=False)
    for k in ("rstd", "q", "s"):
        assert torch.equal(only_q[k].float(), full[k].float()), k
    # h in the residual's place, y in x's
    a, b = x.cuda(), r.cuda()
    L.moe_rmsnorm(L.MOE_BF16, 37, 1032, a, b, gamma.cuda(), EPS, b, a, None, None, 0, None)
    assert torch.equal(b, full["h"]) and torch.equal(a, full["y"])
    # x as its own residual, and the other way round in place
    twice = _forward(L, x.cuda(), x.cuda(), gamma.cuda())
    a = x.cuda()
    L.moe_rmsnorm(L.MOE_BF16, 37, 1032, a, a, gamma.cuda(), EPS, a, None, None, None, 0, None)
    assert torch.equal(a, twice["h"])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 1024, 4096])
def test_special_rows_spoil_only_themselves(d):
    """A row of zeros, one of the smallest numbers, one with an infinity, one
    with a NaN, a group of zeros: the other rows are as without them."""
    L = lib()
    dt = torch.float32
    x = _rows(8, d, dt, 1)
    clean = _forward(L, x.cuda(), None, torch.ones(d).cuda(), 32)
    x[1] = 0
    x[2] = 1e-38
    x[3, 5] = float("inf")
    x[4, 6] = float("nan")
    x[5, 32:64] = 0
    x[6] *= 1e17
    gamma = torch.ones(d)
    out = _forward(L, x.cuda(), None, gamma.cuda(), 32)
    for i in (0, 7):
        for k in ("rstd", "y", "q", "s"):
            assert torch.equal(out[k][i].float(), clean[k][i].float()), (k, i)
    for i in (1, 2, 5, 6):
        one = {k: v[i:i + 1] for k, v in out.items()}
        if i != 2:
            _check_forward(x[i:i + 1], None, gamma, one, 32)
        assert all(torch.isfinite(v.float()).all() for v in one.values()), i
    assert (out["s"][1] == 1).all() and (out["q"][1].float() == 0).all() and out["s"][5, 1] == 1
    assert not torch.isfinite(out["y"][3]).all() and not torch.isfinite(out["y"][4]).all()


def _backward(L, dy, h, gamma, rstd, dh, dx_dt, dx=None, ws=None):
    rows, d = h.shape
    dt = h.dtype
    raw, view = _guarded(rows, d, dx_dt)
    dx = view if dx is None else dx
    dgamma = torch.full((d + 8,), 7.0, device="cuda")
    if ws is None:
        ws = torch.full((L.moe_rmsnorm_bwd_workspace_size(rows, d),), 255, dtype=torch.uint8, device="cuda")
    L.moe_rmsnorm_bwd(_code(L, dt), _code(L, dy.dtype), _code(L, dx_dt), rows, d, dy, h, gamma, rstd,
                      dh, dx, dgamma[:d], ws)
    torch.cuda.synchronize()
    assert _intact(raw) and (dgamma[d:] == 7).all()
    return dx, dgamma[:d]


def _reference_bwd(dy, h, gamma, rstd, dh):
    """dx, dgamma in 64 bits, and the magnitudes that their roundings go by."""
    dy, h, gamma, r = dy.double(), h.double(), gamma.double(), rstd.double()[:, None]
    xh, g = h * r, dy * gamma
    m = (g * xh).mean(1, keepdim=True)
    dx = r * (g - xh * m)
    mag = r * (g.abs() + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    if dh is not None:
        dx, mag = dx + dh.double(), mag + dh.double().abs()
    return dx, mag, (dy * xh).sum(0), (dy * xh).abs().sum(0)


BWD_TYPES = [(torch.float32, torch.float32, torch.float32), (torch.bfloat16, torch.float32, torch.float32),
             (torch.bfloat16, torch.float32, torch.bfloat16), (torch.bfloat16, torch.bfloat16, torch.float32),
             (torch.bfloat16, torch.bfloat16, torch.bfloat16)]


@pytest.mark.gpu
@pytest.mark.parametrize("types", BWD_TYPES, ids=lambda t: "-".join(str(x)[6:] for x in t))
@pytest.mark.parametrize("rows,d", [(1, 8), (3, 72), (700, 256), (33, 1032), (305, 2048), (5, 3584), (400, 4104),
                                    (2, 8192), (37, 8200), (200, 12288), (3, 16384), (90, 16392),
                                    (1, 32768), (77, 32768)])
def test_backward(rows, d, types):
    L = lib()
    dt, dy_dt, dx_dt = types
    if dt == torch.float32:
        d = min(d, 16384)
        d += 4 if d in (8, 72, 1032, 4104, 8200) else 0
    h, dy, dh = _rows(rows, d, dt, 1, 2.0), _rows(rows, d, dy_dt, 2, 0.3), _rows(rows, d, dt, 3, 0.3)
    gamma = (1 + 0.3 * _rows(1, d, torch.float32, 4)[0]).to(dt)
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    for use_dh in (True, False):
        dx, dgamma = _backward(L, dy.cuda(), h.cuda(), gamma.cuda(), rstd.cuda(), dh.cuda() if use_dh else None, dx_dt)
        ref, mag, gref, gmag = _reference_bwd(dy, h, gamma, rstd, dh if use_dh else None)
        assert ((dx.cpu().double() - ref).abs() <= 64 * U * mag + HALF[dx_dt] * (ref.abs() + 64 * U * mag)).all()
        assert ((dgamma.cpu().double() - gref).abs() <= U * (rows / 100 + 80) * gmag).all()


@pytest.mark.gpu
def test_backward_against_differences():
    """The gradients of sum(dy y) + sum(dh h) by central differences of the
    64-bit forward at a few places."""
    L = lib()
    rows, d = 4, 64
    h, dy, dh = (_rows(rows, d, torch.float32, k) for k in (1, 2, 3))
    gamma = 1 + 0.3 * _rows(1, d, torch.float32, 4)[0]
    rstd = torch.rsqrt(h.square().mean(1) + EPS)
    dx, dgamma = _backward(L, dy.cuda(), h.cuda(), gamma.cuda(), rstd.cuda(), dh.cuda(), torch.float32)

    def f(h, gamma):
        y = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * gamma
        return float((dy.double() * y).sum() + (dh.double() * h).sum())

    step = 1e-5   # second differences cancel: error step^2 f''' and 1e-16 |f| / step, both under 1e-8
    for i, j in ((0, 0), (1, 17), (3, 63)):
        e = torch.zeros(rows, d, dtype=torch.float64)
        e[i, j] = step
        num = (f(h.double() + e, gamma.double()) - f(h.double() - e, gamma.double())) / (2 * step)
        assert abs(num - float(dx[i, j])) <= 1e-5 * max(1.0, abs(num))
    for j in (0, 31):
        e = torch.zeros(d, dtype=torch.float64)
        e[j] = step
        num = (f(h.double(), gamma.double() + e) - f(h.double(), gamma.double() - e)) / (2 * step)
        assert abs(num - float(dgamma[j])) <= 1e-5 * max(1.0, abs(num))


@pytest.mark.gpu
def test_backward_in_place_repeatable_and_empty():
    L = lib()
    rows, d = 513, 520
    h, dh = _rows(rows, d, torch.bfloat16, 1).cuda(), _rows(rows, d, torch.bfloat16, 2).cuda()
    dy, gamma = _rows(rows, d, torch.float32, 3).cuda(), _rows(1, d, torch.bfloat16, 4)[0].cuda()
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    dx, dg = _backward(L, dy, h, gamma, rstd, dh, torch.float32)
    dx2, dg2 = _backward(L, dy, h, gamma, rstd, dh, torch.float32)
    assert torch.equal(dx, dx2) and torch.equal(dg, dg2)
    a = dy.clone()
    _, dg3 = _backward(L, a, h, gamma, rstd, dh, torch.float32, dx=a)     # dx in dy's place
    assert torch.equal(a, dx) and torch.equal(dg3, dg)
    b = dh.clone()
    dxb, _ = _backward(L, dy, h, gamma, rstd, dh, torch.bfloat16)
    _backward(L, dy, h, gamma, rstd, b, torch.bfloat16, dx=b)            # in dh's place
    assert torch.equal(b, dxb)
    # no rows: dgamma is zero, the rest is not touched
    dgamma = torch.full((d,), 7.0, device="cuda")
    L.moe_rmsnorm_bwd(L.MOE_BF16, 0, 0, 0, d, None, None, None, None, None, None, dgamma, None, ws_bytes=0)
    L.moe_rmsnorm(L.MOE_BF16, 0, d, None, None, None, EPS, dx, None, None, None, 0, None)
    torch.cuda.synchronize()
    assert (dgamma == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [256, 1024, 4096, 16384, 32768])   # each kernel of the backward
def test_on_another_stream_and_captured(d):
    """On a side stream, and in two graphs that share the workspace and are
    replayed one after the other with new contents."""
    L = lib()
    rows = 65
    dt = torch.bfloat16
    x, gamma = _rows(rows, d, dt, 1).cuda(), _rows(1, d, dt, 2)[0].cuda()
    dy, dh = _rows(rows, d, torch.float32, 3).cuda(), _rows(rows, d, dt, 4).cuda()
    y, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    q = torch.empty(rows, d, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(rows, d // 128, device="cuda")
    dx, dg = torch.empty(rows, d, device="cuda"), torch.empty(d, device="cuda")
    ws = torch.empty(L.moe_rmsnorm_bwd_workspace_size(rows, d), dtype=torch.uint8, device="cuda")

    def step(stream=None):
        L.moe_rmsnorm(L.MOE_BF16, rows, d, x, None, gamma, EPS, None, y, q, s, 128, rstd, stream)
        L.moe_rmsnorm_bwd(L.MOE_BF16, 0, 0, rows, d, dy, x, gamma, rstd, dh, dx, dg, ws, stream)

    def results():
        torch.cuda.synchronize()
        return [t.float().clone() for t in (y, q, s, rstd, dx, dg)]

    step()
    first = results()
    side = torch.cuda.Stream()
    for t in (y, rstd, dx, dg):
        t.zero_()
    torch.cuda.synchronize()
    step(side)
    assert all(torch.equal(a, b) for a, b in zip(results(), first))
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            step()
    x.copy_(_rows(rows, d, dt, 9))
    graphs[0].replay()
    graphs[1].replay()
    again = results()
    step()
    assert all(torch.equal(a, b) for a, b in zip(results(), again))
    assert not torch.equal(again[0], first[0])
