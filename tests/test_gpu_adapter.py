"""Low-rank adapters chosen per token, forward and backward, against the
formulas in 64 bits with derived bounds."""
import pytest

torch = pytest.importorskip("torch")

from tests.adapter_util import backward, forward, rng_tensor, within  # noqa: E402
from tests.gpu_util import lib  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16
SEED, OFFSET = 2 ** 63 + 99, 2 ** 40 + 3


class Batch:
    """A shape, its tensors and its adapters' indices; everything that the calls write starts as NaN."""

    def __init__(self, T, d_in, d_out, n, rank, dt, p=0.0, bare=0.2, ids=None, seed=0, scaled=True, wide=0):
        self.L = L = lib()
        g = torch.Generator(device="cuda").manual_seed(seed + 1000 * T + rank)
        randn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.p, self.dt, self.T = p, dt, T
        ld = [d + wide for d in (d_in, d_out)]   # rows as slices of wider matrices

        def rows(d, i):
            return randn(T, ld[i]).to(dt)[:, wide // 2:wide // 2 + d]

        self.x, self.dy, self.base = rows(d_in, 0), rows(d_out, 1), rows(d_out, 1)
        self.A = (randn(n, rank, d_in) / d_in ** 0.5).to(dt)
        self.B = (randn(n, d_out, rank) / rank ** 0.5).to(dt)
        self.scale = torch.rand(n, device="cuda", generator=g) + 0.5 if scaled else None
        if ids is None:
            ids = torch.randint(0, n, (T,), device="cuda", generator=g)
            ids[torch.rand(T, device="cuda", generator=g) < bare] = -1
        self.ids = ids.int().cuda()
        self.rng = rng_tensor(SEED, OFFSET)
        self.shape = L.MoEAdapterShape(T=T, d_in=d_in, d_out=d_out, n=n, rank=rank,
                                       dtype=L.MOE_BF16 if dt == BF16 else L.MOE_F32, dropout=p,
                                       ld_in=ld[0] if wide else 0, ld_out=ld[1] if wide else 0)
        self.ws = torch.zeros(L.moe_adapter_workspace_size(self.shape), dtype=torch.uint8, device="cuda")
        self.map = torch.zeros(L.moe_adapter_map_size(self.shape), dtype=torch.uint8, device="cuda")
        L.moe_adapter_map(self.shape, self.ids, self.map, self.ws)
        self.u = torch.randn(T, rank, device="cuda", generator=g)
        self.u[self.ids < 0] = 0

    def new(self, *s, dt=F32):
        return torch.full(s, float("nan"), dtype=dt, device="cuda")

    def forward(self, rowwise=False, base=True, ids=True):
        y = torch.full_like(self.base, float("nan")) if self.shape.ld_out == 0 else \
            self.new(self.T, self.shape.ld_out, dt=self.dt)[:, :self.shape.d_out]
        u = self.new(self.T, self.shape.rank)
        self.L.moe_adapter(self.shape, self.x, self.A, self.B, self.scale, self.ids if ids else None,
                           None if rowwise else self.map, self.rng if self.p else None, self.base if base else None, y, u,
                           self.ws)
        assert self.status() == 0
        return y, u

    def backward(self, dx_t=F32, dx_in=None, map=True):
        dx, dA, dB = self.new(self.T, self.shape.d_in, dt=dx_t), self.new(*self.A.shape), self.new(*self.B.shape)
        self.L.moe_adapter_bwd(self.shape, self.L.MOE_BF16 if dx_t == BF16 else self.L.MOE_F32, self.dy, self.x, self.A,
                               self.B, self.scale, self.map if map else None, self.rng if self.p else None, self.u, dx_in, dx,
                               dA, dB, self.ws)
        assert self.status() == 0
        return {"dx": dx, "dA": dA, "dB": dB}

    def status(self):
        return self.L.moe_get_status(self.ws)[0]

    def check_forward(self, **kw):
        y, u = self.forward(**kw)
        ids = self.ids if kw.get("ids", True) else torch.zeros_like(self.ids)
        wy, by, wu, bu = forward(self.x, self.A, self.B, self.scale, ids, self.base if kw.get("base", True) else None,
                                 self.p, SEED, OFFSET)
        within("u", u, wu, bu)
        within("y", y, wy, by)
        bare = ids < 0
        if kw.get("base", True):
            assert torch.equal(y[bare], self.base[bare])
        return y, u

    def check_backward(self, dx_t=F32, dx_in=True, map=True):
        g = torch.randn(self.T, self.shape.d_in, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(dx_t)
        got = self.backward(dx_t, g if dx_in else None, map)
        ids = self.ids if map else torch.zeros_like(self.ids)
        want, bound = backward(self.dy, self.x, self.A, self.B, self.scale, ids, self.u, g if dx_in else None, dx_t, self.p,
                               SEED, OFFSET)
        for k in want:
            within(k, got[k], want[k], bound[k])
        return got


# T, d_in, d_out, n, rank
SHAPES = [(1, 8, 8, 1, 8), (1, 512, 264, 5, 16), (2, 72, 1024, 3, 24), (127, 200, 136, 2, 8), (128, 64, 64, 1, 16),
          (129, 1032, 72, 3, 40), (300, 256, 520, 70, 32), (700, 648, 392, 4, 64), (1021, 384, 640, 12, 128),
          (1500, 136, 264, 1, 72), (2300, 264, 200, 3, 120), (517, 2056, 1544, 600, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_forward(shape, dt, p):
    b = Batch(*shape, dt, p)
    b.check_forward()
    b.check_forward(rowwise=True)
    b.check_forward(base=False)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dt,dx_t", [(BF16, BF16), (BF16, F32), (F32, F32)], ids=["bf16", "bf16-f32", "f32"])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_backward(shape, dt, dx_t, p):
    b = Batch(*shape, dt, p)
    b.check_backward(dx_t)
    b.check_backward(dx_t, dx_in=False)


@pytest.mark.gpu
@pytest.mark.parametrize("rank", [4, 12, 36, 100])
def test_f32_ranks_of_four(rank):
    b = Batch(300, 68, 76, 3, rank, F32, 0.2)
    b.check_forward()
    b.check_forward(rowwise=True)
    b.check_backward()


@pytest.mark.gpu
@pytest.mark.parametrize("dt,rank", [(BF16, 16), (BF16, 88), (F32, 20)])
def test_slices_of_wider_matrices(dt, rank):
    """Rows further apart than they are wide; what lies between them stays."""
    b = Batch(333, 200, 264, 5, rank, dt, 0.1, wide=48)
    for rowwise in (False, True):
        b.check_forward(rowwise=rowwise)
    b.check_backward(F32)
    L, wide = b.L, torch.full((333, 512), 7.0, dtype=dt, device="cuda")
    b.shape.ld_out = 512
    y = wide[:, 128:128 + 264]
    L.moe_adapter(b.shape, b.x, b.A, b.B, b.scale, None, b.map, b.rng, None, y, None, b.ws)
    wy, by, _, _ = forward(b.x, b.A, b.B, b.scale, b.ids, None, 0.1, SEED, OFFSET)
    within("y", y, wy, by)
    assert bool((wide[:, :128] == 7).all()) and bool((wide[:, 392:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dt,shape", [(BF16, (700, 264, 136, 1, 16)), (BF16, (33, 264, 136, 2, 64)), (F32, (300, 64, 72, 1, 12))])
def test_one_adapter_without_a_map(dt, shape):
    b = Batch(*shape, dt, 0.2, scaled=False)
    b.check_forward(rowwise=True, ids=False)
    got = b.check_backward(F32, map=False)
    assert all(bool((got[k][1:] == 0).all()) for k in ("dA", "dB"))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_packed_batches_and_long_groups(dt):
    """Requests one after another, groups of many tiles and several chunks, an adapter without tokens, results that do not
    depend on the other tokens' order."""
    d = 136
    ids = torch.cat([torch.full((n,), a) for a, n in ((3, 1500), (-1, 77), (0, 129), (3, 640), (5, 1), (1, 128), (-1, 3), (0, 31))])
    b = Batch(len(ids), d, 72, 7, 24 if dt == BF16 else 8, dt, 0.1, ids=ids)
    y, u = b.check_forward()
    got = b.check_backward(BF16 if dt == BF16 else F32)
    assert all(bool((got[k][a] == 0).all()) for k in ("dA", "dB") for a in (2, 4, 6))
    again = b.backward(BF16 if dt == BF16 else F32, None)
    assert all(torch.equal(again[k], got[k]) for k in ("dA", "dB"))   # bit for bit
    flat = b.ids.long()
    # the same tokens' rows through another grouping: row by row results agree with the tiles' within their bounds
    yr, ur = b.forward(rowwise=True)
    wy, by, wu, bu = forward(b.x, b.A, b.B, b.scale, b.ids, b.base, 0.1, SEED, OFFSET)
    within("y by rows", yr, wy, by)
    assert torch.equal(y[flat < 0], b.base[flat < 0])


@pytest.mark.gpu
@pytest.mark.parametrize("T,n", [(5000, 4096), (40000, 3), (1, 4096), (4097, 1), (33000, 100)])
def test_map(T, n):
    """Header, order, tiles and chunks against a stable sort."""
    b = Batch(T, 8, 8, n, 8, BF16, bare=0.3, seed=T)
    w = b.map.view(torch.int32).cpu()
    assert w[:2].tolist() == [T, n]
    ids = b.ids.cpu().long()
    key = torch.where(ids < 0, n, ids)
    order = key.sort(stable=True).indices
    assert torch.equal(w[16:16 + T].long(), order)
    at = 16 + (T + 3) // 4 * 4
    tiles = w[at:at + 4 * int(w[2])].view(-1, 4)
    covered = torch.zeros(T, dtype=torch.int32)
    for a, start, rows, _ in tiles.tolist():
        assert 1 <= rows <= 128 and bool((ids[order[start:start + rows]] == a).all())
        covered[start:start + rows] += 1
    assert bool((covered == 1).all())
    live = key.bincount(minlength=n + 1)
    assert int(w[2]) == int(((live + 127) // 128).sum())
    assert b.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("rowwise", [True, False])
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_in_place_and_bare_rows(rowwise, dt):
    """y on base: the same values; rows without an adapter stay, whatever is in them; u and dx of theirs."""
    b = Batch(300, 72, 200, 4, 16, dt, bare=0.5)
    y, u = b.forward(rowwise=rowwise)
    onto = b.base.clone()
    bare = b.ids < 0
    onto[bare] = float("nan")
    b.L.moe_adapter(b.shape, b.x, b.A, b.B, b.scale, b.ids, None if rowwise else b.map, None, onto, onto, None, b.ws)
    assert torch.equal(onto[~bare], y[~bare]) and bool(torch.isnan(onto[bare]).all())
    assert bool((u[bare] == 0).all())
    g = torch.randn(300, 72, device="cuda")
    got = b.backward(F32, g)
    assert torch.equal(got["dx"][bare], g[bare])
    over = g.clone()
    b.L.moe_adapter_bwd(b.shape, b.L.MOE_F32, b.dy, b.x, b.A, b.B, b.scale, b.map, None, b.u, over, over, None, None, b.ws)
    assert torch.equal(over, got["dx"])
    dA, dB = b.new(*b.A.shape), b.new(*b.B.shape)
    b.L.moe_adapter_bwd(b.shape, b.L.MOE_F32, b.dy, b.x, b.A, b.B, b.scale, b.map, None, b.u, None, None, dA, dB, b.ws)
    assert torch.equal(dA, got["dA"]) and torch.equal(dB, got["dB"])
    assert b.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_a_users_nan_stays_with_that_user(dt):
    """NaN and infinity in one adapter's weights, rows and gradients reach nothing of another adapter's."""
    ids = torch.arange(700) * 5 // 700
    ids = torch.where(torch.arange(700) % 9 == 8, 4 - ids, ids)   # the sick adapter's tokens beside every other's
    b = Batch(700, 136, 200, 5, 16, dt, ids=ids)
    y, u = b.forward()
    back = b.backward(F32, None)
    sick = b.ids == 2
    b.A[2, 3] = float("nan")
    b.B[2, :, 1] = float("inf")
    b.x[sick] = float("inf")
    b.dy[sick] = float("nan")
    b.u[sick] = float("nan")
    for rowwise in (False, True):
        y2, u2 = b.forward(rowwise=rowwise)
        ok = torch.equal if not rowwise else (lambda p, q: bool(torch.isfinite(p).all()))
        assert ok(y2[~sick], y[~sick]) and ok(u2[~sick], u[~sick])
        assert not bool(torch.isfinite(y2[sick]).any())
    back2 = b.backward(F32, None)
    assert torch.equal(back2["dx"][~sick], back["dx"][~sick])
    for k in ("dA", "dB"):
        assert all(torch.equal(back2[k][a], back[k][a]) for a in (0, 1, 3, 4))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_indices_out_of_range_and_foreign_maps(dt):
    """Out of range: no adapter, and reported. A map of another batch size: reported, nothing written. Words of a map that
    make no sense: reported, and nothing out of the batch touched."""
    ids = torch.tensor([0, 2, 7, -1, -5, 1, 3, 2 ** 30])
    b = Batch(8, 64, 72, 3, 8, dt, ids=ids)
    ids = torch.tensor([0, 2, -1, -1, -1, 1, -1, -1])
    L = b.L
    assert L.moe_get_status(b.ws) == (5, 0x500)
    L.moe_clear_status(b.ws)
    y = torch.full_like(b.base, float("nan"))
    L.moe_adapter(b.shape, b.x, b.A, b.B, b.scale, None, b.map, None, b.base, y, None, b.ws)
    assert L.moe_get_status(b.ws)[0] == 0
    wy, by, _, _ = forward(b.x, b.A, b.B, b.scale, ids.cuda(), b.base)
    within("y", y, wy, by)
    y.fill_(float("nan"))
    L.moe_adapter(b.shape, b.x, b.A, b.B, b.scale, b.ids, None, None, b.base, y, None, b.ws)
    within("y", y, wy, by)
    assert L.moe_get_status(b.ws) == (5, 0x500)
    for at, value in ((0, 9), (1, 4)):
        L.moe_clear_status(b.ws)
        other = b.map.clone()
        other.view(torch.int32)[at] = value
        y.fill_(float("nan"))
        L.moe_adapter(b.shape, b.x, b.A, b.B, b.scale, None, other, None, b.base, y, None, b.ws)
        assert L.moe_get_status(b.ws) == (5, 0x600) and bool(torch.isnan(y).all())
    garbage = b.map.clone()
    g = garbage.view(torch.int32)
    g[2:] = torch.randint(-2 ** 31, 2 ** 31 - 1, (g.numel() - 2,), generator=torch.Generator().manual_seed(3)).int().cuda()
    room = torch.full((24, 72), 3.0, dtype=dt, device="cuda")
    L.moe_clear_status(b.ws)
    L.moe_adapter(b.shape, b.x, b.A, b.B, b.scale, None, garbage, None, None, room[8:16], None, b.ws)
    b.backward_with(garbage)
    assert L.moe_get_status(b.ws) == (5, 0x600)
    assert bool((room[:8] == 3).all()) and bool((room[16:] == 3).all())


def _backward_with(self, map):
    dx, dA, dB = self.new(self.T, self.shape.d_in), self.new(*self.A.shape), self.new(*self.B.shape)
    self.L.moe_adapter_bwd(self.shape, self.L.MOE_F32, self.dy, self.x, self.A, self.B, self.scale, map, None, self.u, None, dx,
                           dA, dB, self.ws)


Batch.backward_with = _backward_with


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_streams_graphs_and_calls_at_the_same_time(dt):
    a, b = Batch(600, 264, 136, 6, 16, dt, 0.1, seed=1), Batch(600, 264, 136, 6, 16, dt, 0.1, seed=2)
    want = [(x.forward(), x.backward(F32)) for x in (a, b)]

    def same(got, ref):
        (y, u), back = got
        (wy, wu), wback = ref
        assert torch.equal(y, wy) and torch.equal(u, wu) and all(torch.equal(back[k], wback[k]) for k in back)

    def once(x, y, u, back):
        L = x.L
        L.moe_adapter_map(x.shape, x.ids, x.map, x.ws)
        L.moe_adapter(x.shape, x.x, x.A, x.B, x.scale, None, x.map, x.rng, x.base, y, u, x.ws)
        L.moe_adapter_bwd(x.shape, L.MOE_F32, x.dy, x.x, x.A, x.B, x.scale, x.map, x.rng, x.u, None, back["dx"], back["dA"],
                          back["dB"], x.ws)

    outs = [(torch.empty_like(x.base), x.new(x.T, 16), {k: torch.empty_like(v) for k, v in want[0][1].items()}) for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for x, o, s in zip((a, b), outs, streams):
            with torch.cuda.stream(s):
                once(x, *o)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        same(((o[0], o[1]), o[2]), w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once(a, *outs[0])
    # replayed on other tokens, adapters and masks
    a.x.copy_(b.x), a.dy.copy_(b.dy), a.ids.copy_(b.ids), a.base.copy_(b.base), a.u.copy_(b.u)
    for k in ("A", "B", "scale"):
        getattr(a, k).copy_(getattr(b, k))
    a.rng.copy_(rng_tensor(5, 6)), b.rng.copy_(rng_tensor(5, 6))
    graph.replay()
    torch.cuda.synchronize()
    same(((outs[0][0], outs[0][1]), outs[0][2]), (b.forward(), b.backward(F32)))


@pytest.mark.gpu
def test_nothing_to_do():
    L = lib()
    s = L.MoEAdapterShape(T=0, d_in=64, d_out=72, n=3, rank=8, dtype=1)
    L.moe_adapter_map(s, None, None, None)
    L.moe_adapter(s, None, None, None, None, None, None, None, None, None, None, None)
    dA, dB = torch.ones(3, 8, 64, device="cuda"), torch.ones(3, 72, 8, device="cuda")
    L.moe_adapter_bwd(s, 0, None, None, None, None, None, None, None, None, None, None, dA, dB, None)
    assert not bool(dA.any()) and not bool(dB.any())
    L.moe_dropout(1, 0, None, None, 0.5, None, None)


@pytest.mark.gpu
def test_past_32_bits():
    """Rows that start beyond 2^32 elements, and beyond 2^31 rows times columns of the generator's matrix."""
    L = lib()
    T, d, n = 300, 64, 3
    ld = 1 << 24   # 300 rows 32 MB apart: 10 GB
    g = torch.Generator("cuda").manual_seed(4)
    wide = torch.empty(T * ld // 2, dtype=torch.int32, device="cuda").view(torch.bfloat16).view(T, ld)
    x = wide[:, 8:8 + d]
    x.copy_(torch.randn(T, d, device="cuda", generator=g))
    y = wide[:, 4096:4096 + d]
    A, B = (torch.randn(n, *s, device="cuda", generator=g).bfloat16() for s in ((16, d), (d, 16)))
    ids = torch.randint(-1, n, (T,), device="cuda", generator=g).int()
    s = L.MoEAdapterShape(T=T, d_in=d, d_out=d, n=n, rank=16, dtype=1, dropout=0.25, ld_in=ld, ld_out=ld)
    ws = torch.zeros(L.moe_adapter_workspace_size(s), dtype=torch.uint8, device="cuda")
    m = torch.empty(L.moe_adapter_map_size(s), dtype=torch.uint8, device="cuda")
    L.moe_adapter_map(s, ids, m, ws)
    want, bound, _, _ = forward(x.contiguous(), A, B, None, ids, None, 0.25, SEED, OFFSET)
    for map in (m, None):
        L.moe_adapter(s, x, A, B, None, ids, map, rng_tensor(SEED, OFFSET), None, y, None, ws)
        within("y", y, want, bound)
    assert L.moe_get_status(ws)[0] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("order", ["packed", "mixed", "one"])
@pytest.mark.parametrize("rank", [8, 16])
def test_long_batches_with_dropout(order, rank):
    """Chunks of several tiles, ragged ends, columns past the last whole block, bare rows with and without a base and in
    place."""
    dropout_backwards(8705, 264, 72, order, rank)


@pytest.mark.gpu
def test_ranks_side_by_side():
    """Calls of three shapes on three streams at once, whose CTAs share SMs and their tensor memory, each call right behind
    the one before on the same workspace: the same bits as alone."""
    batches = [Batch(4200, 2048, 1536, 5, 128, BF16), Batch(4100, 4096, 1032, 3, 16, BF16, 0.25),
               Batch(6000, 1544, 2048, 9, 40, BF16)]
    want = [(b.forward(), b.backward(BF16)) for b in batches]
    outs = [(b.new(b.T, b.shape.d_out, dt=BF16), b.new(b.T, b.shape.rank), {k: torch.zeros_like(v) for k, v in w[1].items()})
            for b, w in zip(batches, want)]
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    for _ in range(6):
        for b, (y, u, back), s in zip(batches, outs, streams):
            with torch.cuda.stream(s):
                rng = b.rng if b.p else None
                b.L.moe_adapter(b.shape, b.x, b.A, b.B, b.scale, None, b.map, rng, b.base, y, u, b.ws)
                b.L.moe_adapter_bwd(b.shape, b.L.MOE_BF16, b.dy, b.x, b.A, b.B, b.scale, b.map, rng, b.u, None, back["dx"],
                                    back["dA"], back["dB"], b.ws)
    torch.cuda.synchronize()
    for b, (y, u, back), ((wy, wu), w) in zip(batches, outs, want):
        assert b.status() == 0 and torch.equal(y, wy) and torch.equal(u, wu)
        assert all(torch.equal(back[k], w[k]) for k in w)


@pytest.mark.gpu
@pytest.mark.parametrize("order", ["packed", "mixed", "one"])
@pytest.mark.parametrize("T,d_in,rank", [(8705, 648, 16), (700, 3464, 8), (700, 3464, 16), (130, 9736, 16), (1, 9736, 8)])
def test_one_pass_of_the_backward(T, d_in, order, rank):
    """With dropout, ranks up to 16, a bf16 dx and enough blocks of columns dA and dx are made in one pass."""
    dropout_backwards(T, d_in, 40, order, rank)


def dropout_backwards(T, d_in, d_out, order, rank):
    n = 5
    t = torch.arange(T)
    ids = {"packed": (t * 7 // T).clamp_max(5) - 1, "mixed": None, "one": torch.zeros(T)}[order]
    b = Batch(T, d_in, d_out, 1 if order == "one" else n, rank, BF16, 0.25, bare=0.3, ids=ids)
    b.check_forward()
    got = b.check_backward(BF16, map=order != "one")
    b.check_backward(BF16, dx_in=False, map=order != "one")
    g = torch.randn(T, d_in, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(BF16)
    over, dA, dB = g.clone(), b.new(*b.A.shape), b.new(*b.B.shape)
    b.L.moe_adapter_bwd(b.shape, b.L.MOE_BF16, b.dy, b.x, b.A, b.B, b.scale, None if order == "one" else b.map, b.rng, b.u, over,
                        over, dA, dB, b.ws)
    assert torch.equal(over, got["dx"]) and torch.equal(dA, got["dA"]) and torch.equal(dB, got["dB"])
    assert b.status() == 0
    # dA is the one of the two separate passes within the bounds, dx without dA bit for bit
    alone = b.new(T, d_in, dt=BF16)
    b.L.moe_adapter_bwd(b.shape, b.L.MOE_BF16, b.dy, b.x, b.A, b.B, b.scale, None if order == "one" else b.map, b.rng, b.u, g,
                        alone, None, None, b.ws)
    assert torch.equal(alone, got["dx"])
    b.check_backward(F32, map=order != "one")


@pytest.mark.gpu
@pytest.mark.parametrize("T,n,rank", [(20000, 1, 64), (9000, 200, 128), (16500, 3, 40)])
def test_long_batches(T, n, rank):
    b = Batch(T, 136, 200, n, rank, BF16, 0.0, bare=0.1)
    b.check_forward()
    b.check_backward(BF16)
