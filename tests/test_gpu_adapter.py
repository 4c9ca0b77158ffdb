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
