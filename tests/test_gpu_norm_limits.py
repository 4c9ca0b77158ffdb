"""moe_rmsnorm at the ends of the fp32 range, with the bounds of test_gpu_norm:
rows just below the size at which the sum of their squares overflows, rows above
it (y = 0, nothing else touched), and rows of subnormal numbers."""
import pytest

torch = pytest.importorskip("torch")

from tests.gpu_util import lib  # noqa: E402
from tests.test_gpu_norm import _backward, _check_forward, _forward, _rows  # noqa: E402

MAX = float(torch.finfo(torch.float32).max)
# one register layout each: a row per warp, per CTA with two and with four vectors a thread
SIZES = [(d, dt) for dt in (torch.bfloat16, torch.float32) for d in (64, 4096, 32768 if dt == torch.bfloat16 else 16384)]


@pytest.mark.gpu
@pytest.mark.parametrize("d,dt", SIZES, ids=lambda v: str(v).replace("torch.", ""))
def test_rows_up_to_the_overflow_of_their_squares(d, dt):
    """The limit is on the sum of the squares: an rms of sqrt(3.4e38 / d)."""
    L = lib()
    x = _rows(9, d, torch.float32, 1)
    gamma = (1 + 0.3 * _rows(1, d, torch.float32, 2)[0]).to(dt)
    clean = x.to(dt)
    unit = x.square().mean(1).sqrt()
    limit = (MAX / d) ** 0.5
    for i, f in ((1, 0.99), (3, 1.01), (4, 1e3), (6, 0.5)):   # bf16 rounding moves the rms by less than 2^-8
        x[i] *= f * limit / unit[i]
    x = x.to(dt)
    x[7] = 0
    x[7, d // 2] = 2e19 if dt == torch.float32 else 2.0 ** 65   # one square alone is too large
    want = _forward(L, clean.cuda(), None, gamma.cuda(), 32)
    out = _forward(L, x.cuda(), None, gamma.cuda(), 32)
    for i in (0, 2, 5, 8):   # what lies beside them is as it was
        assert all(torch.equal(out[k][i].float(), want[k][i].float()) for k in out), i
    for i in (1, 6):
        _check_forward(x[i:i + 1], None, gamma, {k: v[i:i + 1] for k, v in out.items()}, 32)
    for i in (3, 4, 7):
        assert out["rstd"][i] == 0 and (out["y"][i] == 0).all(), i
        assert (out["q"][i].float() == 0).all() and (out["s"][i] == 1).all(), i
        assert torch.equal(out["h"][i].cpu(), x[i]), i
    # the backward of y = 0: what reaches h from elsewhere, and nothing for gamma
    dy, dh = _rows(9, d, torch.float32, 3).cuda(), _rows(9, d, dt, 4).cuda()
    for rows in ([3], [4], [7]):
        dx, dgamma = _backward(L, dy[rows], x[rows].cuda(), gamma.cuda(), out["rstd"][rows], dh[rows], torch.float32)
        assert torch.equal(dx, dh[rows].float()) and (dgamma == 0).all(), rows


@pytest.mark.gpu
@pytest.mark.parametrize("d,dt", SIZES, ids=lambda v: str(v).replace("torch.", ""))
def test_rows_of_the_smallest_numbers(d, dt):
    """Their squares are 0 in fp32, so rstd is 1 / sqrt(eps); the rows stay
    what they are times that, and the 8-bit scale stops at its floor."""
    L = lib()
    x = _rows(5, d, torch.float32, 1)
    x[0] = 1e-38
    x[1] *= 1e-38
    x[2] *= 1e-40
    x[3] *= 1e-34      # around the scale's floor after the norm
    x[4] = 0
    x[4, 1] = 2.0 ** -133   # the smallest bf16
    x = x.to(dt)
    gamma = (1 + 0.3 * _rows(1, d, torch.float32, 2)[0]).to(dt)
    for group in (0, 32, 128):
        out = _forward(L, x.cuda(), None, gamma.cuda(), group)
        _check_forward(x, None, gamma, out, group)
    r = x.flip(0)
    out = _forward(L, x.cuda(), r.cuda(), gamma.cuda(), 64)
    _check_forward(x, r, gamma, out, 64)
