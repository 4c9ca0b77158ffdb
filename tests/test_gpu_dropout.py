"""Dropout and its backward against the generator's definition, bit for bit in
the mask and within one rounding in the values."""
import pytest

torch = pytest.importorskip("torch")

from tests.adapter_util import dropped, mask, rng_tensor, round_to, words  # noqa: E402
from tests.gpu_util import lib  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16
SIZES = [1, 7, 8, 9, 255, 8192, 8193, 65543, 300001]
SEED, OFFSET = 2 ** 63 + 12345, 2 ** 62 + 2 ** 33 + 7


def code(L, dt):
    return L.MOE_BF16 if dt == BF16 else L.MOE_F32


def test_the_generator_gives_its_papers_values():
    """The known answers of Philox4x32-10 published with the paper's library."""
    def one(ctr, key):   # the counter's low words are the block's number, the high ones the offset
        w = words([ctr[0] | ctr[1] << 32], key[0] | key[1] << 32, ctr[2] | ctr[3] << 32)[0]
        return [int(v) for v in w]

    assert one([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert one([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert one([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def check(got, x, res, p, dt):
    want = dropped(x, p, SEED, OFFSET)
    bound = want.abs() * 2.0 ** -23   # the factor and the product, fused into the sum or not
    if res is not None:
        want = want + res.double()
    bound = bound + (want.abs() + bound) * round_to(dt)
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), float((err - bound).max())
    if res is None and p:
        keep = mask(x.numel(), p, SEED, OFFSET).to(x.device)
        assert torch.equal(got.view(-1) != 0, keep & (x.view(-1) != 0))


@pytest.mark.gpu
@pytest.mark.parametrize("n", SIZES)
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("res", [True, False], ids=["residual", "bare"])
def test_forward(n, dt, res):
    L = lib()
    g = torch.Generator().manual_seed(n)
    x = torch.randn(n, generator=g).to(dt).cuda()
    r = torch.randn(n, generator=g).to(dt).cuda() if res else None
    rng = rng_tensor(SEED, OFFSET)
    for p in (0.1, 0.5, 0.999, 2.0 ** -16):
        out = torch.full_like(x, float("nan"))
        L.moe_dropout(code(L, dt), n, x, r, p, rng, out)
        check(out, x, r, p, dt)
    out = torch.full_like(x, float("nan"))
    L.moe_dropout(code(L, dt), n, x, r, 0.0, None, out)   # keeps everything, without a generator
    assert torch.equal(out, x if r is None else (x.float() + r.float()).to(dt))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 9, 4096, 65543])
@pytest.mark.parametrize("dy_t", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("dx_t", [F32, BF16], ids=["f32", "bf16"])
def test_backward(n, dy_t, dx_t):
    L = lib()
    dy = torch.randn(n, generator=torch.Generator().manual_seed(n)).to(dy_t).cuda()
    rng, dx = rng_tensor(SEED, OFFSET), torch.full((n,), float("nan"), dtype=dx_t, device="cuda")
    L.moe_dropout_bwd(code(L, dy_t), code(L, dx_t), n, dy, 0.3, rng, dx)
    check(dx, dy, None, 0.3, dx_t)


@pytest.mark.gpu
def test_in_place_and_not_finite():
    """In place gives the same; what is dropped is 0 whatever it was; neighbours of the buffer stay."""
    L = lib()
    n, p = 4103, 0.4
    rng = rng_tensor(5, 9)
    x = torch.randn(n, device="cuda").bfloat16()
    r = torch.randn(n, device="cuda").bfloat16()
    want = torch.empty_like(x)
    L.moe_dropout(L.MOE_BF16, n, x, r, p, rng, want)
    for place in (x, r):
        wide = torch.full((n + 64,), 3.0, dtype=BF16, device="cuda")
        wide[:n] = place
        a, b = (wide[:n], r) if place is x else (x, wide[:n])
        L.moe_dropout(L.MOE_BF16, n, a, b, p, rng, wide[:n])
        assert torch.equal(wide[:n], want) and bool((wide[n:] == 3.0).all())
    bad = torch.full((n,), float("inf"), device="cuda")
    bad[::2] = float("nan")
    out = torch.empty_like(bad)
    L.moe_dropout(L.MOE_F32, n, bad, None, p, rng, out)
    keep = mask(n, p, 5, 9).cuda()
    assert bool((out[~keep] == 0).all()) and not bool(torch.isfinite(out[keep]).any())


@pytest.mark.gpu
def test_share_of_kept_and_other_generators():
    L = lib()
    n, p = 1 << 20, 0.1
    x = torch.ones(n, device="cuda")
    outs = []
    for seed, offset in ((1, 0), (1, 1), (2, 0), (1 + (1 << 40), 0), (1, 1 << 40)):
        out = torch.empty_like(x)
        L.moe_dropout(L.MOE_F32, n, x, None, p, rng_tensor(seed, offset), out)
        # five standard deviations of a binomial share
        assert abs(float((out == 0).double().mean()) - p) < 5 * (p * (1 - p) / n) ** 0.5 + 2.0 ** -17
        outs.append(out != 0)
    for i in range(5):
        for j in range(i):   # independent masks agree on 0.82
            assert abs(float((outs[i] == outs[j]).double().mean()) - 0.82) < 5 * (0.82 * 0.18 / n) ** 0.5 + 1e-4


@pytest.mark.gpu
def test_graph_draws_new_masks_and_side_stream():
    """A captured step reads the generator's words when it runs."""
    L = lib()
    n, p = 10007, 0.25
    x, rng, out = torch.randn(n, device="cuda"), rng_tensor(3, 0), torch.empty(n, device="cuda")
    L.moe_dropout(L.MOE_F32, n, x, None, p, rng, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.moe_dropout(L.MOE_F32, n, x, None, p, rng, out)
        rng[1:].add_(1)
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out != 0, mask(n, p, 3, step).cuda())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = torch.empty_like(out)
        L.moe_dropout(L.MOE_F32, n, x, None, p, rng_tensor(3, 2), other)
    side.synchronize()
    assert torch.equal(other, out)


@pytest.mark.gpu
def test_past_32_bits():
    """More than 2^32 elements: blocks and addresses past 32 bits."""
    L = lib()
    n = 2 ** 32 + 2 ** 20 + 3
    x = torch.ones(n, dtype=BF16, device="cuda")
    L.moe_dropout(L.MOE_BF16, n, x, None, 0.5, rng_tensor(7, 1), x)
    for first in (0, 2 ** 31 - 4096, 2 ** 32 - 4096, 2 ** 32 + 2 ** 20 - 4096):
        m = min(8192, n - first)
        assert torch.equal(x[first:first + m] != 0, mask(m, 0.5, 7, 1, first).cuda())
