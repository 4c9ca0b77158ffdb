"""moe_grad_norm and moe_grad_clip against 64-bit sums.

The norm: a thread adds at most 64 squares in fp32 (relative error below
64 * 2^-24 of a positive sum, half of it after the root), everything after that
in fp64, one rounding at the end: 34 * 2^-24. coef and the clipped values are
one division and one product of fp32 numbers that the test has: exact."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.gpu_util import lib  # noqa: E402

U = 2.0 ** -24


def _list(specs, seed=0, scale=1.0):
    """Tensors of (numel, dtype, offset): `offset` elements behind a 256-byte boundary, sentinels around."""
    g = torch.Generator().manual_seed(seed)
    host, dev, raw = [], [], []
    for n, dt, off in specs:
        v = (torch.randn(n, generator=g) * scale).to(dt)
        b = torch.full((off + n + 16,), 7.0, device="cuda").to(dt)
        b[off:off + n] = v.cuda()
        host.append(v), dev.append(b[off:off + n]), raw.append((b, off, n))
    return host, dev, raw


def _intact(raw):
    return all((b[:o].float() == 7).all() and (b[o + n:].float() == 7).all() for b, o, n in raw)


def _norm(L, tensors, stream=None):
    norm = torch.full((1,), -1.0, device="cuda")
    ws = torch.full((L.MOE_GRAD_NORM_WORKSPACE_BYTES,), 255, dtype=torch.uint8, device="cuda")
    L.moe_grad_norm(L.TensorList(tensors), norm, ws, stream)
    torch.cuda.synchronize()
    return float(norm)


def _exact(host):
    return float(torch.sqrt(sum((t.double() ** 2).sum() for t in host))) if host else 0.0


F32, B16 = torch.float32, torch.bfloat16
LISTS = {
    "one element": [(1, F32, 0)],
    "one bf16 element": [(1, B16, 0)],
    "odd": [(1023, F32, 0), (77777, F32, 0), (3, F32, 0)],
    "empty among them": [(0, F32, 0), (129, F32, 0), (0, B16, 0)],
    "unaligned": [(8191, F32, 1), (8192, F32, 2), (5, F32, 3), (40001, B16, 1), (2, B16, 7), (8193, B16, 5)],
    "chunk edges": [(8192, F32, 0), (8193, F32, 0), (16384, B16, 0), (16385, B16, 0), (8190, F32, 3)],
    "mixed types": [(100000, F32, 0), (100000, B16, 0)] * 3,
    "many tiny": [(7 + i % 13, F32 if i % 3 else B16, i % 4) for i in range(300)],
    "many tiny, then a large one": [(3, F32, 0)] * 96 + [(5_000_000, F32, 0)] + [(3, F32, 0)] * 96,
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", LISTS)
def test_norm_and_clip(name):
    L = lib()
    host, dev, raw = _list(LISTS[name])
    want, got = _exact(host), _norm(L, dev)
    assert abs(got - want) <= 34 * U * want
    norm, coef = torch.tensor([got], device="cuda"), torch.full((1,), -1.0, device="cuda")
    for max_norm in (0.5 * got, 2.0 * got, got, 0.0):
        c = np.float32(max_norm) / np.float32(got) if np.float32(got) > np.float32(max_norm) else np.float32(1)
        out = [torch.full((t.numel() + 1,), 9.0, device="cuda").to(t.dtype) for t in dev]
        views = [o[1:] if i % 2 else o[:-1] for i, o in enumerate(out)]   # other alignments than the gradients'
        L.moe_grad_clip(L.TensorList(dev), L.TensorList(views), norm, max_norm, coef)
        torch.cuda.synchronize()
        assert np.float32(float(coef)) == c
        for h, t, v in zip(host, dev, views):
            ref = (h.float() * float(c)).to(h.dtype)
            assert torch.equal(v.cpu(), ref) and torch.equal(t.cpu(), h)
        for i, o in enumerate(out):
            assert float(o[0] if i % 2 else o[-1]) == 9.0
    L.moe_grad_clip(L.TensorList(dev), None, norm, 0.5 * got, None)   # in place
    torch.cuda.synchronize()
    c = float(np.float32(0.5 * got) / np.float32(got))
    assert all(torch.equal(t.cpu(), (h.float() * c).to(h.dtype)) for h, t in zip(host, dev))
    assert _intact(raw)


@pytest.mark.gpu
def test_empty_lists():
    L = lib()
    assert _norm(L, []) == 0.0
    assert _norm(L, [torch.empty(0, device="cuda")]) == 0.0
    coef = torch.full((1,), -1.0, device="cuda")
    L.moe_grad_clip(L.TensorList([]), None, torch.zeros(1, device="cuda"), 1.0, coef)
    torch.cuda.synchronize()
    assert float(coef) == 1.0


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1e30, 3e18, 1e-20, 1e-30, 1e-38, 1e-44])
@pytest.mark.parametrize("dt", [F32, B16], ids=["f32", "bf16"])
def test_norm_over_the_whole_range(scale, dt):
    """Squares that fp32 does not hold: the norm does."""
    L = lib()
    if dt == B16 and scale < 1e-39:
        scale = 1e-39
    host, dev, _ = _list([(5000, dt, 0), (1, dt, 1)], scale=scale)
    want = _exact(host)
    assert abs(_norm(L, dev) - want) <= 34 * U * want + 2.0 ** -150
    host.append(torch.ones(3)), dev.append(torch.ones(3, device="cuda"))
    want = _exact(host)
    assert abs(_norm(L, dev) - want) <= 34 * U * want
    zeros = torch.zeros(100_000, device="cuda")
    assert _norm(L, [zeros, -zeros]) == 0.0


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_norm_that_is_not_finite_leaves_the_gradients(bad):
    L = lib()
    host, dev, _ = _list([(10_000, F32, 0), (33, B16, 1)])
    dev[0][777] = bad
    host[0][777] = bad
    got = _norm(L, dev)
    assert np.isnan(got) if np.isnan(bad) else got == float("inf")
    norm, coef = torch.tensor([got], device="cuda"), torch.zeros(1, device="cuda")
    out = [torch.zeros_like(t) for t in dev]
    L.moe_grad_clip(L.TensorList(dev), L.TensorList(out), norm, 1.0, coef)
    L.moe_grad_clip(L.TensorList(dev), None, norm, 1.0, None)
    torch.cuda.synchronize()
    assert float(coef) == 1.0
    for h, t, o in zip(host, dev, out):
        assert torch.equal(t.cpu().nan_to_num(5.0), h.nan_to_num(5.0))
        assert torch.equal(o.cpu().nan_to_num(5.0), h.nan_to_num(5.0))


@pytest.mark.gpu
def test_beyond_32_bits_of_elements():
    """A bf16 tensor of 2^32 + 5 elements, ones in a few far places."""
    L = lib()
    n = 2 ** 32 + 5
    x = torch.zeros(n, dtype=B16, device="cuda")
    at = [0, 2 ** 31 - 1, 2 ** 31, 2 ** 32 - 1, 2 ** 32, n - 1]
    x[torch.tensor(at, device="cuda")] = 3.0
    got = _norm(L, [x])
    assert abs(got - np.sqrt(54.0)) <= 34 * U * got
    L.moe_grad_clip(L.TensorList([x]), None, torch.tensor([2.0], device="cuda"), 1.0, None)
    torch.cuda.synchronize()
    assert all(float(x[i]) == 1.5 for i in at) and int((x != 0).sum()) == len(at)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [3000, 300_000])   # in one launch, and in two
def test_streams_graphs_and_repeats(n):
    L = lib()
    host, dev, _ = _list([(n, F32, 0), (12345, B16, 1)])
    tl = L.TensorList(dev)
    out = [torch.empty_like(t) for t in dev]
    to = L.TensorList(out)
    ws = torch.empty(L.MOE_GRAD_NORM_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    norm, coef = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")

    def step(stream=None):
        L.moe_grad_norm(tl, norm, ws, stream)
        L.moe_grad_clip(tl, to, norm, 1.0, coef, stream)

    step()
    torch.cuda.synchronize()
    first = [norm.clone(), coef.clone()] + [o.clone() for o in out]
    side = torch.cuda.Stream()
    norm.zero_(), [o.zero_() for o in out]
    torch.cuda.synchronize()
    step(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, [norm, coef] + out))   # bit for bit, on another stream
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    # written by the kernel before on the same stream, then read by the replay at once
    for _ in range(3):
        dev[0].mul_(0.5)
        graph.replay()
    torch.cuda.synchronize()
    want = _exact([host[0] * 0.125, host[1]])
    assert abs(float(norm) - want) <= 34 * U * want
