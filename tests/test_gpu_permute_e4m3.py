"""moe_permute_e4m3 against moe_permute on the rows that the bytes and scales
stand for: the same map, and rows equal bit for bit (one product of two fp32
numbers, one rounding)."""
import pytest

torch = pytest.importorskip("torch")

from tests.gpu_util import lib  # noqa: E402


def _case(L, T, d, E, K, dt, group, kept, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    gs = group or d
    ng = -(-d // gs)
    q = (torch.randn(T, d, device="cuda", generator=g) * 40).clamp(-448, 448).to(torch.float8_e4m3fn)
    s = torch.rand(T, ng, device="cuda", generator=g) * 0.1
    idx = torch.rand(T, E, device="cuda", generator=g).topk(K, dim=1).indices.int()
    keep = (torch.rand(T, K, device="cuda", generator=g) < kept).to(torch.uint8)
    shape = L.MoEShape(T=T, d=d, E=E, K=K, F=64, dtype=L.MOE_BF16 if dt == torch.bfloat16 else L.MOE_F32)
    x = (q.float() * s.repeat_interleave(gs, 1)[:, :d]).to(dt)
    return shape, q, s, idx, keep, x


def _outputs(T, d, E, K, dt):
    i = lambda *n: torch.full(n, 7, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(Xp=torch.full((T * K + 1, d), 7.0, dtype=dt, device="cuda"), row_of=i(T, K), src_of=i(T * K + 1),
                counts=i(E), offsets=i(E + 1))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,d,E,K,group,kept", [
    (1, 8, 1, 1, 0, 1.0), (1, 1024, 64, 8, 128, 1.0), (3, 72, 5, 2, 32, 0.5), (257, 1000, 60, 6, 64, 0.9),
    (777, 2056, 8, 3, 128, 0.7), (513, 3584, 64, 8, 0, 1.0), (300, 136, 8, 2, 64, 0.0), (5, 51200, 4, 2, 128, 1.0), (1030, 6144, 16, 5, 128, 0.95)])
def test_matches_permute_of_the_values(T, d, E, K, group, kept, dt):
    L = lib()
    if dt == torch.float32 and d in (72, 1000, 136):
        d += 4
    shape, q, s, idx, keep, x = _case(L, T, d, E, K, dt, group, kept)
    ws = torch.zeros(L.moe_workspace_size(shape), dtype=torch.uint8, device="cuda")
    a, b = _outputs(T, d, E, K, dt), _outputs(T, d, E, K, dt)
    L.moe_permute(shape, x, idx, keep, a["Xp"], a["row_of"], a["src_of"], a["counts"], a["offsets"], ws)
    L.moe_permute_e4m3(shape, q, s, group, idx, keep, b["Xp"], b["row_of"], b["src_of"], b["counts"], b["offsets"], ws)
    rc, _ = L.moe_get_status(ws)
    assert rc == 0
    for k in a:   # rows past the last kept one stay as they were on both sides
        assert torch.equal(a[k], b[k]), k


@pytest.mark.gpu
def test_bad_expert_and_special_values():
    """An expert index outside the range is skipped and reported; NaN bytes and
    an infinite scale reach only their own row."""
    L = lib()
    T, d, E, K = 40, 64, 4, 2
    shape, q, s, idx, keep, x = _case(L, T, d, E, K, torch.bfloat16, 32, 1.0)
    q.view(torch.uint8)[3, 5] = 0x7F
    s[9, 1] = float("inf")
    idx[20, 1] = 4
    idx[21, 0] = -1
    ws = torch.zeros(L.moe_workspace_size(shape), dtype=torch.uint8, device="cuda")
    o = _outputs(T, d, E, K, torch.bfloat16)
    L.moe_permute_e4m3(shape, q, s, 32, idx, keep, o["Xp"], o["row_of"], o["src_of"], o["counts"], o["offsets"], ws)
    rc, _ = L.moe_get_status(ws)
    assert rc == 5
    row = o["row_of"].cpu()
    assert row[20, 1] == -1 and row[21, 0] == -1 and int(o["offsets"][E]) == T * K - 2
    bad = sorted(int(r) for t in (3, 9) for r in row[t])
    finite = torch.isfinite(o["Xp"][:T * K - 2].float()).all(1).cpu()
    assert [i for i in range(T * K - 2) if not finite[i]] == bad


@pytest.mark.gpu
def test_captured_and_replayed():
    L = lib()
    T, d, E, K = 300, 512, 8, 2
    shape, q, s, idx, keep, x = _case(L, T, d, E, K, torch.bfloat16, 128, 0.9)
    ws = torch.zeros(L.moe_workspace_size(shape), dtype=torch.uint8, device="cuda")
    o = _outputs(T, d, E, K, torch.bfloat16)
    call = lambda st=None: L.moe_permute_e4m3(shape, q, s, 128, idx, keep, o["Xp"], o["row_of"], o["src_of"],  # noqa: E731
                                              o["counts"], o["offsets"], ws, st)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    _, q2, s2, idx2, keep2, _ = _case(L, T, d, E, K, torch.bfloat16, 128, 0.9, seed=5)
    q.copy_(q2), s.copy_(s2), idx.copy_(idx2), keep.copy_(keep2)
    graph.replay()
    torch.cuda.synchronize()
    n = int(o["offsets"][E])
    got = {k: v.clone() for k, v in o.items()}
    call()
    torch.cuda.synchronize()
    assert n == int(keep2.sum()) and torch.equal(got["Xp"][:n], o["Xp"][:n]) and torch.equal(got["row_of"], o["row_of"])
