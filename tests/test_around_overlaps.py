"""Buffers that share memory where the operators around the layer would race or
overwrite what they still read: refused before anything is launched. No GPU is
needed; the addresses are never dereferenced."""
import pytest

from tests.test_around_refusals import A, L, _shape, refused  # noqa: F401

T, D, E, K, N_SUB = 64, 64, 8, 2, 4   # _shape's; sub-sequences of 16 tokens


def over(address, bytes_, other_bytes):
    """Places of a buffer of `other_bytes` that touch one of `bytes_` at `address`: at its start, over its first and
    over its last 16 bytes."""
    return [address, address + 16 - other_bytes // 16 * 16 if other_bytes >= 16 else address, address + (bytes_ - 1) // 16 * 16]


def test_balance_loss(L):  # noqa: F811
    s = _shape(L)
    size = dict(logits=T * E * 4, idx=T * K * 4, mask=T, loss=4, counts=N_SUB * E * 4, prob=N_SUB * E * 4,
                coef=(N_SUB * E + 1) * 4, ws=L.moe_workspace_size(s))
    at = dict(zip(size, A))

    def call(**kw):
        a = {**at, **kw}
        refused(L, 1, "moe_balance_loss", s, a["logits"], a["idx"], a["mask"], 0.1, a["loss"], a["counts"], a["prob"],
                a["coef"], a["ws"], 0)

    outs = ["loss", "counts", "prob", "coef"]
    for i, o in enumerate(outs):
        for other in ["logits", "idx", "mask"] + outs[i + 1:]:
            for place in over(at[other], size[other], size[o]):
                call(**{o: place})
        call(**{o: at["ws"]})                       # the status word
        call(**{o: at["ws"] + size["ws"] - 256})    # the partial sums, which lie last
    for i in ("logits", "idx", "mask"):
        call(**{i: at["ws"] + size["ws"] - 256})


def test_balance_loss_bwd(L):  # noqa: F811
    s = _shape(L)
    size = dict(logits=T * E * 4, mask=T, coef=(N_SUB * E + 1) * 4, dloss=4)
    at = dict(zip(size, A))
    for other in size:
        for place in over(at[other], size[other], T * E * 4):
            if place != at["logits"]:               # the logits' own place is allowed
                refused(L, 1, "moe_balance_loss_bwd", s, at["logits"], at["mask"], at["coef"], at["dloss"], place, 0)


def test_route_bwd_add(L):  # noqa: F811
    """dlogits_add inside the workspace, where the logits' gradient is written
    while it is read."""
    s = _shape(L)
    ws, n = A[9], L.moe_workspace_size(_shape(L))
    for add in range(ws - T * E * 4 + 16, ws + n, 256):
        refused(L, 1, "moe_route_bwd_add", s, A[0], A[1], None, A[2], A[3], A[4], A[5], A[6], None, add, None, A[7], None, None,
                A[8], ws, 0)


@pytest.mark.parametrize("dtype,group", [(0, 32), (1, 0)])
def test_permute_e4m3(L, dtype, group):  # noqa: F811
    s = _shape(L, dtype=dtype)
    ng = -(-D // group) if group else 1
    size = dict(q=T * D, s=T * ng * 4, idx=T * K * 4, keep=T * K, Xp=T * K * D * (2 if dtype else 4), row=T * K * 4,
                src=T * K * 4, cnt=E * 4, off=(E + 1) * 4, ws=L.moe_workspace_size(s))
    at = dict(zip(size, A))

    def call(**kw):
        refused(L, 1, "moe_permute_e4m3", s, *[{**at, **kw}[k] for k in ("q", "s")], group,
                *[{**at, **kw}[k] for k in ("idx", "keep", "Xp", "row", "src", "cnt", "off", "ws")], 0)

    outs = ["Xp", "row", "src", "cnt", "off"]
    for i, o in enumerate(outs):
        for other in ["q", "s", "idx", "keep"] + outs[i + 1:]:
            for place in over(at[other], size[other], size[o]):
                call(**{o: place})
        call(**{o: at["ws"]})         # the status word and the counts behind it
    for i in ("q", "s", "idx", "keep"):
        call(**{i: at["ws"]})


def test_permute_e4m3_misplaced_words(L):  # noqa: F811
    """32-bit words that do not start on 4 bytes would fault."""
    at = dict(zip(("q", "s", "idx", "keep", "Xp", "row", "src", "cnt", "off", "ws"), A))
    for k in ("s", "idx", "row", "src", "cnt", "off"):
        v = {**at, k: at[k] + 2}
        refused(L, 1, "moe_permute_e4m3", _shape(L), v["q"], v["s"], 32, *list(v.values())[2:], 0)


class List:
    """A list of tensors as the C calls take it: (address, elements, type) each."""

    def __init__(self, L, *t):  # noqa: F811
        import ctypes
        self.n = len(t)
        self.array = (L.MoETensor * max(1, len(t)))(*[L.MoETensor(*x) for x in t])
        self.address = ctypes.addressof(self.array)
        self.device = None


@pytest.mark.parametrize("n", [3, 100])
def test_grad_clip(L, n):  # noqa: F811
    """n gradients of 100 fp32 elements 1 KB apart, in descending order of their addresses."""
    grads = [(A[0] + (n - i) * 1024, 100, 0) for i in range(n)]
    outs = [(A[1] + (i * 7 % n if n % 7 else i) * 1024, 100, 0) for i in range(n)]
    grads[1] = (None, 0, 0)                      # an empty one is nowhere
    outs[1] = (outs[1][0], 0, 0)

    def clip(g, o, norm=A[2], coef=A[3]):
        refused(L, 1, "moe_grad_clip", List(L, *g), None if o is None else List(L, *o), norm, 1.0, coef, 0)

    def put(t, i, address):
        return t[:i] + [(address, *t[i][1:])] + t[i + 1:]

    first, last = grads[0][0], grads[-1][0]
    clip(put(grads, 0, last), None)              # the same tensor twice, in place
    clip(put(grads, 0, last + 396), None)        # its last element shared
    clip(grads, put(outs, 0, last))              # over another gradient
    clip(grads, put(outs, n - 1, first - 4))     # over another gradient's front
    clip(grads, put(grads, 0, last))             # in place but for one, which is another's
    clip(grads, put(outs, 0, outs[-1][0] + 4))   # two outputs in one place
    for place in (first, last + 396):
        clip(grads, None, norm=place)            # the norm inside a gradient that is scaled
        clip(grads, None, coef=place)
        clip(grads, outs, coef=place)            # the factor over a gradient that is read
    for place in (outs[0][0], outs[-1][0] + 396):
        clip(grads, outs, norm=place)
        clip(grads, outs, coef=place)
    clip(grads, outs, norm=A[2], coef=A[2])      # every CTA reads the norm
    clip([], None, norm=A[2], coef=A[2])


@pytest.mark.parametrize("n", [1, 100])
def test_grad_norm(L, n):  # noqa: F811
    """The partial sums over a gradient that is still read."""
    grads = [(A[0] + i * 1024, 100, 0) for i in range(n)]
    for ws in (A[0], A[0] + (n - 1) * 1024 + 384, A[0] - L.MOE_GRAD_NORM_WORKSPACE_BYTES + 16):
        refused(L, 1, "moe_grad_norm", List(L, *grads), A[2], ws, 0, ws_bytes=1 << 20)


@pytest.mark.gpu
def test_buffers_that_touch_are_taken():
    """Every buffer of a call cut from one block, end to end: nothing is shared
    and the results are those of separate buffers."""
    torch = pytest.importorskip("torch")
    from tests.gpu_util import lib
    L = lib()  # noqa: F811
    s = _shape(L)

    def cut(block, *parts):
        out, at = [], 0
        for dtype, *dims in parts:
            t = torch.empty(dims, dtype=dtype, device="meta")
            n = t.numel() * t.element_size()
            out.append(block[at:at + n].view(dtype).view(dims))
            at += -(-n // 16) * 16
        assert at <= block.numel()
        return out

    g = torch.Generator(device="cuda").manual_seed(1)
    f, i, b = torch.float32, torch.int32, torch.uint8
    rand = torch.randn(T, E, device="cuda", generator=g)
    idx = rand.topk(K, dim=1).indices.int()
    got = []
    for together in (True, False):
        block = torch.zeros(1 << 16, dtype=b, device="cuda")
        parts = [(f, T, E), (i, T, K), (b, T), (f, 1), (i, N_SUB, E), (f, N_SUB, E), (f, N_SUB * E + 1), (f, T, E)]
        ts = cut(block, *parts)
        if not together:
            ts = [t.clone() for t in ts]
        logits, topk, mask, loss, counts, prob, coef, dl = ts
        logits.copy_(rand)
        topk.copy_(idx)
        mask.fill_(1)
        ws = torch.zeros(L.moe_workspace_size(s), dtype=b, device="cuda")
        L.moe_balance_loss(s, logits, topk, mask, 0.1, loss, counts, prob, coef, ws)
        L.moe_balance_loss_bwd(s, logits, mask, coef, None, dl)
        got.append([t.clone() for t in (loss, counts, prob, coef, dl)])
        block = torch.zeros(1 << 16, dtype=b, device="cuda")
        parts = [(b, T, D), (f, T, 2), (i, T, K), (b, T, K), (torch.bfloat16, T * K, D), (i, T, K), (i, T * K), (i, E), (i, E + 1)]
        ts = cut(block, *parts)
        if not together:
            ts = [t.clone() for t in ts]
        q, scale, topk, keep, *outs = ts
        q.copy_(torch.randint(0, 0x78, (T, D), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).to(b))
        scale.fill_(0.5)
        topk.copy_(idx)
        keep.fill_(1)
        L.moe_permute_e4m3(s, q, scale, 32, topk, keep, *outs, ws)
        assert L.moe_get_status(ws)[0] == 0
        got[-1] += [t.clone() for t in outs]
    assert all(torch.equal(x, y) for x, y in zip(*got))
    assert int(got[0][1].sum()) == T * K and bool(got[0][5].any())
    # gradients and outputs in turn in one block; every third in place
    for n in (5, 100):
        block = torch.randn(2 * n * 8, device="cuda", generator=g)
        before = block.clone()
        ins = [block[2 * k * 8:(2 * k + 1) * 8] for k in range(n)]
        outs = [t if k % 3 == 0 else block[(2 * (n - k) - 1) * 8:2 * (n - k) * 8] for k, t in enumerate(ins)]
        want = torch.linalg.vector_norm(torch.cat(ins).double())
        norm, coef = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
        grads, out = L.TensorList(ins), L.TensorList(outs)
        ws = torch.empty(L.MOE_GRAD_NORM_WORKSPACE_BYTES, dtype=b, device="cuda")
        L.moe_grad_norm(grads, norm, ws)
        L.moe_grad_clip(grads, out, norm, 0.5, coef)
        torch.cuda.synchronize()
        assert abs(float(norm) - float(want)) <= 1e-6 * float(want)
        for k in range(n):
            assert torch.equal(outs[k], before[2 * k * 8:(2 * k + 1) * 8] * coef), k
            if k % 3:
                assert torch.equal(ins[k], before[2 * k * 8:(2 * k + 1) * 8]), k
