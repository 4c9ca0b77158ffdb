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
