"""Arguments and tensors that the dropout and the adapters refuse, before
anything is launched: no GPU is needed."""
import ctypes
import dataclasses
import inspect

import pytest

torch = pytest.importorskip("torch")

from synthetic import get_config  # noqa: E402
from tests.test_around_refusals import A, L, refused  # noqa: E402,F401
from tests.test_layer_arguments import calls  # noqa: E402,F401

F32, BF16 = torch.float32, torch.bfloat16


def test_dropout(L):  # noqa: F811
    def call(code, dtype=1, n=1024, x=A[0], res=A[1], p=0.1, rng=A[2], out=A[3]):
        refused(L, code, "moe_dropout", dtype, n, x, res, p, rng, out, 0)

    for kw in (dict(dtype=2), dict(n=-1), dict(p=1.0), dict(p=-0.1), dict(p=float("nan")), dict(x=None), dict(out=None),
               dict(rng=None), dict(x=A[0] + 8), dict(res=A[1] + 2), dict(out=A[3] + 4), dict(rng=A[2] + 4),
               dict(out=A[0] + 16), dict(out=A[1] - 16), dict(out=A[2]), dict(rng=A[3] + 1024)):
        call(1, **kw)
    call(2, n=1 << 42)
    L.moe_dropout(1, 0, None, None, 0.5, None, None, 0)

    def back(code, dy_t=0, dx_t=1, n=1024, dy=A[0], p=0.1, rng=A[1], dx=A[2]):
        refused(L, code, "moe_dropout_bwd", dy_t, dx_t, n, dy, p, rng, dx, 0)

    for kw in (dict(dy_t=2), dict(dx_t=-1), dict(p=2.0), dict(dy=None), dict(dx=None), dict(rng=None), dict(dx=A[0]),
               dict(dx=A[0] + 2048), dict(dy_t=1, dx=A[0] + 16), dict(n=-8)):
        back(1, **kw)


def shape(L, **kw):  # noqa: F811
    return L.MoEAdapterShape(**{**dict(T=64, d_in=64, d_out=128, n=4, rank=16, dtype=1, dropout=0.1), **kw})


BAD = (dict(T=-1), dict(d_in=0), dict(d_in=60), dict(d_out=132), dict(n=0), dict(rank=0), dict(rank=12), dict(dtype=2),
       dict(dropout=1.0), dict(dropout=-0.5), dict(dropout=float("nan")), dict(ld_in=56), dict(ld_in=68), dict(ld_out=120),
       dict(ld_out=-8), dict(dtype=0, rank=6), dict(dtype=0, d_in=66))
LARGE = (dict(T=1 << 31), dict(n=4097), dict(rank=136), dict(d_in=1 << 21), dict(d_out=(1 << 20) + 8), dict(ld_in=1 << 31))


def test_shapes(L):  # noqa: F811
    for kw in BAD + LARGE:
        s, code = shape(L, **kw), 1 if kw in BAD else 2
        assert L.moe_adapter_workspace_size(s) == 0 and L.moe_adapter_map_size(s) == 0 and not L.moe_adapter_rowwise(s)
        refused(L, code, "moe_adapter_map", s, A[0], A[1], A[2], 0)
        refused(L, code, "moe_adapter", s, *A[:4], None, None, A[4], None, A[5], None, A[6], 0)
        refused(L, code, "moe_adapter_bwd", s, 0, *A[:5], None, A[5], A[6], None, A[7], A[8], A[9], A[10], 0)
    small = shape(L)
    assert L.moe_adapter_workspace_size(small) % 256 == 0 and L.moe_adapter_map_size(small) % 256 == 0
    assert L.moe_adapter_rowwise(small) and not L.moe_adapter_rowwise(shape(L, T=8192, d_in=4096, d_out=4096))
    assert L.moe_adapter_workspace_size(shape(L, T=0)) >= 256


def test_map(L):  # noqa: F811
    def call(code, s=None, ids=A[0], m=A[1], ws=A[2]):
        refused(L, code, "moe_adapter_map", s or shape(L), ids, m, ws, 0)

    n = L.moe_adapter_map_size(shape(L))
    for kw in (dict(ids=None), dict(m=None), dict(ws=None), dict(ids=A[0] + 2), dict(m=A[1] + 8), dict(ws=A[2] + 4),
               dict(m=A[2]), dict(ids=A[1] + n - 4), dict(ids=A[2] + 16), dict(m=A[0] - n + 16)):
        call(1, **kw)


def test_adapter(L):  # noqa: F811
    def call(code, s=None, x=A[0], Aw=A[1], B=A[2], sc=A[3], ids=A[4], m=A[5], rng=A[6], base=A[7], y=A[8], u=A[9], ws=A[10]):
        refused(L, code, "moe_adapter", s or shape(L), x, Aw, B, sc, ids, m, rng, base, y, u, ws, 0)

    nws = L.moe_adapter_workspace_size(shape(L))
    for kw in (dict(x=None), dict(Aw=None), dict(B=None), dict(y=None), dict(ws=None), dict(rng=None), dict(x=A[0] + 8),
               dict(Aw=A[1] + 2), dict(B=A[2] + 8), dict(sc=A[3] + 2), dict(ids=A[4] + 1), dict(m=A[5] + 4), dict(rng=A[6] + 4),
               dict(base=A[7] + 8), dict(y=A[8] + 8), dict(u=A[9] + 4), dict(ws=A[10] + 8),
               # overlaps
               dict(y=A[0]), dict(y=A[0] + 64 * 64 * 2 - 16), dict(y=A[7] + 16), dict(y=A[1]), dict(y=A[2] + 16), dict(y=A[3]),
               dict(y=A[5]), dict(y=A[6]), dict(u=A[8]), dict(u=A[0]), dict(u=A[7]), dict(u=A[10] + nws - 16), dict(ws=A[1]),
               dict(ws=A[7]), dict(ws=A[8]), dict(u=A[2]), dict(m=None, y=A[4])):
        call(1, **kw)
    call(2, s=shape(L, T=1 << 28), m=None)
    # x and y as columns of one matrix: 64 columns of x, then 128 of y, rows of 256
    wide = dict(ld_in=256, ld_out=256)
    for x, y in ((A[0], A[0] + 112), (A[0], A[0] - 2 * 120), (A[0], A[0] + 2 * 200)):   # part of the rows in each other
        call(1, s=shape(L, **wide), x=x, y=y)
    call(1, s=shape(L, ld_in=256, ld_out=512), x=A[0], y=A[0] + 128)    # other distances: spans decide
    call(1, s=shape(L, **wide), x=A[0], y=A[0] + 128, ws=A[0] + 384)


def test_adapter_bwd(L):  # noqa: F811
    def call(code, s=None, t=0, dy=A[0], x=A[1], Aw=A[2], B=A[3], sc=A[4], m=A[5], rng=A[6], u=A[7], dx_in=None, dx=A[8], dA=A[9],
             dB=A[10], ws=A[11]):
        refused(L, code, "moe_adapter_bwd", s or shape(L), t, dy, x, Aw, B, sc, m, rng, u, dx_in, dx, dA, dB, ws, 0)

    for kw in (dict(t=2), dict(s=shape(L, dtype=0), t=1), dict(dy=None), dict(x=None), dict(Aw=None), dict(B=None), dict(u=None),
               dict(rng=None), dict(ws=None), dict(dA=None), dict(dB=None), dict(dx=None, dA=None, dB=None), dict(dy=A[0] + 8),
               dict(x=A[1] + 2), dict(Aw=A[2] + 8), dict(B=A[3] + 4), dict(sc=A[4] + 1), dict(m=A[5] + 8), dict(rng=A[6] + 2),
               dict(u=A[7] + 8), dict(dx_in=A[8] + 8), dict(dx=A[8] + 8), dict(dA=A[9] + 4), dict(dB=A[10] + 8), dict(ws=A[11] + 8),
               dict(dx=A[0]), dict(dx=A[1] + 16), dict(dx=A[2]), dict(dx=A[7]), dict(dx=A[9]), dict(dA=A[10]), dict(dA=A[1]),
               dict(dB=A[3]), dict(dB=A[7] + 16), dict(ws=A[0]), dict(ws=A[5]), dict(dx=A[11]), dict(dx_in=A[8] + 16),
               dict(dA=A[6]), dict(dx_in=A[9])):
        call(1, **kw)
    refused(L, 1, "moe_adapter_bwd", shape(L, T=0), 0, *[None] * 10, A[0], A[0] + 16, None, 0)


# ------------------------------------------------------------------------------------------------------------ tensors

NUMBERS = {"dtype": 1, "dy_dtype": 0, "dx_dtype": 0, "n": 64, "p": 0.1, "stream": 0}


@pytest.mark.parametrize("name", ["moe_dropout", "moe_dropout_bwd", "moe_adapter_map", "moe_adapter", "moe_adapter_bwd"])
def test_every_place(L, monkeypatch, name):  # noqa: F811
    """Tensors on another device or not contiguous, in every place of every call (slices where slices are wanted)."""
    made = []
    monkeypatch.setattr(L, "_call", lambda *args: made.append(args))
    args, places = {}, []
    for i, p in enumerate(inspect.signature(getattr(L, name)).parameters):
        if p in NUMBERS:
            args[p] = NUMBERS[p]
        elif p == "shape":
            args[p] = shape(L)
        else:
            args[p] = 1 << 32 | i << 24
            places.append(p)
    for current, bad in ((0, torch.zeros(8)), (-1, torch.zeros(8, 8).t()), (-1, torch.zeros(8)[::2])):
        monkeypatch.setattr(L, "_current", (lambda: 0, lambda: current))
        for p in places:
            with pytest.raises(ValueError):
                getattr(L, name)(**{**args, p: bad})
            assert not made, p
    monkeypatch.setattr(L, "_current", (lambda: 0, lambda: -1))
    tensors = {p: torch.zeros(8) for p in places}
    getattr(L, name)(**{**args, **tensors})
    getattr(L, name)(**{**args, **{p: t.data_ptr() for p, t in tensors.items()}})
    plain = [[None if isinstance(v, type(ctypes.byref(ctypes.c_int()))) else v for v in call] for call in made]
    assert plain[0] == plain[1]
    assert [v for v in plain[0] if v in {t.data_ptr() for t in tensors.values()}] == [t.data_ptr() for t in tensors.values()]


def test_slices(L, monkeypatch):  # noqa: F811
    """Rows as far apart as the shape says, and no others."""
    made = []
    monkeypatch.setattr(L, "_call", lambda *args: made.append(args))
    monkeypatch.setattr(L, "_current", (lambda: 0, lambda: -1))
    s = shape(L, ld_in=256, ld_out=384)
    x, y = torch.zeros(64, 256)[:, 32:96], torch.zeros(64, 384)[:, :128]
    rest = [None] * 5
    L.moe_adapter(s, x, 1, 1, *rest[:3], 1, y, y, None, 1, 0)
    assert len(made) == 1 and made[0][2] == x.data_ptr()
    for bad_x, bad_y in ((torch.zeros(64, 64), y), (x, torch.zeros(64, 512)[:, :128]), (torch.zeros(256, 64).t()[:, :64], y),
                         (x, torch.zeros(64, 128))):
        with pytest.raises(ValueError):
            L.moe_adapter(s, bad_x, 1, 1, *rest[:3], 1, bad_y, bad_y, None, 1, 0)
    with pytest.raises(ValueError):   # a slice where the shape says dense
        L.moe_adapter(shape(L), x, 1, 1, *rest[:3], 1, 1, 1, None, 1, 0)
    assert len(made) == 1


# --------------------------------------------------------------------------------------------------------------- layer

def _weights(cfg, n=3, rank=8, **more):
    dt = BF16 if cfg.dtype == "bf16" else F32
    w = {"W_r": torch.zeros(cfg.E, cfg.d, dtype=dt), "W_gu": torch.zeros(cfg.E, 2 * cfg.F, cfg.d, dtype=dt),
         "W_down": torch.zeros(cfg.E, cfg.d, cfg.F, dtype=dt), "gamma": torch.ones(cfg.d, dtype=dt),
         "lora_A": torch.zeros(n, rank, cfg.d, dtype=dt), "lora_B": torch.zeros(n, cfg.d, rank, dtype=dt)}
    w.update(more)
    return {k: v for k, v in w.items() if v is not None}


def _layer(dtype="bf16", weights=None, **kw):
    from token_dispatch_expert_moe_gb300.layer import MoELayer
    cfg = dataclasses.replace(get_config("tiny_f32"), T=48, dtype=dtype, backward=True)
    return cfg, MoELayer(cfg, _weights(cfg, **(weights or {})), device="cpu", backward=True, **kw)


def test_layer_options(calls):  # noqa: F811
    bad = [dict(weights=dict(lora_A=None)), dict(weights=dict(lora_B=None)), dict(weights=dict(rank=4)), dict(weights=dict(rank=136)),
           dict(weights=dict(lora_A=torch.zeros(3, 8, 64))), dict(weights=dict(lora_B=torch.zeros(3, 8, 64, dtype=BF16))),
           dict(weights=dict(lora_scale=torch.ones(3, dtype=BF16))), dict(weights=dict(lora_scale=torch.ones(4))),
           dict(weights=dict(lora_A=torch.zeros(3, 64, 8, dtype=BF16).transpose(1, 2))),
           dict(dropout=1.0), dict(dropout=-0.1), dict(adapter_dropout=1.5), dict(dropout=float("nan")),
           dict(dropout=0.1, weights=dict(gamma=None)), dict(adapter_dropout=0.1, weights=dict(lora_A=None, lora_B=None)),
           dict(weights=dict(lora_A=None, lora_B=None, lora_scale=torch.ones(3)))]
    for kw in bad:
        with pytest.raises(ValueError):
            _layer(**kw)
    assert not calls


def test_layer_calls(calls):  # noqa: F811
    cfg, layer = _layer(dropout=0.1, adapter_dropout=0.05, weights=dict(lora_scale=torch.ones(3)))
    T, d = cfg.T, cfg.d
    x, ids, rng = torch.zeros(T, d, dtype=BF16), torch.zeros(T, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.int64)
    for kw in (dict(adapter=ids.long()), dict(adapter=ids[1:]), dict(adapter=torch.zeros(T, 2, dtype=torch.int32)[:, 0]),
               dict(adapter=ids.to("meta")), dict(rng=rng[0]), dict(rng=rng.int()), dict(rng=rng.to("meta")),
               dict(rng=torch.zeros(2, 4, dtype=torch.int64)[:, ::2])):
        with pytest.raises(ValueError):
            layer.forward(x, residual=x, **kw)
        assert not calls, kw
    layer.forward(x, residual=x, adapter=ids, rng=rng)
    names = [c[0] for c in calls]
    assert names[0] == "moe_dropout" and names[1] == "moe_rmsnorm" and names[-2:] == ["moe_adapter_map", "moe_adapter"]
    assert calls[0][1][-3] == rng.data_ptr() and calls[-1][1][8 - 1] == rng.data_ptr() + 16
    del calls[:]
    layer.backward(x)
    assert [c[0] for c in calls][-1] == "moe_dropout_bwd" and "moe_adapter_bwd" in [c[0] for c in calls]
    del calls[:]
    layer.forward(x, residual=x)   # evaluation, one adapter for all
    names = [c[0] for c in calls]
    assert "moe_dropout" not in names and names[-1] == "moe_adapter" and "moe_adapter_map" not in names
    assert layer.adapter_shape.dropout == 0.0
    g = layer.backward(x)
    assert g["dx_drop"] is g["dx"] and {"dlora_A", "dlora_B"} <= set(g)
    assert len(layer.weight_grads()) == 6
    bare, plain = _layer(weights=dict(lora_A=None, lora_B=None))
    with pytest.raises(ValueError):
        plain.forward(x, adapter=ids)
