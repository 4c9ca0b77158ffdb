"""Tensors that MoELayer refuses before anything is launched. The layer is
built on the host and its calls are recorded instead of made: no GPU is
needed."""
import dataclasses

import pytest

torch = pytest.importorskip("torch")

from synthetic import get_config  # noqa: E402
from tests.test_around_refusals import L  # noqa: E402,F401


@pytest.fixture
def calls(L, monkeypatch):  # noqa: F811
    made = []
    monkeypatch.setattr(L, "_call", lambda name, *args: made.append((name, args)))
    monkeypatch.setattr(L, "_current", (lambda: 0, lambda: -1))   # the host in the current device's place
    return made


def _weights(cfg, gamma=True):
    dt = torch.bfloat16 if cfg.dtype == "bf16" else torch.float32
    w = {"W_r": torch.zeros(cfg.E, cfg.d, dtype=dt), "W_gu": torch.zeros(cfg.E, 2 * cfg.F, cfg.d, dtype=dt),
         "W_down": torch.zeros(cfg.E, cfg.d, cfg.F, dtype=dt)}
    if gamma:
        w["gamma"] = torch.ones(cfg.d, dtype=dt)
    return w


def _layer(dtype, gamma=True, **kw):
    from token_dispatch_expert_moe_gb300.layer import MoELayer
    cfg = dataclasses.replace(get_config("tiny_f32"), T=48, dtype=dtype, backward=True)
    return cfg, MoELayer(cfg, _weights(cfg, gamma), device="cpu", backward=True, **kw)


F32, BF16 = torch.float32, torch.bfloat16
# what a [T, d] tensor of the layer's type dt may not be
BAD = {"another type": lambda T, d, dt: torch.zeros(T, d, dtype=F32 if dt == BF16 else BF16),
       "half": lambda T, d, dt: torch.zeros(T, d, dtype=torch.float16),
       "a row less": lambda T, d, dt: torch.zeros(T - 1, d, dtype=dt),
       "strided": lambda T, d, dt: torch.zeros(d, T, dtype=dt).t(),
       "elsewhere": lambda T, d, dt: torch.zeros(T, d, dtype=dt, device="meta")}
# and, where every element of it is meant
WORSE = {**BAD, "transposed": lambda T, d, dt: torch.zeros(d, T, dtype=dt),
         "a row more": lambda T, d, dt: torch.zeros(T + 1, d, dtype=dt)}


@pytest.mark.parametrize("dtype,dt", [("bf16", BF16), ("f32", F32)])
@pytest.mark.parametrize("gamma", [True, False], ids=["normed", "bare"])
def test_rows(calls, dtype, dt, gamma):
    cfg, layer = _layer(dtype, gamma)
    T, d = cfg.T, cfg.d
    ok = torch.zeros(T, d, dtype=dt)
    for name, make in BAD.items():
        with pytest.raises(ValueError):
            layer.forward(make(T, d, dt))
        assert not calls, name
    if gamma:
        for name, make in WORSE.items():
            with pytest.raises(ValueError):
                layer.forward(ok, residual=make(T, d, dt))
            assert not calls, name
    layer.forward(ok, residual=ok if gamma else None)
    del calls[:]
    for name, make in BAD.items():
        with pytest.raises(ValueError):
            layer.backward(make(T, d, dt))
        assert not calls, name
    if gamma:
        for name, make in WORSE.items():
            with pytest.raises(ValueError):
                layer.backward(ok, dh=make(T, d, dt))
            assert not calls, name
    layer.backward(ok, dh=ok if gamma else None)
    assert calls


def test_a_bf16_layer_refuses_the_fp32_gradient_of_the_layer_above(calls):
    """dx is fp32 unless dx_dtype="act" asks for the layer's type, in which dh
    and dout are read."""
    for dx_dtype, taken in (("f32", False), ("act", True)):
        cfg, layer = _layer("bf16", dx_dtype=dx_dtype)
        x = torch.zeros(cfg.T, cfg.d, dtype=BF16)
        layer.forward(x)
        g = layer.backward(x, dh=x)
        for kw in (dict(dout=g["dx"], dh=x), dict(dout=x, dh=g["dx"])):
            if taken:
                layer.backward(**kw)
            else:
                with pytest.raises(ValueError, match="dx_dtype"):
                    layer.backward(**kw)


def test_mask_and_dloss(calls):
    cfg, layer = _layer("f32", balance=0.1)
    x = torch.zeros(cfg.T, cfg.d)
    for bad in (torch.ones(cfg.T, dtype=torch.int64), torch.ones(cfg.T), torch.ones(cfg.T, dtype=torch.float8_e4m3fn),
                torch.ones(cfg.T - 1, dtype=torch.uint8), torch.ones(cfg.T + 1, dtype=torch.uint8),
                torch.ones(2 * cfg.T, dtype=torch.uint8)[::2], torch.ones(cfg.T, dtype=torch.uint8, device="meta")):
        with pytest.raises(ValueError):
            layer.forward(x, mask=bad)
        assert not calls
    for mask in (torch.ones(cfg.T, dtype=torch.uint8), torch.ones(2, cfg.T // 2, dtype=torch.bool)):
        layer.forward(x, mask=mask)
    del calls[:]
    for bad in (torch.ones(1, dtype=torch.float64), torch.ones(1, dtype=BF16), torch.ones(2), torch.ones(0),
                torch.ones(1, device="meta")):
        with pytest.raises(ValueError):
            layer.backward(x, dloss=bad)
        assert not calls
    for dloss in (torch.ones(1), torch.tensor(1.0)):
        layer.backward(x, dloss=dloss)


def test_rows_with_more_dimensions(calls):
    """[batch, sequence, d] is the same memory as [T, d]."""
    cfg, layer = _layer("bf16", balance=0.1)
    x = torch.zeros(4, cfg.T // 4, cfg.d, dtype=BF16)
    layer.forward(x, residual=x)
    layer.backward(x, dh=x)
    bare = _layer("bf16", gamma=False)[1]
    bare.forward(torch.zeros(cfg.T + 8, cfg.d, dtype=BF16))   # a longer buffer: its first T rows
    assert calls


def test_gamma(calls):
    from token_dispatch_expert_moe_gb300.layer import MoELayer
    cfg = dataclasses.replace(get_config("tiny_f32"), T=48, dtype="bf16")
    for bad in (torch.ones(cfg.d), torch.ones(cfg.d - 8, dtype=BF16), torch.ones(2 * cfg.d, dtype=BF16)[::2],
                torch.ones(cfg.d, dtype=BF16, device="meta")):
        with pytest.raises(ValueError):
            MoELayer(cfg, {**_weights(cfg), "gamma": bad}, device="cpu")


def test_dx_put_in_another_buffer(calls):
    """layer.dx may be replaced between steps (a ring of outputs): the normed
    layer's gradient lands there, in fp32."""
    from token_dispatch_expert_moe_gb300 import _lib
    cfg, layer = _layer("bf16")
    x = torch.zeros(cfg.T, cfg.d, dtype=BF16)
    layer.forward(x)
    for _ in range(2):
        mine = layer.dx = torch.zeros(cfg.T, cfg.d)
        del calls[:]
        g = layer.backward(x)
        args = dict(calls)["moe_rmsnorm_bwd"]
        assert g["dx"] is mine
        assert args[2] == _lib.MOE_F32 and args[5] == args[10] == mine.data_ptr()


def test_clipping_follows_the_gradients_buffers(calls, L, monkeypatch):  # noqa: F811
    """A gradient put in another buffer after a first clip_grads is the one
    that is clipped."""
    listed = []

    class List:
        def __init__(self, tensors):
            self.tensors = list(tensors)
            listed.append([t.data_ptr() for t in self.tensors])
            self.n, self.address, self.device = len(self.tensors), 0, None

    monkeypatch.setattr(L, "TensorList", List)
    cfg, layer = _layer("bf16")
    layer.clip_grads(1.0)
    layer.clip_grads(1.0)
    assert len(listed) == 1   # the list is laid out once
    layer.dW_gu = torch.zeros_like(layer.dW_gu)
    layer.clip_grads(1.0)
    assert len(listed) == 2 and listed[1] == [t.data_ptr() for t in layer.weight_grads()]
