"""Tensors that the binding of the operators around the layer refuses, in every
place of every call: on the host or another device, or not contiguous. The
calls are recorded instead of made: no GPU is needed."""
import ctypes
import inspect

import pytest

torch = pytest.importorskip("torch")

from tests.test_around_refusals import L, _shape  # noqa: E402,F401

NUMBERS = {"dtype": 1, "dy_dtype": 0, "dx_dtype": 0, "rows": 4, "d": 256, "eps": 1e-5, "group": 128, "alpha": 0.1,
           "max_norm": 1.0, "stream": 0, "ws_bytes": 1 << 20}
CALLS = ["moe_rmsnorm", "moe_rmsnorm_bwd", "moe_balance_loss", "moe_balance_loss_bwd", "moe_route_bwd_add",
         "moe_permute_e4m3", "moe_grad_norm", "moe_grad_clip"]


def _tensors(L, name):  # noqa: F811
    """The call's arguments by name, addresses for its tensors, and the tensors' names."""
    class List:
        n, address, device = 0, 0, None

    args, places = {}, []
    for i, p in enumerate(inspect.signature(getattr(L, name)).parameters):
        if p in NUMBERS:
            args[p] = NUMBERS[p]
        elif p == "shape":
            args[p] = _shape(L)
        elif p == "grads" or (p == "out" and name == "moe_grad_clip"):
            args[p] = List() if p == "grads" else None
        else:
            args[p] = 1 << 32 | i << 24
            places.append(p)
    return args, places


@pytest.mark.parametrize("name", CALLS)
def test_every_place(L, monkeypatch, name):  # noqa: F811
    made = []
    monkeypatch.setattr(L, "_call", lambda *args: made.append(args))
    args, places = _tensors(L, name)
    assert len(places) >= 2
    for current, bad in ((0, torch.zeros(8)), (-1, torch.zeros(8, 8).t()), (-1, torch.zeros(8)[::2])):
        monkeypatch.setattr(L, "_current", (lambda: 0, lambda: current))
        for p in places:
            with pytest.raises(ValueError):
                getattr(L, name)(**{**args, p: bad})
            assert not made, p
    # tensors on the current device, each in its own place of the C call
    monkeypatch.setattr(L, "_current", (lambda: 0, lambda: -1))
    tensors = {p: torch.zeros(8) for p in places}
    getattr(L, name)(**{**args, **tensors})
    getattr(L, name)(**{**args, **{p: t.data_ptr() for p, t in tensors.items()}})
    assert len(made) == 2
    plain = [[None if isinstance(v, type(ctypes.byref(ctypes.c_int()))) else v for v in call] for call in made]
    assert plain[0] == plain[1]
    assert [v for v in plain[0] if v in {t.data_ptr() for t in tensors.values()}] == [t.data_ptr() for t in tensors.values()]
