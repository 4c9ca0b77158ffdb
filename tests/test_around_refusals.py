"""Arguments that the operators around the layer refuse, before anything is
launched: no GPU is needed."""
import ctypes
import os

import pytest


@pytest.fixture(scope="module")
def L():
    from token_dispatch_expert_moe_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    from token_dispatch_expert_moe_gb300 import _lib
    return _lib


A = [1 << 32 | i << 24 for i in range(12)]   # addresses 16 MB apart, never dereferenced


def refused(L, code, fn, *args, **kw):
    with pytest.raises(L.MoEError) as e:
        getattr(L, fn)(*args, **kw)
    assert e.value.code == code, (fn, args, e.value)


def test_rmsnorm(L):
    def call(code, dtype=1, rows=4, d=256, x=A[0], res=A[1], gamma=A[2], eps=1e-5, h=A[3], y=A[4], q=A[5], s=A[6],
             group=128, rstd=A[7]):
        refused(L, code, "moe_rmsnorm", dtype, rows, d, x, res, gamma, eps, h, y, q, s, group, rstd, 0)

    for kw in (dict(dtype=2), dict(rows=-1), dict(d=0), dict(d=252), dict(dtype=0, d=254), dict(x=None),
               dict(gamma=None), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(s=None), dict(q=None), dict(h=None, y=None, q=None, s=None), dict(group=-32), dict(x=A[0] + 8),
               dict(res=A[1] + 2), dict(gamma=A[2] + 4), dict(h=A[3] + 8), dict(y=A[4] + 8), dict(q=A[5] + 8),
               dict(s=A[6] + 2), dict(rstd=A[7] + 1),
               # overlaps: outputs with each other, with part of an input, 8-bit rows in an input's place
               dict(h=A[4]), dict(y=A[5]), dict(q=A[0]), dict(h=A[0] + 512), dict(y=A[1] - 512), dict(h=A[2]),
               dict(rstd=A[0]), dict(s=A[2]), dict(rstd=A[6])):
        call(1, **kw)
    for kw in (dict(group=16), dict(group=256), dict(d=32776), dict(dtype=0, d=16388), dict(rows=1 << 31)):
        call(2, **kw)
    L.moe_rmsnorm(1, 0, 256, None, None, None, 1e-5, A[3], None, None, None, 0, None, 0)   # no rows: nothing to do


def test_rmsnorm_bwd(L):
    assert L.moe_rmsnorm_bwd_workspace_size(1, 8) >= 32
    assert L.moe_rmsnorm_bwd_workspace_size(1 << 20, 8192) == 1024 * 8192 * 4
    for rows, d in ((-1, 8), (1 << 31, 8), (4, 0), (4, 32776)):
        assert L.moe_rmsnorm_bwd_workspace_size(rows, d) == 0
    n = L.moe_rmsnorm_bwd_workspace_size(4, 256)

    def call(code, dtype=1, dy_t=0, dx_t=0, rows=4, d=256, dy=A[0], h=A[1], gamma=A[2], rstd=A[3], dh=A[4], dx=A[5],
             dg=A[6], ws=A[7], nb=n):
        refused(L, code, "moe_rmsnorm_bwd", dtype, dy_t, dx_t, rows, d, dy, h, gamma, rstd, dh, dx, dg, ws, 0, ws_bytes=nb)

    for kw in (dict(dtype=3), dict(dy_t=2), dict(dx_t=-1), dict(dtype=0, dy_t=1), dict(dtype=0, dx_t=1), dict(rows=-1),
               dict(d=12), dict(dy=None), dict(h=None), dict(gamma=None), dict(rstd=None), dict(dx=None), dict(dg=None),
               dict(ws=None), dict(nb=n - 1), dict(dy=A[0] + 8), dict(dx=A[5] + 8), dict(dh=A[4] + 8), dict(ws=A[7] + 8),
               dict(dg=A[6] + 4), dict(rstd=A[3] + 2),
               # dx over h, over half of dy, over dh or dy of another type; dgamma or ws over an input
               dict(dx=A[1]), dict(dx=A[0] + 1024), dict(dx=A[4]), dict(dx=A[0], dx_t=1), dict(dx=A[2]), dict(dx=A[7]),
               dict(dg=A[0]), dict(ws=A[1]), dict(dg=A[7]), dict(dx=A[6])):
        call(1, **kw)
    for kw in (dict(d=32776), dict(dtype=0, d=16388), dict(rows=1 << 31)):
        call(2, **kw)


def _shape(L, **kw):
    return L.MoEShape(**{**dict(T=64, d=64, E=8, K=2, F=64, dtype=1, subseq_len=16), **kw})


def test_balance(L):
    def call(code, shape=None, logits=A[0], idx=A[1], mask=A[2], alpha=0.1, loss=A[3], counts=A[4], prob=A[5], coef=A[6],
             ws=A[7]):
        refused(L, code, "moe_balance_loss", shape or _shape(L), logits, idx, mask, alpha, loss, counts, prob, coef, ws, 0)

    for kw in (dict(shape=_shape(L, E=65)), dict(shape=_shape(L, T=0)), dict(shape=_shape(L, K=9)),
               dict(shape=_shape(L, subseq_len=-1)), dict(logits=None), dict(idx=None), dict(loss=None),
               dict(counts=None), dict(coef=None), dict(ws=None), dict(alpha=float("nan")), dict(alpha=float("inf")),
               dict(logits=A[0] + 4), dict(ws=A[7] + 8), dict(prob=A[5] + 2), dict(idx=A[1] + 1), dict(coef=A[6] + 4)):
        call(1, **kw)

    def back(code, shape=None, logits=A[0], mask=None, coef=A[1], dloss=None, dl=A[2]):
        refused(L, code, "moe_balance_loss_bwd", shape or _shape(L), logits, mask, coef, dloss, dl, 0)

    for kw in (dict(shape=_shape(L, E=0)), dict(logits=None), dict(coef=None), dict(dl=None), dict(dl=A[2] + 4),
               dict(dloss=A[3] + 2), dict(dl=A[0] + 16), dict(coef=A[1] + 8)):
        back(1, **kw)

    def route(add, logits=A[2], shape=None):
        refused(L, 1, "moe_route_bwd_add", shape or _shape(L), A[0], A[1], None, logits, A[3], A[4], A[5], A[6], None, add,
                None, A[7], None, None, A[8], A[9], 0)

    route(None)
    route(A[10] + 2)
    route(A[2])              # the logits themselves, overwritten by moe_balance_loss_bwd
    route(A[2] + 64 * 8 * 4 - 4)
    route(A[10], shape=_shape(L, E=65))


def test_permute_e4m3(L):
    def call(code, shape=None, q=A[0], s=A[1], group=32, idx=A[2], keep=A[3], Xp=A[4], row=A[5], src=A[6], cnt=A[7],
             off=A[8], ws=A[9]):
        refused(L, code, "moe_permute_e4m3", shape or _shape(L), q, s, group, idx, keep, Xp, row, src, cnt, off, ws, 0)

    for k in ("q", "s", "idx", "keep", "Xp", "row", "src", "cnt", "off", "ws"):
        call(1, **{k: None})
    for kw in (dict(group=-1), dict(q=A[0] + 8), dict(s=A[1] + 2), dict(Xp=A[4] + 8), dict(ws=A[9] + 4),
               dict(shape=_shape(L, T=0))):
        call(1, **kw)
    call(2, group=16)
    call(2, group=96)
    call(2, shape=_shape(L, d=102408))
    call(2, shape=_shape(L, d=51204, dtype=0))


def test_grads(L):
    class List:
        def __init__(self, *t):
            self.n = len(t)
            self.array = (L.MoETensor * max(1, len(t)))(*[L.MoETensor(*x) for x in t])
            self.address = ctypes.addressof(self.array)
            self.device = None

    nb = L.MOE_GRAD_NORM_WORKSPACE_BYTES
    ok = List((A[0], 100, 0), (A[1], 100, 1), (None, 0, 0))

    def norm(code, grads=ok, norm=A[2], ws=A[3], nb=nb):
        refused(L, code, "moe_grad_norm", grads, norm, ws, 0, ws_bytes=nb)

    neg = List()
    neg.n = -1
    for kw in (dict(grads=neg), dict(grads=List((A[0], -1, 0))), dict(grads=List((A[0], 1, 2))),
               dict(grads=List((None, 1, 0))), dict(grads=List((A[0] + 2, 1, 0))), dict(grads=List((A[0] + 1, 1, 1))),
               dict(norm=None), dict(norm=A[2] + 2), dict(ws=None), dict(ws=A[3] + 8), dict(nb=nb - 1)):
        norm(1, **kw)

    def clip(code, grads=ok, out=None, norm=A[2], max_norm=1.0, coef=None):
        refused(L, code, "moe_grad_clip", grads, out, norm, max_norm, coef, 0)

    for kw in (dict(norm=None), dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(max_norm=float("inf")),
               dict(coef=A[4] + 2), dict(out=List((A[4], 100, 0))),                              # fewer tensors
               dict(out=List((A[4], 99, 0), (A[5], 100, 1), (None, 0, 0))),                      # another size
               dict(out=List((A[4], 100, 1), (A[5], 100, 1), (None, 0, 0))),                     # another type
               dict(out=List((A[0] + 4, 100, 0), (A[5], 100, 1), (None, 0, 0)))):                # over part of its gradient
        clip(1, **kw)


def test_tensor_list(L):
    torch = pytest.importorskip("torch")
    for bad in (torch.zeros(4), torch.zeros(4, dtype=torch.float64), torch.zeros(4, 4).t()[:, ::2]):
        with pytest.raises(ValueError):
            L.TensorList([bad])
    assert L.TensorList([]).n == 0


@pytest.mark.gpu
def test_tensors_that_the_binding_refuses(L):
    """Strided or host tensors, and lists whose tensors share memory: nothing
    is launched."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    x = torch.zeros(8, 64, device="cuda", dtype=torch.bfloat16)
    g, y = x[0].clone(), torch.empty_like(x)
    for bad in (x.t(), x[:, ::2], x.cpu()):
        with pytest.raises(ValueError):
            L.moe_rmsnorm(1, 8, 64, bad, None, g, 1e-5, None, y, None, None, 0, None)
    flat = torch.zeros(100, device="cuda")
    for shared in ([flat, flat], [flat[:60], flat[59:]], [flat[50:], flat]):
        with pytest.raises(ValueError):
            L.TensorList(shared)
    assert L.TensorList([flat[:60], flat[60:], flat[:0]]).n == 3


def test_constants_match_header(L):
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    txt = open(os.path.join(root, "include", "moe.h")).read()
    m = re.search(r"#define\s+MOE_GRAD_NORM_WORKSPACE_BYTES\s+(\d+)u?", txt)
    assert m and int(m.group(1)) == L.MOE_GRAD_NORM_WORKSPACE_BYTES
