"""The norm's backward from several CUDA contexts of one device: the primary
one, the primary one after its reset, and one more. What was set for the kernels
in an earlier context (their shared memory limit) need not hold in a later one.
A process of its own, with the driver's API and libmoe.so alone."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

from tests.gpu_util import lib  # noqa: E402


def _child():
    import ctypes as C
    cu = C.CDLL("libcuda.so.1")
    moe = C.CDLL(sys.argv[1])
    moe.moe_rmsnorm_bwd_workspace_size.restype = C.c_size_t
    moe.moe_rmsnorm_bwd_workspace_size.argtypes = [C.c_int64, C.c_int32]
    P = C.c_void_p
    moe.moe_rmsnorm_bwd.argtypes = [C.c_int32] * 3 + [C.c_int64, C.c_int32] + [P] * 8 + [C.c_size_t, P]

    def ok(rc):
        assert rc == 0, rc

    ok(cu.cuInit(0))
    dev, seen = C.c_int(), []
    ok(cu.cuDeviceGet(C.byref(dev), 0))
    rows, d = 4, 8192
    nws = moe.moe_rmsnorm_bwd_workspace_size(rows, d)
    n = rows * d * 4
    sizes = dict(dy=n, h=n, gamma=4 * d, rstd=256, dh=n, dx=n, dgamma=4 * d, ws=nws)
    for i in ("primary", "primary after its reset", "another"):
        ctx, at = P(), {}
        if i == "another":
            ok(cu.cuCtxCreate_v2(C.byref(ctx), 0, dev))
        else:
            if seen:
                ok(cu.cuDevicePrimaryCtxReset_v2(dev))
            ok(cu.cuDevicePrimaryCtxRetain(C.byref(ctx), dev))
            ok(cu.cuCtxSetCurrent(ctx))
        for k, b in sizes.items():
            at[k] = C.c_uint64()
            ok(cu.cuMemAlloc_v2(C.byref(at[k]), C.c_size_t(b)))
            ok(cu.cuMemsetD8_v2(at[k], C.c_ubyte(0x3f), C.c_size_t(b)))   # 0.747 in fp32
        ok(cu.cuCtxSynchronize())
        p = {k: v.value for k, v in at.items()}
        rc = moe.moe_rmsnorm_bwd(0, 0, 0, rows, d, p["dy"], p["h"], p["gamma"], p["rstd"], p["dh"], p["dx"], p["dgamma"],
                                 p["ws"], nws, None)
        assert rc == 0, f"{i}: status {rc}"
        ok(cu.cuCtxSynchronize())
        out = (C.c_float * (rows * d))()
        ok(cu.cuMemcpyDtoH_v2(out, at["dx"], C.c_size_t(n)))
        seen.append(list(out))
    assert seen[0] == seen[1] == seen[2]
    v = 0.747058808803558   # g = v v, xhat = v v: dx = v (g - xhat^2 g) + v
    want = v * (v * v - v * v * v ** 4) + v
    assert all(abs(x - want) <= 1e-5 * want for x in seen[0][::997]), (seen[0][0], want)
    ok(cu.cuCtxDestroy_v2(ctx))


@pytest.mark.gpu
def test_contexts_one_after_the_other():
    L = lib()
    r = subprocess.run([sys.executable, os.path.abspath(__file__), L.LIB_PATH], capture_output=True, text=True, timeout=120,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       env={**os.environ, "PYTHONPATH": os.path.dirname(os.path.dirname(os.path.abspath(__file__)))})
    assert r.returncode == 0, r.stderr[-1500:]


if __name__ == "__main__":
    _child()
