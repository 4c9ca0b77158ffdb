"""The dropout's mask and the adapters' formulas in plain 64-bit form, with the error that the kernels' arithmetic may
leave on each result.

Rounding units: a sum of n terms in fp32 is off by at most n 2^-23 times the sum of the terms' sizes, whatever its order and
whether additions round (2^-24) or truncate (2^-23, tensor cores). bf16 kernels hold u and du in two bf16 parts: what is left
out is 2^-8 of the second part, which is 2^-8 of the first: 2^-16. A result in bf16 is rounded by at most 2^-8 of itself."""
import numpy as np
import torch

U32 = 2.0 ** -23
PARTS = 2.0 ** -16


def threshold(p):
    return min(65535, int(np.floor(float(np.float32(p)) * 65536 + 0.5)))


def factor(p):
    return 65536.0 / (65536 - threshold(p))


def words(blocks, seed, offset):
    """Philox4x32-10 of 64-bit counters `blocks`: [n, 4] 32-bit words."""
    b = np.asarray(blocks, np.uint64)
    m = np.uint64(0xFFFFFFFF)
    s32 = np.uint64(32)
    x = [b & m, b >> s32, np.full_like(b, offset & 0xFFFFFFFF), np.full_like(b, offset >> 32)]
    for i in range(10):
        k = [np.uint64((seed + i * 0x9E3779B9) & 0xFFFFFFFF), np.uint64(((seed >> 32) + i * 0xBB67AE85) & 0xFFFFFFFF)]
        a, c = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(c >> s32) ^ x[1] ^ k[0], c & m, (a >> s32) ^ x[3] ^ k[1], a & m]
    return np.stack(x, 1)


def mask(n, p, seed, offset, first=0):
    """Kept elements first .. first + n (first a multiple of 8)."""
    w = words(np.arange(first // 8, (first + n + 7) // 8), seed, offset)
    halves = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], 2).reshape(-1)
    return torch.from_numpy(halves[:n] >= threshold(p))


def rng_tensor(seed, offset, device="cuda"):
    return torch.from_numpy(np.array([seed, offset], np.uint64).view(np.int64)).to(device)


def dropped(x, p, seed, offset):
    """drop(x) of a dense matrix, in 64 bits."""
    if p == 0:
        return x.double()
    keep = mask(x.numel(), p, seed, offset).view(x.shape).to(x.device)
    return torch.where(keep, x.double() * factor(p), 0.0)


def round_to(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24


def forward(x, A, B, scale, ids, base, p=0.0, seed=0, offset=0):
    """(y, bound of y, u, bound of u)."""
    parts = PARTS if x.dtype == torch.bfloat16 else 0.0
    xd = dropped(x, p, seed, offset)
    T, r, d = x.shape[0], A.shape[1], A.shape[2]
    u = torch.zeros(T, r, dtype=torch.float64, device=x.device)
    eu = torch.zeros_like(u)
    y = torch.zeros(T, B.shape[1], dtype=torch.float64, device=x.device) if base is None else base.double()
    ey = y.abs() * 0
    for a in ids.unique().tolist():
        if a < 0:
            continue
        t = torch.nonzero(ids == a)[:, 0]
        Aa, Ba, s = A[a].double(), B[a].double(), 1.0 if scale is None else float(scale[a])
        u[t] = xd[t] @ Aa.T
        eu[t] = (d + 4) * U32 * (xd[t].abs() @ Aa.abs().T)
        delta = u[t] @ Ba.T * s
        ey[t] = s * (eu[t] @ Ba.abs().T + ((r + 4) * U32 + parts) * (u[t].abs() @ Ba.abs().T))
        y[t] += delta
    ey = ey * (1 + 2.0 ** -7) + (y.abs() + ey) * (round_to(x.dtype) + 2 * U32)
    return y, ey, u, eu + u.abs() * 2 * U32


def backward(dy, x, A, B, scale, ids, u, dx_in, dx_dtype, p=0.0, seed=0, offset=0):
    """({dx, dA, dB}, their bounds)."""
    parts = PARTS if x.dtype == torch.bfloat16 else 0.0
    xd = dropped(x, p, seed, offset)
    keep = dropped(torch.ones_like(x, dtype=torch.float64), p, seed, offset)
    T, d, dout, r = x.shape[0], A.shape[2], B.shape[1], A.shape[1]
    zero = lambda *s: torch.zeros(*s, dtype=torch.float64, device=x.device)  # noqa: E731
    dx = zero(T, d) if dx_in is None else dx_in.double()
    dA, dB, edx, edA, edB = zero(*A.shape), zero(*B.shape), zero(T, d), zero(*A.shape), zero(*B.shape)
    for a in ids.unique().tolist():
        if a < 0:
            continue
        t = torch.nonzero(ids == a)[:, 0]
        n = len(t)
        Aa, Ba, s = A[a].double(), B[a].double(), 1.0 if scale is None else float(scale[a])
        g = dy[t].double()
        du = s * (g @ Ba)
        edu = s * (dout + 4) * U32 * (g.abs() @ Ba.abs()) + du.abs() * 2 * U32
        edu = edu + parts * (du.abs() + edu)
        dx[t] += du @ Aa * keep[t]
        edx[t] = (edu @ Aa.abs() + (r + 6) * U32 * (du.abs() @ Aa.abs())) * keep[t]
        dA[a] = du.T @ xd[t]
        edA[a] = edu.T @ xd[t].abs() + (n + 20) * U32 * (du.abs().T @ xd[t].abs())
        ud = u[t].double()
        dB[a] = s * (g.T @ ud)
        edB[a] = s * ((n + 20) * U32 + parts) * (g.abs().T @ ud.abs())
    edx = edx * (1 + 2.0 ** -7) + (dx.abs() + edx) * (round_to(dx_dtype) + 2 * U32)
    return {"dx": dx, "dA": dA, "dB": dB}, {"dx": edx, "dA": edA * (1 + 2.0 ** -7), "dB": edB * (1 + 2.0 ** -7)}


def within(name, got, want, bound):
    assert got.shape == want.shape, (name, got.shape, want.shape)
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), (f"{name}: {int(bad.sum())} of {bad.numel()} outside, first at {torch.nonzero(bad)[0].tolist()}, "
                                 f"largest error {float(err[bad].max()):.3e} where {float(bound[bad].min()):.3e} is allowed")
