"""Workloads of the low-rank adapters beside a projection, chosen per token, and of the dropout whose mask is never stored,
each forward and backward. `own` chooses between the framework's kernels and the operators' plain form in elementary torch
operations."""
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


# ---------------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token on the Mixtral-8x22B hidden size, a server with 64 adapters in memory
        dict(name="adapter one token", op="adapter", T=1, d_in=6144, d_out=6144, n=64, rank=16, dtype="bf16", p=0.0,
             order="mixed", bare=0.0),
        # a decode batch of 64 requests, nearly all with adapters of their own
        dict(name="adapter decode", op="adapter", T=64, d_in=6144, d_out=6144, n=128, rank=16, dtype="bf16", p=0.0,
             order="mixed", bare=0.1),
        # a ragged prefill batch of the Qwen2-57B-A14B hidden size: packed requests into an expert's gate and up columns
        dict(name="adapter ragged prefill", op="adapter", T=1021, d_in=3584, d_out=5120, n=12, rank=24, dtype="bf16", p=0.0,
             order="packed", bare=0.2),
        # a large serving batch, G8T8-sized, of higher rank
        dict(name="adapter large prefill", op="adapter", T=16384, d_in=6144, d_out=6144, n=32, rank=64, dtype="bf16", p=0.0,
             order="packed", bare=0.0),
        # fine-tuning one adapter with dropout on the Llama3-8x70B training batch
        dict(name="adapter training", op="adapter", T=32768, d_in=8192, d_out=8192, n=1, rank=16, dtype="bf16", p=0.1,
             order="packed", bare=0.0),
        # the checking case's sizes, tokens of four adapters in any order
        dict(name="adapter bwd tiny f32", op="adapter_bwd", T=512, d_in=64, d_out=64, n=4, rank=4, dtype="f32", p=0.0,
             order="mixed", bare=0.1, dx="f32"),
        # eight users' adapters trained at once on a Qwen2-57B-A14B batch, fp32 gradient joined to the layer's
        dict(name="adapter bwd several", op="adapter_bwd", T=8192, d_in=3584, d_out=3584, n=8, rank=32, dtype="bf16", p=0.0,
             order="packed", bare=0.1, dx="f32"),
        # the backward of the fine-tuning step
        dict(name="adapter bwd training", op="adapter_bwd", T=32768, d_in=8192, d_out=8192, n=1, rank=16, dtype="bf16", p=0.1,
             order="packed", bare=0.0, dx="bf16"),
        # the residual dropout of the checking case
        dict(name="dropout tiny f32", op="dropout", rows=512, d=64, dtype="f32", p=0.1, residual=True),
        # ... and of the Llama3-8x70B training batch
        dict(name="dropout training", op="dropout", rows=32768, d=8192, dtype="bf16", p=0.1, residual=True),
        # a ragged batch's gradient, fp32 from the norm's backward to the layer below's bf16
        dict(name="dropout bwd ragged", op="dropout_bwd", rows=1021, d=3584, dtype="bf16", dy="f32", p=0.05),
        # the training batch's gradient in bf16
        dict(name="dropout bwd training", op="dropout_bwd", rows=32768, d=8192, dtype="bf16", dy="bf16", p=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["adapter", "adapter", "adapter_bwd", "adapter_bwd", "dropout", "dropout_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("adapter"):
        T, n = _log(rng, 1, 32768), _log(rng, 1, 128)
        d_in, d_out = 8 * _log(rng, 8, 1024), 8 * _log(rng, 8, 1024)
        rank = 8 * _log(rng, 1, 16) if dtype == "bf16" else 4 * _log(rng, 1, 16)
        while T * (d_in + d_out) * (1 if dtype == "bf16" else 4) * max(rank, 16) > 32768 * 16384 * 16:
            T = (T + 1) // 2
        c = dict(op=op, T=T, d_in=d_in, d_out=d_out, n=n, rank=rank, dtype=dtype, p=rng.choice([0.0, 0.0, 0.05, 0.1, 0.5]),
                 order=rng.choice(["packed", "packed", "mixed"]), bare=rng.choice([0.0, 0.1, 0.4]))
        if op == "adapter_bwd":
            c["dx"] = "f32" if dtype == "f32" else rng.choice(["f32", "bf16"])
        return c
    rows, d = _log(rng, 1, 32768), 4 * _log(rng, 4, 2048) + rng.choice([0, 0, 0, 1, 2, 3])
    while rows * d * (2 if dtype == "f32" else 1) > 32768 * 8192:
        rows //= 2
    c = dict(op=op, rows=rows, d=d, dtype=dtype, p=rng.choice([0.02, 0.1, 0.1, 0.5]))
    if op == "dropout":
        c["residual"] = rng.random() < 0.7
    else:
        c["dy"] = rng.choice(["f32", "bf16"])
    return c


# --------------------------------------------------------------------------------------------------------------- inputs

def _requests(c, g):
    """Adapter of each token, -1 for none: requests of different lengths one after another, or any token any adapter."""
    T, n = c["T"], c["n"]
    rand = lambda *s: torch.rand(*s, device="cuda", generator=g)  # noqa: E731
    if c["order"] == "mixed":
        ids = (rand(T) * n).int().clamp_max(n - 1)
        return torch.where(rand(T) < c["bare"], -1, ids)
    m = min(T, n + n // 4 + 1) if n > 1 else 1          # some adapters serve more than one request
    cut = (rand(m) + 0.05).cumsum(0)
    end = (cut / cut[-1] * T).round().long()
    who = (rand(m) * n).int().clamp_max(n - 1)
    who = torch.where(rand(m) < c["bare"], -1, who)
    t = torch.arange(T, device="cuda")
    return who[torch.searchsorted(end, t, right=True).clamp_max(m - 1)]


def prepare(case, seed):
    c, g = dict(case), torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s, dt="f32", std=1.0: torch.randn(*s, device="cuda", generator=g).mul_(std).to(DT[dt])  # noqa: E731
    s = dict(case=c)
    # seed and offset of the generator, as a training step counts them up
    s["rng"] = torch.randint(0, 2 ** 62, (2,), device="cuda", generator=g)
    if c["op"].startswith("adapter"):
        T, d_in, d_out, n, r, dt = c["T"], c["d_in"], c["d_out"], c["n"], c["rank"], c["dtype"]
        s["x"] = randn(T, d_in, dt=dt)
        s["A"] = randn(n, r, d_in, dt=dt, std=d_in ** -0.5)
        s["B"] = randn(n, d_out, r, dt=dt, std=r ** -0.5)
        s["scale"] = 0.25 + 1.5 * torch.rand(n, device="cuda", generator=g)   # alpha / rank
        s["ids"] = _requests(c, g)
        # a program knows its requests on the host: each adapter's tokens, and the tokens without one
        ids = s["ids"].cpu()
        s["groups"] = [(a, (ids == a).nonzero()[:, 0].cuda()) for a in ids.unique().tolist()]
        if c["op"] == "adapter":
            s["base"] = randn(T, d_out, dt=dt)
        else:
            s["dy"] = randn(T, d_out, dt=dt, std=0.1)
            s["dx_in"] = randn(T, d_in, dt=c["dx"], std=0.1)
            s["u"] = randn(T, r)
            s["u"][s["ids"] < 0] = 0
    else:
        rows, d = c["rows"], c["d"]
        if c["op"] == "dropout":
            s["x"] = randn(rows, d, dt=c["dtype"])
            s["r"] = randn(rows, d, dt=c["dtype"], std=2.0) if c["residual"] else None
        else:
            s["dy"] = randn(rows, d, dt=c["dy"], std=0.1)
    return s


# ----------------------------------------------------------------------------------------------------------- plain forms

M32 = 0xFFFFFFFF


def _threshold(p):
    return min(65535, int(p * 65536 + 0.5))


def _kept(n, rng, p):
    """The kept ones of n elements: Philox4x32-10, one block of eight 16-bit numbers for eight elements."""
    b = torch.arange((n + 7) // 8, device="cuda")
    c0, c1, c2, c3 = b & M32, b >> 32, rng[1] & M32, (rng[1] >> 32) & M32
    k0, k1 = rng[0] & M32, (rng[0] >> 32) & M32
    for _ in range(10):
        a, e = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((e >> 32) & M32) ^ c1 ^ k0, e & M32, ((a >> 32) & M32) ^ c3 ^ k1, a & M32
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    u = torch.stack([v for w in (c0, c1, c2, c3) for v in (w & 0xFFFF, w >> 16)], dim=1)
    return (u >= _threshold(p)).view(-1)[:n]


def _dropped(x, rng, p):
    if p == 0.0:
        return x.float()
    return x.float() * _kept(x.numel(), rng, p).view(x.shape) * (65536.0 / (65536 - _threshold(p)))


def _plain_adapter(s):
    c = s["case"]
    T, r, dt = c["T"], c["rank"], DT[c["dtype"]]
    x = _dropped(s["x"], s["rng"], c["p"])
    if T <= 64:   # a decode batch: each token's adapter gathered, in a few batched steps
        a = s["ids"].long().clamp_min(0)
        has = (s["ids"] >= 0)[:, None]
        u = (s["A"][a].float() * x[:, None, :]).sum(2) * has
        y = s["base"].float() + s["scale"][a][:, None] * (s["B"][a].float() * u[:, None, :]).sum(2)
        return {"y": y.to(dt), "u": u}
    y, u = s["base"].float(), torch.zeros(T, r, device="cuda")
    for a, at in s["groups"]:
        if a >= 0:
            ua = x[at] @ s["A"][a].float().T
            u[at] = ua
            y[at] += s["scale"][a] * (ua @ s["B"][a].float().T)
    return {"y": y.to(dt), "u": u}


def _plain_adapter_bwd(s):
    c = s["case"]
    x, dy = _dropped(s["x"], s["rng"], c["p"]), s["dy"].float()
    dx = torch.zeros_like(x)
    dA = torch.zeros(s["A"].shape, device="cuda")
    dB = torch.zeros(s["B"].shape, device="cuda")
    for a, at in s["groups"]:
        if a >= 0:
            g = dy[at] * s["scale"][a]
            du = g @ s["B"][a].float()
            dx[at] = du @ s["A"][a].float()
            dA[a] = du.T @ x[at]
            dB[a] = g.T @ s["u"][at]
    return {"dx": (s["dx_in"].float() + _dropped(dx, s["rng"], c["p"])).to(DT[c["dx"]]), "dA": dA, "dB": dB}


def _plain_dropout(s):
    out = _dropped(s["x"], s["rng"], s["case"]["p"])
    if s["r"] is not None:
        out = out + s["r"].float()
    return {"out": out.to(DT[s["case"]["dtype"]])}


def _plain_dropout_bwd(s):
    return {"dx": _dropped(s["dy"], s["rng"], s["case"]["p"]).to(DT[s["case"]["dtype"]])}


# ---------------------------------------------------------------------------------------------------- the framework's

def _code(L, name):
    return L.MOE_BF16 if name == "bf16" else L.MOE_F32


def _plan(s, L):
    """The shape, the workspace and the map's buffer; the library says which batches go forward row by row, without a map."""
    c = s["case"]
    sh = s["shape"] = L.MoEAdapterShape(T=c["T"], d_in=c["d_in"], d_out=c["d_out"], n=c["n"], rank=c["rank"],
                                        dtype=_code(L, c["dtype"]), dropout=c["p"])
    s["ws"] = torch.zeros(L.moe_adapter_workspace_size(sh), dtype=torch.uint8, device="cuda")
    s["map"] = torch.empty(L.moe_adapter_map_size(sh), dtype=torch.uint8, device="cuda")
    s["rowwise"] = L.moe_adapter_rowwise(sh)


def _own_adapter(s, L):
    c, b = s["case"], s.get("buf")
    if b is None:
        _plan(s, L)
        b = s["buf"] = {"y": torch.empty_like(s["base"]), "u": torch.empty(c["T"], c["rank"], device="cuda")}
    rng = s["rng"] if c["p"] else None
    if s["rowwise"]:
        L.moe_adapter(s["shape"], s["x"], s["A"], s["B"], s["scale"], s["ids"], None, rng, s["base"], b["y"], b["u"], s["ws"])
        return b
    L.moe_adapter_map(s["shape"], s["ids"], s["map"], s["ws"])
    L.moe_adapter(s["shape"], s["x"], s["A"], s["B"], s["scale"], s["ids"], s["map"], rng, s["base"], b["y"], b["u"], s["ws"])
    return b


def _own_adapter_bwd(s, L):
    c, b = s["case"], s.get("buf")
    if b is None:
        _plan(s, L)
        b = s["buf"] = {"dx": torch.empty_like(s["dx_in"]), "dA": torch.empty(s["A"].shape, device="cuda"),
                        "dB": torch.empty(s["B"].shape, device="cuda")}
    L.moe_adapter_map(s["shape"], s["ids"], s["map"], s["ws"])
    L.moe_adapter_bwd(s["shape"], _code(L, c["dx"]), s["dy"], s["x"], s["A"], s["B"], s["scale"], s["map"],
                      s["rng"] if c["p"] else None, s["u"], s["dx_in"], b["dx"], b["dA"], b["dB"], s["ws"])
    return b


def _own_dropout(s, L):
    c, b = s["case"], s.get("buf")
    if b is None:
        b = s["buf"] = {"out": torch.empty_like(s["x"])}
    L.moe_dropout(_code(L, c["dtype"]), c["rows"] * c["d"], s["x"], s["r"], c["p"], s["rng"], b["out"])
    return b


def _own_dropout_bwd(s, L):
    c, b = s["case"], s.get("buf")
    if b is None:
        b = s["buf"] = {"dx": torch.empty(c["rows"], c["d"], dtype=DT[c["dtype"]], device="cuda")}
    L.moe_dropout_bwd(_code(L, c["dy"]), _code(L, c["dtype"]), c["rows"] * c["d"], s["dy"], c["p"], s["rng"], b["dx"])
    return b


def run(state):
    op = state["case"]["op"]
    if own:
        from token_dispatch_expert_moe_gb300 import _lib as L
        return {"adapter": _own_adapter, "adapter_bwd": _own_adapter_bwd, "dropout": _own_dropout,
                "dropout_bwd": _own_dropout_bwd}[op](state, L)
    return {"adapter": _plain_adapter, "adapter_bwd": _plain_adapter_bwd, "dropout": _plain_dropout,
            "dropout_bwd": _plain_dropout_bwd}[op](state)


# --------------------------------------------------------------------------------------------------- work and definition

def work(case):
    c, op = case, case["op"]
    b = SIZE[c["dtype"]]
    if op == "dropout":
        n = c["rows"] * c["d"]
        return {"bytes": n * b * (2 + c["residual"]), "flops": 2 * n}
    if op == "dropout_bwd":
        n = c["rows"] * c["d"]
        return {"bytes": n * (b + SIZE[c["dy"]]), "flops": 2 * n}
    T, d_in, d_out, n, r = c["T"], c["d_in"], c["d_out"], c["n"], c["rank"]
    live = T if T == 1 else int(T * (1 - c["bare"]))
    # adapters that occur: the expected number of different ones among the tokens or requests
    draws = T if c["order"] == "mixed" else min(T, n + n // 4 + 1)
    used = max(1, round(n * (1 - (1 - 1 / n) ** (draws * (1 - c["bare"]))))) if n > 1 else 1
    weights = used * r * (d_in + d_out) * b + 4 * used
    if op == "adapter":
        return {"bytes": live * d_in * b + 2 * T * d_out * b + weights + 4 * T * (r + 1), "flops": 2 * live * r * (d_in + d_out)}
    return {"bytes": live * (d_in + d_out) * b + 2 * T * d_in * SIZE[c["dx"]] + weights + 4 * T * (r + 1)
            + 4 * n * r * (d_in + d_out), "flops": 4 * live * r * (d_in + d_out)}


def _mask(n, rng, p):
    """The mask from the generator's definition, the high words of products put together from 16-bit pieces."""
    def mul(a, b):
        ah, al, bh, bl = a >> 16, a & 0xFFFF, b >> 16, b & 0xFFFF
        low = al * bl
        mid = ah * bl + (low >> 16)
        mid2 = al * bh + (mid & 0xFFFF)
        return ah * bh + (mid >> 16) + (mid2 >> 16), ((mid2 & 0xFFFF) << 16) | (low & 0xFFFF)

    seed, offset = (int(v) % 2 ** 64 for v in rng.tolist())
    out = torch.empty((n + 7) // 8, 8, dtype=torch.bool, device="cuda")
    for lo in range(0, len(out), 1 << 23):
        block = torch.arange(lo, min(len(out), lo + (1 << 23)), device="cuda")
        x = [block % 2 ** 32, block // 2 ** 32, torch.full_like(block, offset % 2 ** 32), torch.full_like(block, offset // 2 ** 32)]
        for i in range(10):
            k = ((seed + i * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + i * 0xBB67AE85) % 2 ** 32)
            (h0, l0), (h1, l1) = mul(x[0], 0xD2511F53), mul(x[2], 0xCD9E8D57)
            x = [h1 ^ x[1] ^ k[0], l1, h0 ^ x[3] ^ k[1], l0]
        for j in range(8):
            out[lo:lo + len(block), j] = (x[j // 2] >> (16 * (j % 2))) % 65536 >= _threshold(p)
    return out.view(-1)[:n]


def exact(case, seed):
    """The definitions in 64 bits; gradients by differentiating the forward formula."""
    s, c = prepare(case, seed), case
    op, p = c["op"], c["p"]

    def drop(x):
        if p == 0.0:
            return x
        factor = 65536.0 / (65536 - _threshold(p))
        return torch.where(_mask(x.numel(), s["rng"], p).view(x.shape), x * factor, 0.0)

    if op == "dropout":
        out = drop(s["x"].double())
        return {"out": out if s["r"] is None else out.add_(s["r"])}
    if op == "dropout_bwd":
        return {"dx": drop(s["dy"].double())}
    ids, n = s["ids"].long(), c["n"]
    if op == "adapter":
        x, y = drop(s["x"].double()), s["base"].double()
        u = torch.zeros(c["T"], c["rank"], dtype=torch.float64, device="cuda")
        for a in range(n):
            t = torch.nonzero(ids == a)[:, 0]
            if len(t):
                u[t] = torch.einsum("tk,jk->tj", x[t], s["A"][a].double())
                y[t] += torch.einsum("tj,cj->tc", u[t], s["scale"][a].double() * s["B"][a].double())
        return {"y": y, "u": u}
    out = {"dx": s["dx_in"].double(), "dA": torch.zeros(s["A"].shape, dtype=torch.float64, device="cuda"),
           "dB": torch.zeros(s["B"].shape, dtype=torch.float64, device="cuda")}
    keep = None if p == 0.0 else drop(torch.ones_like(s["x"], dtype=torch.float64))
    for a in range(n):
        t = torch.nonzero(ids == a)[:, 0]
        if len(t):
            # of <dy, s B A (x * keep)>; u is what the forward kept, so B's gradient takes it as it is
            x, A, B = s["x"][t].double().requires_grad_(), s["A"][a].double().requires_grad_(), s["B"][a].double().requires_grad_()
            dy, scale = s["dy"][t].double(), s["scale"][a].double()
            up = (x if keep is None else x * keep[t]) @ A.T
            gx, gA = torch.autograd.grad(up @ B.detach().T * scale, (x, A), dy)
            gB, = torch.autograd.grad(s["u"][t].double() @ B.T * scale, B, dy)
            out["dx"][t] += gx
            out["dA"][a], out["dB"][a] = gA, gB
    return out
