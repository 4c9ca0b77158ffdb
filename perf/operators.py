"""Workloads of the operators around the MoE layer: the norm in front of it, the router's balance loss, the permutation
of 8-bit rows, and the clipping of the gradients. `own` chooses between the framework's kernels and the operators' plain
form in elementary torch operations."""
import torch
import torch.nn.functional as F

own = False

EPS = 1e-6
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token in front of a Mixtral-8x22B-sized layer
        dict(name="norm one token", op="norm", rows=1, d=6144, dtype="bf16", residual=True, y=True, group=0, quant=False),
        # a ragged prefill batch on the Qwen2-57B-A14B hidden size, rows sent on in 8 bits
        dict(name="norm ragged 8-bit", op="norm", rows=1021, d=3584, dtype="bf16", residual=True, y=True, group=128, quant=True),
        # the training batch of the Llama3-8x70B shape: residual stream, router input and 8-bit rows
        dict(name="norm training 8-bit", op="norm", rows=32768, d=8192, dtype="bf16", residual=True, y=True, group=128, quant=True),
        # the checking case's sizes in fp32
        dict(name="norm bwd tiny f32", op="norm_bwd", rows=512, d=64, dtype="f32", dy="f32", dx="f32", dh=True),
        # the backward of the training batch: fp32 gradient of the layer, bf16 gradient of the residual stream
        dict(name="norm bwd training", op="norm_bwd", rows=32768, d=8192, dtype="bf16", dy="f32", dx="f32", dh=True),
        # the checking case's router
        dict(name="balance tiny", op="balance", T=512, E=4, K=2, S=0, mask=False),
        # G8T8-sized batch, per-sequence loss, sequences padded to 4096
        dict(name="balance padded sequences", op="balance", T=16384, E=64, K=8, S=4096, mask=True),
        # a whole accumulation of 32 sequences
        dict(name="balance long batch", op="balance", T=262144, E=64, K=8, S=8192, mask=False),
        # odd batch and odd hidden size, groups that end inside the row, fp32 layer
        dict(name="permute e4m3 odd f32", op="permute", T=777, d=1000, E=60, K=6, dtype="f32", group=64, kept=1.0),
        # G8T8 training batch with token dropping
        dict(name="permute e4m3 training", op="permute", T=16384, d=6144, E=64, K=8, dtype="bf16", group=128, kept=0.9),
        # gradients of the checking case
        dict(name="clip tiny", op="clip", layers=1, d=64, E=4, F=128, Fs=0, dtype="f32", clips=True),
        # gradients of one Qwen2-57B-A14B layer, its shared expert and its norm
        dict(name="clip one large layer", op="clip", layers=1, d=3584, E=64, F=2560, Fs=20480, dtype="f32", clips=True),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "balance", "permute", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_bwd"):
        rows = _log(rng, 1, 32768)
        d = 8 * _log(rng, 8, 1024)
        while rows * d * (2 if dtype == "f32" else 1) > 32768 * 8192:
            rows //= 2
        if op == "norm":
            quant = rng.random() < 0.6
            return dict(op=op, rows=rows, d=d, dtype=dtype, residual=rng.random() < 0.7, y=not quant or rng.random() < 0.7,
                        group=rng.choice([0, 32, 64, 128]) if quant else 0, quant=quant)
        return dict(op=op, rows=rows, d=d, dtype=dtype, dy="f32" if dtype == "f32" else rng.choice(["f32", "bf16"]),
                    dx="f32" if dtype == "f32" else rng.choice(["f32", "bf16"]), dh=rng.random() < 0.7)
    if op == "balance":
        T, E = _log(rng, 1, 262144), rng.randint(1, 64)
        return dict(op=op, T=T, E=E, K=rng.randint(1, min(E, 8)), S=rng.choice([0, _log(rng, 64, 8192), _log(rng, 64, 8192)]),
                    mask=rng.random() < 0.5)
    if op == "permute":
        T, d, E = _log(rng, 1, 16384), 8 * _log(rng, 8, 768), rng.randint(1, 64)
        while T * d * (2 if dtype == "f32" else 1) > 16384 * 6144:
            T //= 2
        return dict(op=op, T=T, d=d, E=E, K=rng.randint(1, min(E, 8)), dtype=dtype, group=rng.choice([0, 32, 64, 128]),
                    kept=rng.choice([1.0, 0.9, 0.5]))
    return dict(op=op, layers=rng.randint(1, 6), d=8 * _log(rng, 8, 256), E=rng.randint(1, 24), F=_log(rng, 16, 1024),
                Fs=rng.choice([0, _log(rng, 16, 4096)]), dtype=dtype, clips=rng.random() < 0.7)


# --------------------------------------------------------------------------------------------------------------- inputs

def _groups(d, group):
    g = group or d
    return g, -(-d // g)


def _grad_shapes(c):
    d, E, Fe, Fs = c["d"], c["E"], c["F"], c["Fs"]
    one = [(E, d), (E,), (E, 2 * Fe, d), (E, d, Fe), (d,)]
    if Fs:
        one += [(2 * Fs, d), (d, Fs), (d,)]
    return one * c["layers"]


def prepare(case, seed):
    c, g = dict(case), torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s, dt="f32", std=1.0: torch.randn(*s, device="cuda", generator=g).mul_(std).to(DT[dt])  # noqa: E731
    rand = lambda *s: torch.rand(*s, device="cuda", generator=g)  # noqa: E731
    s = dict(case=c)
    op = c["op"]
    if op in ("norm", "norm_bwd"):
        rows, d, dt = c["rows"], c["d"], c["dtype"]
        # a residual stream whose channels differ in scale, and a gain around one
        h = (torch.randn(rows, d, device="cuda", generator=g) * (0.3 + 2.0 * rand(d))).to(DT[dt])
        s["gamma"] = (1.0 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(DT[dt])
        if op == "norm":
            s["x"] = h
            s["r"] = randn(rows, d, dt=dt) if c["residual"] else None
        else:
            s["h"] = h
            s["rstd"] = torch.rsqrt(h.float().square().mean(1) + EPS)
            s["dy"] = randn(rows, d, dt=c["dy"], std=0.1)
            s["dh"] = randn(rows, d, dt=dt, std=0.1) if c["dh"] else None
    elif op == "balance":
        T, E, K = c["T"], c["E"], c["K"]
        # logits with per-expert skew; the Top-K of their softmax
        s["logits"] = torch.randn(T, E, device="cuda", generator=g) + 0.7 * torch.randn(E, device="cuda", generator=g)
        s["idx"] = s["logits"].topk(K, dim=1).indices.int()
        s["mask"] = None
        if c["mask"]:   # every sequence ends in padding of its own length
            S = c["S"] or T
            length = (rand(-(-T // S)) * S).long() + 1
            t = torch.arange(T, device="cuda")
            s["mask"] = ((t % S) < length[t // S]).to(torch.uint8)
        s["alpha"] = 0.01
        s["dloss"] = 0.5 + rand(1)
    elif op == "permute":
        T, d, E, K = c["T"], c["d"], c["E"], c["K"]
        gs, ng = _groups(d, c["group"])
        y = torch.randn(T, d, device="cuda", generator=g) * (0.3 + 2.0 * rand(d))
        yg = F.pad(y, (0, ng * gs - d)).view(T, ng, gs)
        s["scale"] = (yg.abs().amax(2) / 448.0).clamp_min(1e-12)
        s["q"] = (yg / s["scale"][:, :, None]).clamp(-448, 448).view(T, ng * gs)[:, :d].contiguous().to(torch.float8_e4m3fn)
        s["idx"] = (rand(T, E) + 0.5 * rand(E)).topk(K, dim=1).indices.int()
        s["keep"] = (rand(T, K) < c["kept"]).to(torch.uint8)
    else:
        s["grads"] = []
        for shape in _grad_shapes(c):
            x = torch.randn(*shape, device="cuda", generator=g, dtype=DT[c["dtype"]])
            x.mul_(10.0 ** (-3 + 2 * float(torch.rand(1, generator=g, device="cuda"))))
            if len(shape) == 3:   # some experts saw no token
                x[1::7] = 0
            s["grads"].append(x)
        s["max_norm"] = 1e-3 if c["clips"] else 1e9
    return s


# ----------------------------------------------------------------------------------------------------------- plain forms

def _plain_norm(s):
    c = s["case"]
    dt, d = DT[c["dtype"]], c["d"]
    out = {}
    h = s["x"]
    if s["r"] is not None:
        h = out["h"] = (s["x"].float() + s["r"].float()).to(dt)
    hf = h.float()
    rstd = torch.rsqrt(hf.square().mean(1) + EPS)
    y = hf * rstd[:, None] * s["gamma"].float()
    out["rstd"] = rstd
    if c["y"]:
        out["y"] = y.to(dt)
    if c["quant"]:
        g, n = _groups(d, c["group"])
        yg = F.pad(y, (0, n * g - d)).view(-1, n, g)
        amax = yg.abs().amax(2)
        scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        q = (yg / scale[:, :, None]).clamp(-448.0, 448.0).view(-1, n * g)[:, :d]
        out["scale"], out["q"] = scale, q.to(torch.float8_e4m3fn)
    return out


def _plain_norm_bwd(s):
    c = s["case"]
    dy, xhat = s["dy"].float(), s["h"].float() * s["rstd"][:, None]
    g = dy * s["gamma"].float()
    dx = s["rstd"][:, None] * (g - xhat * (g * xhat).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(DT[c["dx"]]), "dgamma": (dy * xhat).sum(0)}


def _plain_balance(s):
    c = s["case"]
    T, E, K = c["T"], c["E"], c["K"]
    S = c["S"] or T
    n_sub = -(-T // S)
    seq = torch.arange(T, device="cuda") // S
    live = torch.ones(T, device="cuda") if s["mask"] is None else (s["mask"] != 0).float()
    p = torch.softmax(s["logits"], 1)
    pl = F.pad(p * live[:, None], (0, 0, 0, n_sub * S - T)).view(n_sub, S, E)
    n_j = F.pad(live, (0, n_sub * S - T)).view(n_sub, S).sum(1)
    one = torch.zeros(T, E, device="cuda").scatter_add_(1, s["idx"].long(), live[:, None].expand(T, K).contiguous())
    counts = F.pad(one, (0, 0, 0, n_sub * S - T)).view(n_sub, S, E).sum(1)
    some = n_j.clamp_min(1)
    n = n_j.sum()
    prob = pl.sum(1) / some[:, None]
    loss = s["alpha"] * E / K * (counts * prob).sum() / n.clamp_min(1)
    a = s["alpha"] * (E * counts - K * n_j[:, None]) / (K * some[:, None])   # sum_e p_e = 1: a constant is free
    at = a[seq]
    dl = (s["dloss"] / n.clamp_min(1)) * live[:, None] * p * (at - (p * at).sum(1, keepdim=True))
    return {"loss": loss.view(1), "counts": counts.int(), "prob": prob, "dlogits": dl}


def _plain_permute(s):
    c = s["case"]
    T, d, E, K = c["T"], c["d"], c["E"], c["K"]
    g, n = _groups(d, c["group"])
    key = torch.where(s["keep"] != 0, s["idx"], E).view(-1)
    order = key.sort(stable=True).indices            # expert-major, token-ascending, dropped slots last
    counts = (key[:, None] == torch.arange(E, device="cuda")).sum(0)
    offsets = F.pad(counts.cumsum(0), (1, 0))
    place = torch.arange(T * K, device="cuda")
    there = place < offsets[E]
    row_of = torch.empty(T * K, dtype=torch.int64, device="cuda").scatter_(0, order, torch.where(there, place, -1))
    x = F.pad(s["q"].float(), (0, n * g - d)).view(T, n, g) * s["scale"][:, :, None]
    x = x.view(T, n * g)[:, :d].to(DT[c["dtype"]])
    return {"Xp": torch.where(there[:, None], x[order // K], 0), "row_of": row_of.int().view(T, K),
            "src_of": torch.where(there, order, 0).int(), "counts": counts.int(), "offsets": offsets.int()}


def _plain_clip(s):
    norm = torch.stack([x.float().square().sum() for x in s["grads"]]).sum().sqrt().view(1)
    coef = torch.where((norm > s["max_norm"]) & torch.isfinite(norm), s["max_norm"] / norm, torch.ones_like(norm))
    return {"norm": norm, "coef": coef, "grads": [(x.float() * coef).to(x.dtype) for x in s["grads"]]}


# ---------------------------------------------------------------------------------------------------- the framework's

def _code(L, name):
    return L.MOE_BF16 if name == "bf16" else L.MOE_F32


def _own_norm(s, L):
    c, b = s["case"], s.get("buf")
    rows, d, dt = c["rows"], c["d"], DT[c["dtype"]]
    if b is None:
        new = lambda *shape, dtype=dt: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
        b = s["buf"] = {"rstd": new(rows, dtype=torch.float32)}
        if s["r"] is not None:
            b["h"] = new(rows, d)
        if c["y"]:
            b["y"] = new(rows, d)
        if c["quant"]:
            b["q"] = new(rows, d, dtype=torch.float8_e4m3fn)
            b["scale"] = new(rows, _groups(d, c["group"])[1], dtype=torch.float32)
    L.moe_rmsnorm(_code(L, c["dtype"]), rows, d, s["x"], s["r"], s["gamma"], EPS, b.get("h"), b.get("y"), b.get("q"),
                  b.get("scale"), c["group"], b["rstd"])
    return b


def _own_norm_bwd(s, L):
    c, b = s["case"], s.get("buf")
    rows, d = c["rows"], c["d"]
    if b is None:
        b = s["buf"] = {"dx": torch.empty(rows, d, dtype=DT[c["dx"]], device="cuda"),
                        "dgamma": torch.empty(d, dtype=torch.float32, device="cuda")}
        s["ws"] = torch.empty(L.moe_rmsnorm_bwd_workspace_size(rows, d), dtype=torch.uint8, device="cuda")
    L.moe_rmsnorm_bwd(_code(L, c["dtype"]), _code(L, c["dy"]), _code(L, c["dx"]), rows, d, s["dy"], s["h"], s["gamma"],
                      s["rstd"], s["dh"], b["dx"], b["dgamma"], s["ws"])
    return b


def _own_balance(s, L):
    c, b = s["case"], s.get("buf")
    T, E = c["T"], c["E"]
    if b is None:
        n_sub = -(-T // (c["S"] or T))
        f = lambda *shape: torch.empty(*shape, device="cuda")  # noqa: E731
        b = s["buf"] = {"loss": f(1), "counts": torch.empty(n_sub, E, dtype=torch.int32, device="cuda"), "prob": f(n_sub, E),
                        "dlogits": f(T, E)}
        s["coef"] = f(n_sub * E + 1)
        s["shape"] = L.MoEShape(T=T, d=64, E=E, K=c["K"], F=64, dtype=L.MOE_BF16, subseq_len=c["S"])
        s["ws"] = torch.zeros(L.moe_workspace_size(s["shape"]), dtype=torch.uint8, device="cuda")
    L.moe_balance_loss(s["shape"], s["logits"], s["idx"], s["mask"], s["alpha"], b["loss"], b["counts"], b["prob"], s["coef"],
                       s["ws"])
    L.moe_balance_loss_bwd(s["shape"], s["logits"], s["mask"], s["coef"], s["dloss"], b["dlogits"])
    return b


def _own_permute(s, L):
    c, b = s["case"], s.get("buf")
    T, d, E, K = c["T"], c["d"], c["E"], c["K"]
    if b is None:
        i = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device="cuda")  # noqa: E731
        b = s["buf"] = {"Xp": torch.zeros(T * K, d, dtype=DT[c["dtype"]], device="cuda"), "row_of": i(T, K),
                        "src_of": i(T * K), "counts": i(E), "offsets": i(E + 1)}
        s["shape"] = L.MoEShape(T=T, d=d, E=E, K=K, F=64, dtype=_code(L, c["dtype"]))
        s["ws"] = torch.zeros(L.moe_workspace_size(s["shape"]), dtype=torch.uint8, device="cuda")
    L.moe_permute_e4m3(s["shape"], s["q"], s["scale"], c["group"], s["idx"], s["keep"], b["Xp"], b["row_of"], b["src_of"],
                       b["counts"], b["offsets"], s["ws"])
    return b


def _own_clip(s, L):
    b = s.get("buf")
    if b is None:
        b = s["buf"] = {"norm": torch.empty(1, device="cuda"), "coef": torch.empty(1, device="cuda"),
                        "grads": [torch.empty_like(x) for x in s["grads"]]}
        s["in"], s["out"] = L.TensorList(s["grads"]), L.TensorList(b["grads"])
        s["ws"] = torch.empty(L.MOE_GRAD_NORM_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    L.moe_grad_norm(s["in"], b["norm"], s["ws"])
    L.moe_grad_clip(s["in"], s["out"], b["norm"], s["max_norm"], b["coef"])
    return b


def run(state):
    op = state["case"]["op"]
    if own:
        from token_dispatch_expert_moe_gb300 import _lib as L
        return {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "balance": _own_balance, "permute": _own_permute,
                "clip": _own_clip}[op](state, L)
    return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "balance": _plain_balance, "permute": _plain_permute,
            "clip": _plain_clip}[op](state)


# --------------------------------------------------------------------------------------------------- work and definition

def work(case):
    c, size = case, {"f32": 4, "bf16": 2}
    op = c["op"]
    if op in ("norm", "norm_bwd"):
        n, b = c["rows"] * c["d"], size[c["dtype"]]
        if op == "norm":
            ng = _groups(c["d"], c["group"])[1]
            each = b * (1 + 2 * c["residual"] + c["y"]) + c["quant"]
            return {"bytes": n * each + c["d"] * b + 4 * c["rows"] * (1 + c["quant"] * ng), "flops": n * (4 + 3 * c["quant"])}
        each = size[c["dy"]] + b + size[c["dx"]] + b * c["dh"]
        return {"bytes": n * each + c["d"] * (b + 4) + 4 * c["rows"], "flops": n * 10}
    if op == "balance":
        T, E, K = c["T"], c["E"], c["K"]
        n_sub = -(-T // (c["S"] or T))
        return {"bytes": T * (8 * E + 4 * K + c["mask"]) + 8 * n_sub * E, "flops": 12 * T * E}
    if op == "permute":
        T, d, E, K = c["T"], c["d"], c["E"], c["K"]
        ng = _groups(d, c["group"])[1]
        kept = int(T * K * c["kept"])
        return {"bytes": T * (d + 4 * ng) + kept * d * size[c["dtype"]] + T * K * 9 + kept * 4 + 8 * E, "flops": T * d}
    n = sum(torch.Size(x).numel() for x in _grad_shapes(c))
    return {"bytes": 2 * n * size[c["dtype"]], "flops": 3 * n}


def exact(case, seed):
    """The definitions in 64 bits; gradients by differentiating the forward formula."""
    s, c = prepare(case, seed), case
    op = c["op"]
    if op == "norm":
        h = s["x"].double()
        if s["r"] is not None:
            h = (h + s["r"].double()).to(DT[c["dtype"]]).double()   # the residual stream is held in the layer's type
        rstd = 1.0 / torch.sqrt(torch.einsum("ij,ij->i", h, h) / c["d"] + EPS)
        y = torch.einsum("ij,i,j->ij", h, rstd, s["gamma"].double())
        out = {"rstd": rstd}
        if s["r"] is not None:
            out["h"] = h
        if c["y"]:
            out["y"] = y
        if c["quant"]:
            g = c["group"] or c["d"]
            parts = y.split(g, dim=1)
            scale = [p.abs().max(dim=1, keepdim=True).values / 448.0 for p in parts]
            out["q"] = torch.cat([p / a for p, a in zip(parts, scale)], 1)
            out["scale"] = torch.cat(scale, 1)
        return out
    if op == "norm_bwd":
        h, gamma = s["h"].double().requires_grad_(), s["gamma"].double().requires_grad_()
        y = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * gamma
        dx, dgamma = torch.autograd.grad(y, (h, gamma), s["dy"].double())
        return {"dx": dx if s["dh"] is None else dx.add_(s["dh"]), "dgamma": dgamma}
    if op == "balance":
        T, E, K = c["T"], c["E"], c["K"]
        S = c["S"] or T
        logits = s["logits"].double().requires_grad_()
        live = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"] != 0
        loss, probs = 0.0, []
        for lo in range(0, T, S):
            at = live[lo:lo + S]
            e = logits[lo:lo + S][at].exp()
            P = (e / e.sum(1, keepdim=True)).mean(0) if bool(at.any()) else torch.zeros(E, dtype=torch.float64, device="cuda")
            n_j = int(at.sum())
            # sum_e P_e = 1, so the load's mean is taken out before the product and added after it
            over = (torch.bincount(s["idx"][lo:lo + S][at].view(-1).long(), minlength=E).double() * E - K * n_j) / K
            loss = loss + s["alpha"] * ((over * P).sum() + n_j) / live.sum()
            probs.append(P.detach())
        dl, = torch.autograd.grad(loss, logits, s["dloss"].double()[0])
        return {"loss": loss.detach().view(1), "counts": None, "prob": torch.stack(probs), "dlogits": dl}
    if op == "permute":
        T, d, K = c["T"], c["d"], c["K"]
        x = s["q"].double() * s["scale"].double().repeat_interleave(c["group"] or d, dim=1)[:, :d]
        at = torch.cat([((s["idx"] == e) & (s["keep"] != 0)).any(1).nonzero()[:, 0] for e in range(c["E"])])
        out = torch.zeros(T * K, d, dtype=torch.float64, device="cuda")
        out[:len(at)] = x[at]
        return {"Xp": out, "row_of": None, "src_of": None, "counts": None, "offsets": None}
    norm = torch.sqrt(sum(torch.linalg.vector_norm(x.double()) ** 2 for x in s["grads"]))
    coef = s["max_norm"] / norm if s["max_norm"] < float(norm) < float("inf") else torch.ones_like(norm)
    return {"norm": norm.view(1), "coef": coef.view(1), "grads": [x.double() * coef for x in s["grads"]]}
