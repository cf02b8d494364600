"""Further operators of a feed-forward block, as they are measured: cases, inputs, plain forms and definitions in 64 bits.

* ``add_layer_norm``: layer norm (mean and variance) with the residual's addition, and its backward pass with the
  reductions of the weight's and the bias's gradient.
* ``lora``: low-rank adapters of many requests at once, added to a shared projection's output:
  D = act(R + s[a] (X A[a]^T) B[a]^T), a = ids[row].
* ``moe_ffn_gated``: a whole mixture-of-experts layer for a few tokens: the router's product, the choice of the top k,
  the chosen experts' gated feed-forward, and their weighted sum onto the residual stream.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5


# ---------------------------------------------------------------------------------------------- cases

def listed():
    lora = {"op": "lora", "act": "none", "residual": True}
    moe = {"op": "moe", "residual": True, "renormalize": True}
    return [
        # The norm in front of a block for one new token: pure latency.
        {"op": "ln_fwd", "name": "ln_fwd_1x4096", "m": 1, "d": 4096, "residual": True, "bias": True},
        # Training, forward: the residual's addition and the norm in one pass.
        {"op": "ln_fwd", "name": "ln_fwd_8192x4096", "m": 8192, "d": 4096, "residual": True, "bias": True},
        # Training, backward: the gradients of the residual stream, of the weight and of the bias.
        {"op": "ln_bwd", "name": "ln_bwd_8192x4096", "m": 8192, "d": 4096, "dh": True, "bias": True},
        # The same with rows of an odd width (none but every eighth starts on 16 bytes).
        {"op": "ln_bwd", "name": "ln_bwd_3001x4099", "m": 3001, "d": 4099, "dh": True, "bias": True},
        # One new token of one request beside a projection of a 4096-wide model: the smallest adapter, pure latency.
        dict(lora, name="lora_1x4096x4096_r16", m=1, n=4096, k=4096, r=16, adapters=32, requests=1),
        # 48 requests decoded together, nearly each with an adapter of its own, on a wide projection.
        dict(lora, name="lora_48x14336x4096_r64", m=48, n=14336, k=4096, r=64, adapters=40, requests=48),
        # Prompts of a dozen requests in one batch.
        dict(lora, name="lora_8192x4096x4096_r16", m=8192, n=4096, k=4096, r=16, adapters=16, requests=12),
        # Odd rows and columns, with the projection's activation after the adapters.
        dict(lora, name="lora_1000x4099x14336_r32", m=1000, n=4099, k=14336, r=32, adapters=8, requests=30,
             act="gelu_tanh"),
        # One new token through two of eight wide experts: the weights' bytes.
        dict(moe, name="moe_1x4096x14336_2of8", m=1, d=4096, i=14336, experts=8, k=2),
        # Five drafted tokens through small experts: launches and joins count.
        dict(moe, name="moe_5x2048x1408_6of64", m=5, d=2048, i=1408, experts=64, k=6, renormalize=False),
        # Sixteen sequences decoded together: every wide expert is read.
        dict(moe, name="moe_16x4096x14336_2of8", m=16, d=4096, i=14336, experts=8, k=2),
        # 64 sequences on many experts, each with a few of the tokens.
        dict(moe, name="moe_64x4096x2048_8of64", m=64, d=4096, i=2048, experts=64, k=8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "lora", "lora", "moe", "moe"])
    if op in ("ln_fwd", "ln_bwd"):
        d = _log(rng, 64, 16384)
        d = d // 8 * 8 if rng.random() < 0.6 else d
        case = {"op": op, "m": min(_log(rng, 1, 16384), 8192 * 4096 // d), "d": d, "bias": rng.random() < 0.7}
        return case | {"residual" if op == "ln_fwd" else "dh": rng.random() < 0.8}
    if op == "lora":
        k = 8 * _log(rng, 8, 2048)
        n = _log(rng, 64, 16384)
        n = n // 8 * 8 if rng.random() < 0.6 else n
        m = min(_log(rng, 1, 8192), 8192 * 8192 // (n + k))
        r = rng.choice([8, 16, 16, 32, 64, 128])
        adapters = min(_log(rng, 1, 64), max(1, 1024 // r))
        return {"op": op, "m": m, "n": n, "k": k, "r": r, "adapters": adapters, "requests": _log(rng, 1, min(m, 256)),
                "act": rng.choice(["none", "none", "gelu_tanh", "silu", "relu"]), "residual": rng.random() < 0.8}
    experts = _log(rng, 2, 128)
    d = 8 * _log(rng, 256 // 8, 8192 // 8)
    most = min(14336, 64 * 2048 * 4096 // (experts * d))
    return {"op": op, "m": _log(rng, 1, 64), "d": d, "i": 8 * _log(rng, 64 // 8, max(64, most) // 8),
            "experts": experts, "k": min(experts, rng.choice([1, 2, 2, 4, 6, 8])), "residual": rng.random() < 0.7,
            "renormalize": rng.random() < 0.5}


# ---------------------------------------------------------------------------------------------- inputs

def _normal(gen, *shape, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16) * std


def _rows_of_requests(gen, m, adapters, requests):
    """ids [m] int32: rows of one request lie together and share an adapter; one request in ten has none (-1)."""
    cuts = torch.randint(0, m, (requests,), generator=gen, device="cuda") if requests < m else torch.arange(m, device="cuda")
    starts = torch.zeros(m, dtype=torch.int64, device="cuda")
    starts[cuts] = 1
    starts[0] = 0
    choice = torch.randint(0, adapters, (m,), generator=gen, device="cuda")
    if m > 1:
        choice = torch.where(torch.rand(m, generator=gen, device="cuda") < 0.1, -1, choice)
    return choice[torch.cumsum(starts, dim=0)].to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 23)
    s = {"case": dict(case)}
    op = case["op"]
    if op == "lora":
        m, n, k, r, count = case["m"], case["n"], case["k"], case["r"], case["adapters"]
        s["x"] = _normal(gen, m, k)
        s["a"] = _normal(gen, count, r, k, std=k ** -0.5)
        s["b"] = _normal(gen, count, n, r, std=0.3 * r ** -0.5)
        s["scale"] = 0.5 + 1.5 * torch.rand(count, generator=gen, device="cuda")
        s["r"] = _normal(gen, m, n) if case["residual"] else None
        s["ids"] = _rows_of_requests(gen, m, count, case["requests"])
        return s
    if op == "moe":
        m, d, i, e = case["m"], case["d"], case["i"], case["experts"]
        s["x"] = _normal(gen, m, d)
        s["router"] = _normal(gen, e, d, std=1.5 * d ** -0.5)
        s["w1"], s["w3"] = (_normal(gen, e, i, d, std=d ** -0.5) for _ in range(2))
        s["w2"] = _normal(gen, e, d, i, std=i ** -0.5)
        s["r"] = _normal(gen, m, d) if case["residual"] else None
        return s
    m, d = case["m"], case["d"]
    s["weight"] = (torch.rand((d,), generator=gen, device="cuda") + 0.5).to(torch.bfloat16)
    s["bias"] = _normal(gen, d, std=0.1) if case["bias"] else None
    # a residual stream: some channels much larger than the others, and a mean that is not zero
    stream = 1.0 + 6.0 * (torch.rand((d,), generator=gen, device="cuda") < 0.01)
    if op == "ln_bwd":
        s["dy"] = _normal(gen, m, d, std=0.05)
        s["dh"] = _normal(gen, m, d, std=0.05) if case["dh"] else None
        s["h"] = (torch.randn((m, d), generator=gen, device="cuda") * stream + 0.3).to(torch.bfloat16)
        h = s["h"].float()
        s["mean"] = h.mean(dim=1)
        s["rstd"] = torch.rsqrt((h - s["mean"][:, None]).square().mean(dim=1) + EPS)
        return s
    s["x"] = _normal(gen, m, d)
    s["r"] = (torch.randn((m, d), generator=gen, device="cuda") * stream + 0.3).to(torch.bfloat16) if case["residual"] else None
    return s


# ---------------------------------------------------------------------------------------------- one pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import dense_bf16_gemm_persistent_gb300 as gb
    c = s["case"]
    op = c["op"]
    if op == "lora":
        return gb.lora(s["x"], s["a"], s["b"], s["ids"], s["scale"], R=s["r"], act=c["act"])
    if op == "moe":
        d, ids, weights = gb.moe_ffn_gated(s["x"], s["router"], s["w1"], s["w3"], s["w2"], c["k"], R=s["r"],
                                           renormalize=c["renormalize"])
        return {"d": d, "ids": ids, "weights": weights}
    if op == "ln_fwd":
        y, h, mean, rstd = gb.add_layer_norm(s["x"], s["weight"], s["bias"], s["r"], eps=EPS)
        return {"y": y, "h": h, "mean": mean, "rstd": rstd}
    dx, dr, dw, db = gb.add_layer_norm_backward(s["dy"], s["h"], s["weight"], s["mean"], s["rstd"], dH=s["dh"])
    return {"dr": dr, "dweight": dw, "dbias": db}


# ---- plain forms: elementary torch operations in 32 bits, rounded once at the end

def _act(v, act):
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    return v.clamp_min(0.0) if act == "relu" else v


def _plain_lora(s):
    c = s["case"]
    x, a, b = s["x"].float(), s["a"].float(), s["b"].float()
    count, r, k = a.shape
    ids = s["ids"].long()
    live = (ids >= 0) & (ids < count)
    ids = torch.where(live, ids, 0)
    scale = torch.where(live, s["scale"][ids], 0.0)
    if c["m"] < count:  # each row with its own adapter's matrices
        low = torch.bmm(a[ids], x[:, :, None])
        v = torch.bmm(b[ids], low)[:, :, 0] * scale[:, None]
    else:               # all rows with all adapters, and all products but the row's own left out
        low = (x @ a.reshape(count * r, k).T).reshape(c["m"], count, r)
        keep = torch.arange(count, device="cuda")[None, :] == ids[:, None]
        low = torch.where(keep[:, :, None], low * scale[:, None, None], 0.0)
        v = low.reshape(c["m"], count * r) @ b.permute(0, 2, 1).reshape(count * r, c["n"])
    if s["r"] is not None:
        v = v + s["r"].float()
    return _act(v, c["act"]).to(torch.bfloat16)


def _plain_moe(s):
    c = s["case"]
    # (the choice is between values that may be nearly equal: 64 bits)
    logits = s["x"].double() @ s["router"].double().T
    order = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    p = torch.exp(logits - logits.amax(dim=1, keepdim=True))
    p = p / p.sum(dim=1, keepdim=True)
    weights = torch.gather(p, 1, order)
    if c["renormalize"]:
        weights = weights / weights.sum(dim=1, keepdim=True)
    weights = weights.float()
    x = s["x"].float()
    if c["m"] * c["k"] < c["experts"]:  # the chosen experts' matrices, a pair of a token and an expert each
        at = order.reshape(-1)
        xp = x.repeat_interleave(c["k"], dim=0)[:, :, None]
        act = _act(torch.bmm(s["w1"][at].float(), xp), "silu") * torch.bmm(s["w3"][at].float(), xp)
        each = torch.bmm(s["w2"][at].float(), act)[:, :, 0].reshape(c["m"], c["k"], c["d"])
        v = (each * weights[:, :, None]).sum(dim=1)
    else:                               # all experts, weighted by 0 where they are not chosen
        share = torch.zeros((c["m"], c["experts"]), device="cuda").scatter_(1, order, weights)
        act = _act(torch.matmul(x, s["w1"].float().transpose(1, 2)), "silu") * torch.matmul(x, s["w3"].float().transpose(1, 2))
        act = act * share.T[:, :, None]
        v = torch.matmul(act, s["w2"].float().transpose(1, 2)).sum(dim=0)
    if s["r"] is not None:
        v = v + s["r"].float()
    return {"d": v.to(torch.bfloat16), "ids": order.to(torch.int32), "weights": weights}


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "lora":
        return _plain_lora(s)
    if op == "moe":
        return _plain_moe(s)
    w = s["weight"].float()
    if op == "ln_bwd":
        rstd, dy = s["rstd"][:, None], s["dy"].float()
        xhat = (s["h"].float() - s["mean"][:, None]) * rstd
        g = dy * w
        dr = rstd * (g - g.mean(dim=1, keepdim=True) - xhat * (g * xhat).mean(dim=1, keepdim=True))
        if s["dh"] is not None:
            dr = dr + s["dh"].float()
        return {"dr": dr.to(torch.bfloat16), "dweight": (dy * xhat).sum(dim=0), "dbias": dy.sum(dim=0)}
    h = s["x"].float()
    if s["r"] is not None:
        h = h + s["r"].float()
    mean = h.mean(dim=1)
    off = h - mean[:, None]
    rstd = torch.rsqrt(off.square().mean(dim=1) + EPS)
    y = off * rstd[:, None] * w
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return {"y": y.to(torch.bfloat16), "h": h.to(torch.bfloat16), "mean": mean, "rstd": rstd}


# ---------------------------------------------------------------------------------------------- work

def _distinct(count, share, draws):
    """How many of `count` things are expected to be met when each of `draws` meets a share of them."""
    return count * (1.0 - (1.0 - share) ** draws)


def work(case):
    op = case["op"]
    if op == "lora":
        m, n, k, r = case["m"], case["n"], case["k"], case["r"]
        live = 1.0 if m == 1 else 0.9
        met = _distinct(case["adapters"], live / case["adapters"], min(m, case["requests"]))
        # X and R read, D written, the met adapters' two matrices
        b = 2 * m * (k + n * (1 + case["residual"])) + 2 * met * r * (k + n) + 4 * m
        return {"bytes": b, "flops": 2 * live * m * r * (k + n)}
    if op == "moe":
        m, d, i, e, k = case["m"], case["d"], case["i"], case["experts"], case["k"]
        met = _distinct(e, k / e, m)
        # the met experts' three matrices and the router, X and R read, D, the choice and its weights written
        b = 2 * met * 3 * i * d + 2 * e * d + 2 * m * d * (2 + case["residual"]) + 8 * m * k
        return {"bytes": b, "flops": 6 * m * k * i * d + 2 * m * e * d}
    m, d = case["m"], case["d"]
    if op == "ln_bwd":
        # dY, H and dH read, dR written; the mean and the deviation, the weight, its gradient and the bias's
        return {"bytes": 2 * m * d * (3 + case["dh"]) + 8 * m + 10 * d, "flops": 14 * m * d}
    # X and R read, Y and H (where it is not X itself) written
    return {"bytes": 2 * m * d * (2 + 2 * case["residual"]) + 8 * m + (2 + 2 * case["bias"]) * d, "flops": 9 * m * d}


# ---------------------------------------------------------------------------------------------- 64 bits

def _exact_act(v, act):
    if act == "gelu_tanh":
        return v * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
    if act == "silu":
        return v * torch.sigmoid(v)
    return torch.maximum(v, torch.zeros_like(v)) if act == "relu" else v


def _exact_moe(s, c):
    logits = torch.einsum("td,ed->te", s["x"].double(), s["router"].double()).cpu().numpy()
    order = np.argsort(-logits, axis=1, kind="stable")[:, :c["k"]]
    top = np.exp(logits - logits.max(axis=1, keepdims=True))
    weights = np.take_along_axis(top, order, axis=1)
    weights = weights / (weights if c["renormalize"] else top).sum(axis=1, keepdims=True)
    v = s["r"].double() if s["r"] is not None else torch.zeros((c["m"], c["d"]), dtype=torch.float64, device="cuda")
    for e in np.unique(order):
        rows, places = np.nonzero(order == e)
        t = torch.from_numpy(rows).cuda()
        x = s["x"][t].double()
        up, gate = x @ s["w3"][e].double().T, x @ s["w1"][e].double().T
        y = (gate * torch.sigmoid(gate) * up) @ s["w2"][e].double().T
        v = v.index_add(0, t, y * torch.from_numpy(weights[rows, places]).cuda()[:, None])
    return {"d": v, "ids": None, "weights": torch.from_numpy(weights).cuda()}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f = lambda t: t.double()  # noqa: E731
    if op == "moe":
        return _exact_moe(s, case)
    if op == "lora":
        v = f(s["r"]) if s["r"] is not None else torch.zeros((case["m"], case["n"]), dtype=torch.float64, device="cuda")
        for a in s["ids"].unique().tolist():
            if 0 <= a < case["adapters"]:
                rows = torch.nonzero(s["ids"] == a)[:, 0]
                low = torch.einsum("mk,rk->mr", f(s["x"][rows]), f(s["a"][a]))
                v[rows] += torch.einsum("mr,nr->mn", low, f(s["b"][a])) * float(s["scale"][a])
        return _exact_act(v, case["act"])
    w = f(s["weight"])
    if op == "ln_bwd":
        r, dy = f(s["rstd"])[:, None], f(s["dy"])
        off = f(s["h"]) - f(s["mean"])[:, None]
        g = dy * w
        n = case["d"]
        dr = r * g - r * g.sum(dim=1, keepdim=True) / n - r ** 3 * off * (g * off).sum(dim=1, keepdim=True) / n
        if s["dh"] is not None:
            dr += f(s["dh"])
        return {"dr": dr, "dweight": torch.einsum("md,md,mo->d", dy, off, r), "dbias": torch.einsum("md->d", dy)}
    h = f(s["x"])
    if s["r"] is not None:
        h = h + f(s["r"])
    mean = torch.sum(h, dim=1) / case["d"]
    var = torch.sum(h * h, dim=1) / case["d"] - mean * mean
    rstd = 1.0 / torch.sqrt(var + EPS)
    y = (h - mean[:, None]) * rstd[:, None] * w
    if s["bias"] is not None:
        y = y + f(s["bias"])
    return {"y": y, "h": h, "mean": mean, "rstd": rstd}
