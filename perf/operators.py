"""The operators around a linear layer, as they are measured: cases, inputs, plain forms and definitions in 64 bits.

Three operators of the feed-forward block beside its products:

* ``linear_w4`` / ``ffn_gated_w4``: a linear layer, and the gated pair of layers, for a few tokens, with 4-bit
  weights and a scale (and a zero point) for each group of a row:  W[n,k] = (q[n,k] - z[n,k/G]) * s[n,k/G].
* ``add_rms_norm``: root-mean-square norm with the residual's addition (and dropout of the branch before it),
  its output in bf16 for training, with the backward pass, or in 8 bits with scales for serving.
* ``dropout``: dropout from a counter-based generator, with an optional residual; the mask is computed again
  where it is needed (the backward pass is the same call on the gradient).
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
FP8_MAX = 448.0         # the largest finite e4m3 value
MIN_SCALE = 2.0 ** -126  # the smallest scale of an 8-bit row or group (an all-zero one has this scale)


# ---------------------------------------------------------------------------------------------- cases

def listed():
    w4 = {"op": "linear_w4", "act": "none", "bias": False, "residual": False, "zeros": False, "x8": "no"}
    ffn = {"op": "ffn_gated_w4", "zeros": False, "x8": "no"}
    return [
        # The attention output projection of a 4096-wide model, one new token: the smallest product, latency counts.
        dict(w4, name="w4_1x4096x4096", m=1, n=4096, k=4096, group=128, residual=True),
        # The down projection for 16 sequences decoded together, added onto the residual stream; asymmetric weights.
        dict(w4, name="w4_16x4096x14336", m=16, n=4096, k=14336, group=64, zeros=True, residual=True),
        # A biased layer of odd width on 8-bit activations, five drafted tokens; K ends inside a 128-wide block.
        dict(w4, name="w4_5x4099x4128_x8", m=5, n=4099, k=4128, group=32, zeros=True, bias=True, act="gelu_tanh",
             x8="group"),
        # The vocabulary's projection for 8 sequences: the largest weight matrix that a decoding step reads.
        dict(w4, name="w4_8x131072x8192", m=8, n=131072, k=8192, group=128),
        # The gated pair of a feed-forward block, one new token.
        dict(ffn, name="ffn_w4_1x14336x4096", m=1, n=14336, k=4096, group=128),
        # The same pair for 32 sequences, reading the norm's 8-bit output with one scale a row.
        dict(ffn, name="ffn_w4_32x14336x4096_x8", m=32, n=14336, k=4096, group=128, x8="row"),
        # The norm in front of a block for one new token, 8-bit output with one scale a row: pure latency.
        {"op": "norm_q8", "name": "norm_q8_1x4096", "m": 1, "d": 4096, "scale_group": 0},
        # Training, forward: the branch's dropout, the residual's addition and the norm in one pass.
        {"op": "norm_fwd", "name": "norm_fwd_8192x4096_drop", "m": 8192, "d": 4096, "p": 0.1, "residual": True},
        # Training, backward: gradients of the branch, of the residual stream and of the norm's weight.
        {"op": "norm_bwd", "name": "norm_bwd_8192x4096_drop", "m": 8192, "d": 4096, "p": 0.1, "dh": True},
        # The same without dropout, with rows of an odd width (none but every eighth starts on 16 bytes).
        {"op": "norm_bwd", "name": "norm_bwd_3001x4099", "m": 3001, "d": 4099, "p": 0.0, "dh": True},
        # Dropout of a feed-forward block's inner activation in training, added to a second tensor.
        {"op": "dropout", "name": "dropout_8192x14336_add", "m": 8192, "n": 14336, "p": 0.1, "residual": True},
        # Its backward pass on rows of an odd width.
        {"op": "dropout", "name": "dropout_1000x4099", "m": 1000, "n": 4099, "p": 0.25, "residual": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear_w4", "linear_w4", "ffn_gated_w4", "norm_q8", "norm_fwd", "norm_bwd", "dropout"])
    if op in ("linear_w4", "ffn_gated_w4"):
        m = _log(rng, 1, 32)
        k = 32 * _log(rng, 512 // 32, 16384 // 32)
        if rng.random() < 0.5:
            k = max(512, k // 512 * 512)
        mats = 2 if op == "ffn_gated_w4" else 1
        # no more weights than the largest listed product has, and no more multiplications
        n = min(_log(rng, 96, 131072), (1 << 30) * min(1, 8 / m) // (k * mats))
        n = max(96, int(n))
        if rng.random() < 0.5:
            n = max(96, n // 16 * 16)
        case = {"op": op, "m": m, "n": n, "k": k, "group": rng.choice([32, 64, 128, 128]),
                "zeros": rng.random() < 0.5, "x8": rng.choice(["no", "no", "row", "group"])}
        if op == "linear_w4":
            case |= {"act": rng.choice(["none", "gelu_tanh", "silu", "relu"]), "bias": rng.random() < 0.3,
                     "residual": rng.random() < 0.5}
        return case
    if op == "dropout":
        n = _log(rng, 64, 16384)
        m = min(_log(rng, 1, 16384), 8192 * 14336 // n)
        return {"op": op, "m": m, "n": n // 8 * 8 if rng.random() < 0.6 else n, "p": rng.choice([0.05, 0.1, 0.25, 0.5]),
                "residual": rng.random() < 0.5}
    d = _log(rng, 64, 16384)
    d = d // 8 * 8 if rng.random() < 0.6 else d
    m = min(_log(rng, 1, 16384), 8192 * 14336 // (2 * d))
    p = rng.choice([0.0, 0.0, 0.1, 0.3])
    if op == "norm_q8":
        return {"op": op, "m": m, "d": d, "scale_group": rng.choice([0, 128])}
    if op == "norm_fwd":
        return {"op": op, "m": m, "d": d, "p": p, "residual": rng.random() < 0.8}
    return {"op": op, "m": m, "d": d, "p": p, "dh": rng.random() < 0.8}


# ---------------------------------------------------------------------------------------------- inputs

def _normal(gen, *shape, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


def _weights_4bit(gen, n, k, group, zeros):
    """Packed nibbles [n, k/2] (even k in the low nibble), scales [n, groups] and zero points [n, groups] or None."""
    groups = -(-k // group)
    packed = torch.empty((n, k // 2), dtype=torch.uint8, device="cuda")
    rows = max(1, (1 << 26) // k)
    for at in range(0, n, rows):
        part = packed[at:at + rows]
        # weights of a trained layer are near normal: the nibbles gather around the middle of their range
        q = (torch.randn((part.shape[0], k), generator=gen, device="cuda") * 2.6 + 8.0).round_().clamp_(0, 15)
        q = q.to(torch.uint8)
        part.copy_(q[:, 0::2] | (q[:, 1::2] << 4))
    scales = (torch.rand((n, groups), generator=gen, device="cuda") * 0.4 + 0.8) * (0.02 / 2.6)
    z = None
    if zeros:
        z = torch.randint(5, 12, (n, groups), generator=gen, device="cuda").to(torch.uint8)
    return packed, scales.to(torch.bfloat16), z


def _activations(gen, m, k, x8):
    """Rows of unit size, some channels larger than the others: bf16, or e4m3 with scales of a row or of 128 columns."""
    x = torch.randn((m, k), generator=gen, device="cuda")
    x = x * (1.0 + 4.0 * (torch.rand((k,), generator=gen, device="cuda") < 0.01))
    if x8 == "no":
        return x.to(torch.bfloat16), None
    width = 128 if x8 == "group" else k
    scale = torch.stack([part.abs().amax(dim=1) for part in x.split(width, dim=1)], dim=1) / FP8_MAX
    q = x / scale.repeat_interleave(width, dim=1)[:, :k]
    return q.to(torch.float8_e4m3fn), scale.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 11)
    s = {"case": dict(case)}
    op = case["op"]
    if op in ("linear_w4", "ffn_gated_w4"):
        m, n, k, group = case["m"], case["n"], case["k"], case["group"]
        s["x"], s["x_scale"] = _activations(gen, m, k, case["x8"])
        s["w"], s["s"], s["z"] = _weights_4bit(gen, n, k, group, case["zeros"])
        if op == "ffn_gated_w4":
            s["w3"], s["s3"], s["z3"] = _weights_4bit(gen, n, k, group, case["zeros"])
        else:
            s["bias"] = _normal(gen, n, std=0.1) if case["bias"] else None
            s["r"] = _normal(gen, m, n) if case["residual"] else None
        return s
    s["seed"], s["offset"] = int(seed) * 1000003 + 17, 5
    if op == "dropout":
        s["x"] = _normal(gen, case["m"], case["n"])
        s["r"] = _normal(gen, case["m"], case["n"]) if case["residual"] else None
        return s
    m, d = case["m"], case["d"]
    s["weight"] = (torch.rand((d,), generator=gen, device="cuda") + 0.5).to(torch.bfloat16)
    if op == "norm_bwd":
        s["dy"] = _normal(gen, m, d, std=0.05)
        s["dh"] = _normal(gen, m, d, std=0.05) if case["dh"] else None
        s["h"] = _normal(gen, m, d, std=1.5)
        s["rstd"] = torch.rsqrt(s["h"].float().square().mean(dim=1) + EPS)
        return s
    s["x"] = _normal(gen, m, d)
    s["r"] = _normal(gen, m, d, std=1.5) if case.get("residual", True) else None
    return s


# ---------------------------------------------------------------------------------------------- one pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import dense_bf16_gemm_persistent_gb300 as gb
    c = s["case"]
    op = c["op"]
    if op == "linear_w4":
        return gb.linear_w4(s["x"], s["w"], s["s"], s["bias"], s["r"], act=c["act"], zeros=s["z"], group=c["group"],
                            x_scale=s["x_scale"])
    if op == "ffn_gated_w4":
        return gb.ffn_gated_w4(s["x"], s["w"], s["s"], s["w3"], s["s3"], zeros1=s["z"], zeros3=s["z3"],
                               group=c["group"], x_scale=s["x_scale"])
    if op == "dropout":
        return gb.dropout(s["x"], c["p"], s["seed"], s["offset"], R=s["r"])
    if op == "norm_q8":
        q, scale, h = gb.add_rms_norm_q8(s["x"], s["weight"], s["r"], eps=EPS, scale_group=c["scale_group"])
        return {"q": q, "scale": scale, "h": h}
    if op == "norm_fwd":
        y, h, rstd = gb.add_rms_norm(s["x"], s["weight"], s["r"], eps=EPS, p=c["p"], seed=s["seed"],
                                     offset=s["offset"])
        return {"y": y, "h": h, "rstd": rstd}
    dx, dr, dw = gb.add_rms_norm_backward(s["dy"], s["h"], s["weight"], s["rstd"], dH=s["dh"], p=c["p"],
                                          seed=s["seed"], offset=s["offset"])
    return {"dx": dx, "dr": dr, "dweight": dw}


# ---- plain forms: elementary torch operations in 32 bits, rounded once at the end

def _unpack(w, scales, zeros, group, k):
    q = torch.stack([w & 15, w >> 4], dim=2).reshape(w.shape[0], k).float()
    z = zeros.float() if zeros is not None else torch.full_like(scales, 8.0, dtype=torch.float32)
    wide = lambda t: t.repeat_interleave(group, dim=1)[:, :k]  # noqa: E731
    return (q - wide(z)) * wide(scales.float())


def _scaled(x, x_scale):
    if x_scale is None:
        return x.float()
    width = 128 if x_scale.shape[1] > 1 else x.shape[1]
    return x.float() * x_scale.repeat_interleave(width, dim=1)[:, :x.shape[1]]


def _act(v, act):
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    return v.clamp_min(0.0) if act == "relu" else v


def _philox_words(rows, groups, seed, offset):
    """Philox4x32-10 (Salmon, Moraes, Dror, Shaw, 2011) of the counters (group, row, offset), as int64 [rows, groups, 4]."""
    low = 0xFFFFFFFF
    c0 = torch.arange(groups, device="cuda").expand(rows, groups)
    c1 = torch.arange(rows, device="cuda")[:, None].expand(rows, groups)
    c2 = torch.full_like(c0, offset & low)
    c3 = torch.full_like(c0, offset >> 32)
    k0, k1 = seed & low, seed >> 32 & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # (products of 32-bit words wrap in 64 bits; their words are right)
        c0, c1, c2, c3 = (b >> 32 & low) ^ c1 ^ k0, b & low, (a >> 32 & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack([c0, c1, c2, c3], dim=2)


def _dropped(x, p, seed, offset):
    """x where it is kept, times 1 / (1 - p), in 32 bits."""
    if p == 0.0:
        return x.float()
    words = _philox_words(x.shape[0], -(-x.shape[1] // 4), seed, offset)
    keep = words.reshape(x.shape[0], -1)[:, :x.shape[1]] >= round(p * 2 ** 32)
    return torch.where(keep, x.float() * (1.0 / (1.0 - p)), 0.0)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "linear_w4":
        v = _scaled(s["x"], s["x_scale"]) @ _unpack(s["w"], s["s"], s["z"], c["group"], c["k"]).T
        if s["bias"] is not None:
            v = v + s["bias"].float()
        v = _act(v, c["act"])
        return (v + s["r"].float() if s["r"] is not None else v).to(torch.bfloat16)
    if op == "ffn_gated_w4":
        x = _scaled(s["x"], s["x_scale"])
        a = x @ _unpack(s["w"], s["s"], s["z"], c["group"], c["k"]).T
        b = x @ _unpack(s["w3"], s["s3"], s["z3"], c["group"], c["k"]).T
        return (_act(a, "silu") * b).to(torch.bfloat16)
    if op == "dropout":
        v = _dropped(s["x"], c["p"], s["seed"], s["offset"])
        return (v + s["r"].float() if s["r"] is not None else v).to(torch.bfloat16)
    w = s["weight"].float()
    if op == "norm_bwd":
        xhat = s["h"].float() * s["rstd"][:, None]
        g = s["dy"].float() * w
        dr = s["rstd"][:, None] * (g - xhat * (g * xhat).mean(dim=1, keepdim=True))
        if s["dh"] is not None:
            dr = dr + s["dh"].float()
        dw = (s["dy"].float() * xhat).sum(dim=0)
        return {"dx": _dropped(dr, c["p"], s["seed"], s["offset"]).to(torch.bfloat16), "dr": dr.to(torch.bfloat16),
                "dweight": dw}
    h = _dropped(s["x"], c.get("p", 0.0), s["seed"], s["offset"])
    if s["r"] is not None:
        h = h + s["r"].float()
    rstd = torch.rsqrt(h.square().mean(dim=1) + EPS)
    y = h * rstd[:, None] * w
    if op == "norm_fwd":
        return {"y": y.to(torch.bfloat16), "h": h.to(torch.bfloat16), "rstd": rstd}
    width = c["scale_group"] or c["d"]
    pad = -c["d"] % width
    parts = torch.nn.functional.pad(y, (0, pad)).reshape(c["m"], -1, width)
    scale = (parts.abs().amax(dim=2) / FP8_MAX).clamp_min(MIN_SCALE)
    q = (parts / scale[:, :, None]).reshape(c["m"], -1)[:, :c["d"]].to(torch.float8_e4m3fn)
    return {"q": q, "scale": scale, "h": h.to(torch.bfloat16)}


# ---------------------------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op in ("linear_w4", "ffn_gated_w4"):
        m, n, k = case["m"], case["n"], case["k"]
        groups = -(-k // case["group"])
        mats = 2 if op == "ffn_gated_w4" else 1
        b = mats * n * (k // 2 + groups * (3 if case["zeros"] else 2)) + 2 * m * n
        b += m * k * (2 if case["x8"] == "no" else 1)
        b += {"no": 0, "row": 4 * m, "group": 4 * m * -(-k // 128)}[case["x8"]]
        if case.get("residual"):
            b += 2 * m * n
        if case.get("bias"):
            b += 2 * n
        return {"bytes": b, "flops": 2 * mats * m * n * k}
    if op == "dropout":
        e = case["m"] * case["n"]
        return {"bytes": e * (6 if case["residual"] else 4), "flops": 2 * e}
    m, d = case["m"], case["d"]
    e = m * d
    if op == "norm_bwd":
        # dY, H and dH read; dR, and dX where dropout makes it another tensor, written; the weight and its gradient
        return {"bytes": 2 * e * (3 + case["dh"] + (case["p"] > 0)) + 4 * m + 6 * d, "flops": 12 * e}
    if op == "norm_q8":
        # X and R read, H and the 8-bit output written, the weight, the scales
        return {"bytes": 7 * e + 2 * d + 4 * m * (-(-d // case["scale_group"]) if case["scale_group"] else 1),
                "flops": 8 * e}
    apart = case["residual"] or case["p"] > 0  # H is another tensor than X
    return {"bytes": 2 * e * (2 + case["residual"] + apart) + 2 * d + 4 * m, "flops": 8 * e}


# ---------------------------------------------------------------------------------------------- 64 bits

def _exact_keep(m, n, p, seed, offset):
    """The kept elements of an [m, n] matrix, the generator's rounds written with numpy's unsigned words."""
    out = np.empty((m, n), dtype=bool)
    words = -(-n // 4)
    step = max(1, (1 << 16) // words)
    mask, limit = np.uint64(0xFFFFFFFF), int(round(p * 2 ** 32))
    for at in range(0, m, step):
        rows = min(step, m - at)
        ctr = np.zeros((4, rows, words), dtype=np.uint64)
        ctr[0] = np.arange(words, dtype=np.uint64)
        ctr[1] = np.arange(at, at + rows, dtype=np.uint64)[:, None]
        ctr[2], ctr[3] = offset % 2 ** 32, offset // 2 ** 32
        key = [seed % 2 ** 32, seed // 2 ** 32 % 2 ** 32]
        for _ in range(10):
            left, right = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
            ctr = [(right >> np.uint64(32)) ^ ctr[1] ^ np.uint64(key[0]), right & mask,
                   (left >> np.uint64(32)) ^ ctr[3] ^ np.uint64(key[1]), left & mask]
            key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
        out[at:at + rows] = np.stack(ctr, axis=-1).reshape(rows, 4 * words)[:, :n] >= np.uint64(limit)
    return torch.from_numpy(out).cuda()


def _exact_linear(x, x_scale, w, scales, zeros, group):
    """x . W^T group by group, in 64 bits."""
    m, k = x.shape
    xs = x.double()
    total = torch.zeros((m, w.shape[0]), dtype=torch.float64, device="cuda")
    for at in range(0, k, 128):
        to = min(k, at + 128)
        xb = xs[:, at:to]
        if x_scale is not None:
            xb = xb * (x_scale[:, at // 128] if x_scale.shape[1] > 1 else x_scale[:, 0]).double()[:, None]
        bytes_ = w[:, at // 2:to // 2]
        q = torch.empty((w.shape[0], to - at), dtype=torch.float64, device="cuda")
        q[:, 0::2] = torch.bitwise_and(bytes_, 0x0F).double()
        q[:, 1::2] = torch.div(bytes_, 16, rounding_mode="floor").double()
        for g in range(at, to, group):
            i = g // group
            part = slice(g - at, min(to, g + group) - at)
            mid = zeros[:, i].double()[:, None] if zeros is not None else 8.0
            total += (xb[:, part] @ (q[:, part] - mid).T) * scales[:, i].double()
    return total


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f = lambda t: t.double()  # noqa: E731
    if op in ("linear_w4", "ffn_gated_w4"):
        v = _exact_linear(s["x"], s["x_scale"], s["w"], s["s"], s["z"], case["group"])
        if op == "ffn_gated_w4":
            return torch.sigmoid(v) * v * _exact_linear(s["x"], s["x_scale"], s["w3"], s["s3"], s["z3"], case["group"])
        if s["bias"] is not None:
            v += f(s["bias"])
        if case["act"] == "gelu_tanh":
            v = v * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
        elif case["act"] == "silu":
            v = v * torch.sigmoid(v)
        elif case["act"] == "relu":
            v = torch.maximum(v, torch.zeros_like(v))
        return v + f(s["r"]) if s["r"] is not None else v
    p = case.get("p", 0.0)
    m, n = (case["m"], case["n"]) if op == "dropout" else (case["m"], case["d"])
    keep = _exact_keep(m, n, p, s["seed"], s["offset"]) if p > 0 else None
    branch = lambda t: t if keep is None else torch.where(keep, t / (1.0 - p), torch.zeros_like(t))  # noqa: E731
    if op == "dropout":
        v = branch(f(s["x"]))
        return v + f(s["r"]) if s["r"] is not None else v
    w = f(s["weight"])
    if op == "norm_bwd":
        h, r, dy = f(s["h"]), f(s["rstd"])[:, None], f(s["dy"])
        dot = (dy * w * h).sum(dim=1, keepdim=True) / n
        dr = r * (dy * w) - r ** 3 * h * dot
        if s["dh"] is not None:
            dr += f(s["dh"])
        return {"dx": branch(dr), "dr": dr, "dweight": torch.einsum("md,md,mo->d", dy, h, r)}
    h = branch(f(s["x"]))
    if s["r"] is not None:
        h = h + f(s["r"])
    rstd = 1.0 / torch.sqrt(torch.sum(h * h, dim=1) / n + EPS)
    y = h * w * rstd[:, None]
    if op == "norm_fwd":
        return {"y": y, "h": h, "rstd": rstd}
    q, scales = torch.empty_like(y), []
    width = case["scale_group"] or n
    for at in range(0, n, width):
        part = y[:, at:at + width]
        scales.append(torch.clamp(part.abs().max(dim=1).values / FP8_MAX, min=MIN_SCALE))
        q[:, at:at + width] = part / scales[-1][:, None]
    return {"q": q, "scale": torch.stack(scales, dim=1), "h": h}
