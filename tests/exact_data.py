"""Adapters and experts on whole numbers (times powers of two): every fp32 sum of a product is exact in any order, so that a
result shows each term of a long sum.  (A tolerance for rounded sums grows with their length, and beyond a few thousand terms
it is larger than what 32 of them give.)
"""
from __future__ import annotations

import math

import torch

from tests.block_ref import HALF_BF16, TINY, act

BF16 = torch.bfloat16
STEP = 32  # columns that the kernels take at a time


def signs(gen, *shape, of=1.0):
    """+-of, in rows that start 16-byte aligned, NaN between them."""
    t = torch.full((*shape[:-1], -(-shape[-1] // 8) * 8), float("nan"), dtype=BF16, device=gen.device)[..., :shape[-1]]
    return t.copy_((torch.randint(0, 2, shape, generator=gen, device=gen.device) * 2 - 1) * of)


def spans(n):
    """The steps of n columns, the last one cut off."""
    return [(at, min(at + STEP, n)) for at in range(0, n, STEP)]


# ------------------------------------------------------------------------------------------------ adapters

def lora_problem(m, n, k, r, adapters, seed, device):
    gen = torch.Generator(device=device).manual_seed(seed)
    b = signs(gen, adapters, n, r)
    b *= torch.randint(1, 3, b.shape, generator=gen, device=device)
    q = dict(X=signs(gen, m, k), A=signs(gen, adapters, r, k), B=b,
             ids=torch.randint(-1, adapters, (m,), generator=gen, device=device).to(torch.int32),
             scale=2.0 ** torch.randint(-1, 2, (adapters,), generator=gen, device=device),
             R=torch.randint(-64, 65, (m, n), generator=gen, device=device).to(BF16))
    # X A^T has 15 bits at most (two bf16 terms have 16), and the sum over the ranks, in halves, 24
    assert k < 2 ** 15 and 2 * (2 * k * r * 2 + 64) < 2 ** 24
    return q


def lora(q, without=(0, 0)):
    """D as it has to be, bit for bit, or with a range of X's columns left out."""
    x, a, b = q["X"].double(), q["A"].double(), q["B"].double()
    v = q["R"].double().clone()
    x[:, without[0]:without[1]] = 0
    for i in range(a.shape[0]):
        rows = (q["ids"] == i).nonzero()[:, 0]
        v[rows] += (x[rows] @ a[i].T * q["scale"][i].double()) @ b[i].T
    return v.float().to(BF16)  # (exact in fp32: rounded once)


# ------------------------------------------------------------------------------------------------ experts

def moe_problem(t, d, inner, experts, seed, device):
    """W1 x and W3 x are of order 2; W2's rows have few numbers that are not zero, so that a column of the inner activation
    is a good part of some of D's."""
    gen = torch.Generator(device=device).manual_seed(seed)
    unit = 2.0 ** -max(0, round(math.log2(math.sqrt(d) / 2)))
    assert d < 2 ** 23
    few = max(4, -(-inner // d))
    w2 = signs(gen, experts, d, inner)
    at = torch.arange(d, device=device)[:, None] * few + torch.arange(few, device=device)
    keep = torch.zeros((d, inner), dtype=torch.bool, device=device).scatter_(1, at % inner, True)
    assert keep.any(dim=0).all()
    w2 *= keep
    return dict(X=signs(gen, t, d), router=(torch.randn((experts, d), generator=gen, device=device) * 2 * d ** -0.5).to(BF16)
                if d % 8 == 0 else signs(gen, experts, d, of=2.0 ** -4),
                W1=signs(gen, experts, inner, d, of=unit), W3=signs(gen, experts, inner, d, of=unit), W2=w2,
                R=torch.randint(-2, 3, (t, d), generator=gen, device=device).to(BF16))


def moe(q, ids, weights, without=(0, 0), without_inner=(0, 0), only_gate=False):
    """(D, tolerance) for a choice and its weights; or with a range of the first products' columns (of W1's only), or of
    the second's, left out."""
    x, r = q["X"].double(), q["R"].double()
    out, tol = torch.zeros_like(r), torch.zeros_like(r)
    few = int((q["W2"][0] != 0).sum(dim=1).max())
    short = x.clone()
    short[:, without[0]:without[1]] = 0
    for e in ids.unique().tolist():
        at = ids == e
        rows = at.any(dim=1).nonzero()[:, 0]
        w = (weights.double() * at).sum(dim=1)[rows][:, None]
        a = short[rows] @ q["W1"][e].double().T
        b = (x if only_gate else short)[rows] @ q["W3"][e].double().T
        y = act(a, "silu") * b
        # a and b are exact; the activation is computed to 2^-20 of its argument, two bf16 terms keep 2^-16 of y
        off = 2.0 ** -20 * a.abs() * b.abs() + (2.0 ** -16 + 2.0 ** -23) * y.abs()
        y[:, without_inner[0]:without_inner[1]] = 0
        w2 = q["W2"][e].double()
        out[rows] += w * (y @ w2.T)
        # sums of the two terms of `few` numbers (zeros add exactly), what a warp's part adds, and the warps' parts
        n = ids.shape[1] * few
        tol[rows] += w * ((off + (3 * n + 72) * 2.0 ** -23 * y.abs()) @ w2.abs().T)
    out = out + r
    return out, tol + HALF_BF16 * (out.abs() + tol) + 2.0 ** -23 * out.abs() + TINY
