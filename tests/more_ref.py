"""Definitions in 64 bits of layer norm, low-rank adapters and the mixture of experts, with the errors that a
correct implementation may have.

eps / 2 of fp32 is 2^-24: a sum of n fp32 terms, added in chains and trees, is off by at most its longest chain times
2^-24 of the sum of the terms' sizes.
"""
from __future__ import annotations

import torch

from tests import block_ref as ref
from tests.block_ref import HALF_BF16, TINY

U = 2.0 ** -24
# the longest chain of a row's sum: 32 elements a thread, two trees of five steps, and a product or two a term
ROW = 32 + 10 + 4


def layer_norm(x, r, w, b, eps, p=0.0, seed=0, offset=0):
    """{name: (value, tolerance)} of Y, H, mean and rstd."""
    h = ref.dropped(x, p, seed, offset)
    if r is not None:
        h = h + r.double()
    d = h.shape[1]
    w = w.double()
    off_h = (2 if p else 1) * 2 * U * (h.abs() + (r.double().abs() if r is not None else 0))
    mean = h.mean(dim=1, keepdim=True)
    e_mean = ROW * U * h.abs().mean(dim=1, keepdim=True) + off_h.mean(dim=1, keepdim=True)
    dev = h - mean
    var = dev.square().mean(dim=1, keepdim=True)
    # each difference is off by e_mean, its own rounding and h's; the squares' sum by its chain
    e_dev = e_mean + off_h + 2 * U * dev.abs()
    e_var = (2 * dev.abs() * e_dev + e_dev.square()).mean(dim=1, keepdim=True) + 2 * ROW * U * var
    rstd = (var + eps).rsqrt()
    e_rstd = rstd * (0.5 * e_var / (var + eps) * (1 + 2 * e_var / (var + eps)) + 8 * U)
    y = dev * rstd * w
    e_y = (e_dev * rstd + dev.abs() * e_rstd + 4 * U * (dev * rstd).abs()) * w.abs() + 4 * U * y.abs()
    if b is not None:
        y = y + b.double()
        e_y = e_y + U * (y.abs() + b.double().abs())
    up = lambda v, e: (v, HALF_BF16 * v.abs() + e * (1 + HALF_BF16) + TINY)  # noqa: E731
    return {"y": up(y, e_y), "h": up(h, off_h), "mean": (mean[:, 0], e_mean[:, 0] + U * mean[:, 0].abs() + TINY),
            "rstd": (rstd[:, 0], e_rstd[:, 0])}


def layer_norm_gradient(dy, h, w, mean, rstd, dh=None):
    """(dR, dweight, dbias) of y = (h - mean) rstd w + b and of dh . h, from the formula, in 64 bits."""
    dy, h, w, r = dy.double(), h.double(), w.double(), rstd.double()[:, None]
    xhat, g = (h - mean.double()[:, None]) * r, dy * w
    dr = r * (g - g.mean(dim=1, keepdim=True) - xhat * (g * xhat).mean(dim=1, keepdim=True))
    if dh is not None:
        dr = dr + dh.double()
    return dr, (dy * xhat).sum(dim=0), dy.sum(dim=0)


def layer_norm_gradient_tolerances(dy, h, w, mean, rstd, dh, dr):
    """What dR before its rounding, dweight and dbias may be off."""
    dy, h, w, r = dy.double(), h.double(), w.double(), rstd.double()[:, None]
    xhat, g = (h - mean.double()[:, None]) * r, dy * w
    size = g.abs() + g.abs().mean(dim=1, keepdim=True) + xhat.abs() * (g * xhat).abs().mean(dim=1, keepdim=True)
    e = r * (ROW + 8) * U * size + 2 * U * dr.abs() + (U * dh.double().abs() if dh is not None else 0)
    # a column's sum: at least eight blocks' rows one after another (a warp's where a block has eight), eight
    # warps, and the join's chain and tree
    rows = -(-dy.shape[0] // 8) + 8 + 48
    return e, (rows + 3) * U * (dy * xhat).abs().sum(dim=0) + TINY, rows * U * dy.abs().sum(dim=0) + TINY


def routing(x, router, top_k, renormalize):
    """(ids, weights) in 64 bits: the largest logits, the lower expert first where they are equal; NaN last."""
    logits = x.double() @ router.double().T
    nan = torch.isnan(logits)
    order = torch.sort(torch.where(nan, -torch.inf, logits), dim=1, descending=True, stable=True).indices[:, :top_k]
    p = torch.softmax(torch.gather(logits, 1, order) if renormalize else logits, dim=1)
    weights = p if renormalize else torch.gather(p, 1, order)
    return order, torch.where(nan.any(dim=1, keepdim=True), torch.nan, weights)


def moe(x, w1, w3, w2, r, ids, weights):
    """(D, tolerance) for a choice: in 64 bits, expert by expert."""
    t, d = x.shape
    inner = w1.shape[1]
    out = torch.zeros((t, d), dtype=torch.float64, device=x.device)
    tol = torch.zeros_like(out)
    xd = x.double()
    # an fp32 sum of n products in an mma (2^-23 each: the adder may truncate), and the joins of the warps' parts
    first, second = (d + 24) * 2.0 ** -23, (inner + 24) * 2.0 ** -23
    for e in ids.unique().tolist():
        at = (ids == e)
        rows = at.any(dim=1).nonzero()[:, 0]
        w = (weights.double() * at).sum(dim=1)[rows][:, None]
        a, b = xd[rows] @ w1[e].double().T, xd[rows] @ w3[e].double().T
        off_a = first * (xd[rows].abs() @ w1[e].double().abs().T)
        off_b = first * (xd[rows].abs() @ w3[e].double().abs().T)
        gate = ref.act(a, "silu")
        act = gate * b
        # the activation's slope is at most 1.13, it is computed to 2^-20 of its argument; two bf16 terms keep 2^-16
        off = (1.13 * off_a + 2.0 ** -20 * a.abs()) * (b.abs() + off_b) + gate.abs() * off_b + 2.0 ** -16 * act.abs()
        w2d = w2[e].double()
        out[rows] += w * (act @ w2d.T)
        tol[rows] += w.abs() * (off @ w2d.abs().T + second * (act.abs() @ w2d.abs().T)) * (1 + 2.0 ** -10)
    tol = tol + (2.0 ** -20) * out.abs()
    if r is not None:
        out = out + r.double()
    return out, tol + (HALF_BF16 + 2.0 ** -20) * out.abs() + HALF_BF16 * tol + TINY


def lora(x, a, b, ids, scale, r, act="none"):
    """(D, tolerance): row by row's adapter, in 64 bits."""
    m, k = x.shape
    count, n, rank = b.shape
    v = r.double() if r is not None else torch.zeros((m, n), dtype=torch.float64, device=x.device)
    off = U * v.abs()
    for i in ids.unique().tolist():
        if not 0 <= i < count:
            continue
        rows = (ids == i).nonzero()[:, 0]
        s = float(scale[i]) if scale is not None else 1.0
        xd, ad, bd = x[rows].double(), a[i].double(), b[i].double()
        low = xd @ ad.T * s
        # an fp32 sum of k products in an mma (2^-23 each: the adder may truncate) and the joins of its parts; the
        # product by the scale; two bf16 terms; then 2 rank products, and R
        e = (k + 48) * 2.0 ** -23 * (xd.abs() @ ad.abs().T) * abs(s) + (2.0 ** -16 + 2 * U) * low.abs()
        v[rows] += low @ bd.T
        off[rows] += e @ bd.abs().T + (2 * rank + 4) * 2.0 ** -23 * (low.abs() @ bd.abs().T)
    off = off + U * v.abs()
    want = ref.act(v, act)
    # the activations' slopes are at most 1.13; they are computed to 2^-20 of their argument
    tol = 1.13 * off + (2.0 ** -20 * v.abs() if act in ("gelu_tanh", "silu") else 0)
    return want, tol + HALF_BF16 * want.abs() + HALF_BF16 * tol + TINY
