"""Definitions in 64 bits of the operators around the products, and the errors that a correct
implementation may have, each from its own arithmetic.

A bf16 result is at most half a unit away from what it rounds: 2^-8 of its size.  A sum of n
terms in fp32 is off by at most n 2^-24 (2^-23 where the adder may truncate) of the sum of the
terms' sizes.
"""
from __future__ import annotations

import math

import numpy as np
import torch

HALF_BF16 = 2.0 ** -8
TINY = 1e-37  # below the smallest normal fp32 / bf16 number rounding is absolute


def philox(counter, key, rounds: int = 10):
    """Philox4x32 of Salmon et al. (SC 2011): four uint64 arrays that hold 32-bit words in, four out."""
    m32 = np.uint64(0xFFFFFFFF)
    c = [np.asarray(x, dtype=np.uint64) for x in counter]
    k0, k1 = int(key[0]), int(key[1])
    for _ in range(rounds):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), p1 & m32, (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k1),
             p0 & m32]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c


def keep_mask(m: int, n: int, p: float, seed: int, offset: int) -> torch.Tensor:
    groups = -(-n // 4)
    zero = np.zeros((m, groups), dtype=np.uint64)
    c = [zero + np.arange(groups, dtype=np.uint64), zero + np.arange(m, dtype=np.uint64)[:, None],
         zero + np.uint64(offset & 0xFFFFFFFF), zero + np.uint64(offset >> 32)]
    words = np.stack(philox(c, (seed & 0xFFFFFFFF, seed >> 32)), axis=-1).reshape(m, 4 * groups)[:, :n]
    return torch.from_numpy(words >= np.uint64(round(p * 2 ** 32)))


def dropped(x: torch.Tensor, p: float, seed: int, offset: int) -> torch.Tensor:
    x = x.double()
    if p == 0.0:
        return x
    keep = keep_mask(*x.shape, p, seed, offset).to(x.device)
    return torch.where(keep, x / (1.0 - p) if p < 1.0 else x, torch.zeros_like(x))


def unpack_w4(wq, scales, zeros, group: int, k: int) -> torch.Tensor:
    q = torch.stack([wq & 15, wq >> 4], dim=-1).reshape(wq.shape[0], k).double()
    z = zeros.double() if zeros is not None else torch.full(scales.shape, 8.0, dtype=torch.float64, device=wq.device)
    index = torch.arange(k, device=wq.device) // group
    return (q - z[:, index]) * scales.double()[:, index]


def dequantised(x, x_scale) -> torch.Tensor:
    if x_scale is None:
        return x.double()
    s = x_scale.double().reshape(x.shape[0], -1)
    index = torch.arange(x.shape[1], device=x.device) // (128 if s.shape[1] > 1 else max(x.shape[1], 1))
    return x.double() * s[:, index]


def act(v: torch.Tensor, name: str) -> torch.Tensor:
    if name == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    if name == "silu":
        return v * torch.sigmoid(v)
    return v.clamp_min(0.0) if name == "relu" else v


def w4_products(x, x_scale, w) -> tuple[torch.Tensor, torch.Tensor]:
    """(x W^T in 64 bits, the most an fp32 sum of these products may be off)."""
    xd = dequantised(x, x_scale)
    size = xd.abs() @ w.abs().T
    # per group at most 8 accumulations of 16 products each (no product is rounded), then K / 32 groups and the
    # joins of the threads' parts, with a product by the scales in each
    terms = 8 * 16 + x.shape[1] / 32 + 64 + 4
    return xd @ w.T, terms * 2.0 ** -23 * size


def assert_within(got: torch.Tensor, ref: torch.Tensor, tol: torch.Tensor, what: str = "") -> None:
    assert got.shape == ref.shape, (got.shape, ref.shape)
    g = got.double()
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(g), nan), f"{what}: NaN in other places"
    inf = torch.isinf(ref)
    assert torch.equal(g[inf], ref[inf]), f"{what}: infinities differ"
    fine = ~(nan | inf)
    off = (g - ref).abs() - tol
    bad = fine & ~(off <= 0)
    if bad.any():
        at = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values out of tolerance; first at {at}: "
                             f"got {g[at].item()!r}, expected {ref[at].item()!r} within {tol[at].item()!r}")


def norm_gradient(dy, h, w, dh, eps, rstd=None):
    """(dR, dweight) of y = h rstd(h) w and of dh . h, from the formula, in 64 bits."""
    dy, h, w = dy.double(), h.double(), w.double()
    r = ((h.square().mean(dim=1) + eps).rsqrt() if rstd is None else rstd.double())[:, None]
    xhat, g = h * r, dy * w
    dr = r * (g - xhat * (g * xhat).mean(dim=1, keepdim=True))
    if dh is not None:
        dr = dr + dh.double()
    return dr, (dy * xhat).sum(dim=0)
