"""The feed-forward block of examples/ffn_block.py: the training step against a plain step in 64
bits, and the serving step against the same block on the widened 4-bit weights."""
import importlib.util
import os

import pytest
import torch

from tests import block_ref as ref

pytestmark = pytest.mark.gpu

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "ffn_block.py")


@pytest.fixture(scope="module")
def block():
    spec = importlib.util.spec_from_file_location("ffn_block", _PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain_step(t, block, seed):
    names = ("x", "r", "weight", "w1", "w3", "w2")
    v = {k: t[k].double().requires_grad_() for k in names}
    m, d = t["x"].shape

    def drop(z, offset):
        keep = ref.keep_mask(m, d, block.P, seed, offset).to(z.device)
        return torch.where(keep, z / (1 - block.P), torch.zeros_like(z))
    h = drop(v["x"], 0) + v["r"]
    n = h * (h.square().mean(dim=1, keepdim=True) + block.EPS).rsqrt() * v["weight"]
    a = torch.nn.functional.silu(n @ v["w1"].T) * (n @ v["w3"].T)
    out = drop(a @ v["w2"].T, 1) + h
    return out, [v[k] for k in names]


def test_training_step(block):
    t = block.make(tokens=48, width=256, inner=384, seed=3)
    matrices = t["w1"], t["w3"], t["w2"]
    out, saved = block.forward(t["x"], t["r"], t["weight"], *matrices, seed=11)
    dout = torch.randn_like(out)
    grads = block.backward(dout, saved, t["weight"], *matrices, seed=11)
    want, leaves = plain_step(t, block, 11)
    want_grads = torch.autograd.grad(want, leaves, dout.double())
    # each result is a chain of at most ten bf16 roundings of 2^-8 that add up as their squares do: 2^-6 of its norm
    for got, expected in ((out, want), *zip(grads, want_grads)):
        assert (got.double() - expected).norm() < 2.0 ** -6 * expected.norm()


@pytest.mark.parametrize("tokens", [1, 5, 17])
def test_serving_step(block, tokens):
    t = block.make(tokens=tokens, width=256, inner=384, seed=tokens)
    packed = [block.quantize_w4(t[k]) for k in ("w1", "w3", "w2")]
    got = block.serve(t["x"], t["r"], t["weight"], *packed).double()
    w1, w3, w2 = (ref.unpack_w4(*p, block.GROUP, k) for p, k in zip(packed, (256, 256, 384)))
    h = t["x"].double() + t["r"].double()
    n = h * (h.square().mean(dim=1, keepdim=True) + block.EPS).rsqrt() * t["weight"].double()
    want = (torch.nn.functional.silu(n @ w1.T) * (n @ w3.T)) @ w2.T + h
    # e4m3 rounds the norm's output by at most 2^-4: the branch is off by less than 2^-3 of its norm
    assert (got - want).norm() < 2.0 ** -3 * (want - h).norm() + 2.0 ** -7 * want.norm()
    # the 4-bit weights themselves are near the weights they stand for: half a step of 15 for each
    for w, k in ((w1, "w1"), (w3, "w3"), (w2, "w2")):
        parts = t[k].double().view(t[k].shape[0], -1, block.GROUP)
        step = (parts.amax(dim=2).clamp_min(0) - parts.amin(dim=2).clamp_max(0)) / 15
        off = (w.view_as(parts) - parts).abs().amax(dim=2)
        assert (off <= 1.02 * step).all()  # half a step for q, half for z, the scale's own rounding
