"""Layer norm, adapters and experts as a program uses them together: a block that serves many requests' tokens, captured
into a graph and replayed with other requests; and a biased GELU block's training step.  Each step is held to its
definition in 64 bits on the inputs that the steps before really gave."""
import pytest
import torch

import dense_bf16_gemm_persistent_gb300 as gb
from tests import block_ref as ref
from tests import more_ref
from tests.block_ref import HALF_BF16, assert_within

pytestmark = pytest.mark.gpu

DEV, BF16 = "cuda", torch.bfloat16


def normal(*shape, seed, std=1.0, shift=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * std + shift).to(BF16)


def linear_within(got, x, w, bias, r, what):
    want = x.double() @ w.double().T
    off = (x.shape[1] + 8) * 2.0 ** -23 * (x.double().abs() @ w.double().abs().T)
    for t in (bias, r):
        if t is not None:
            want = want + t.double()
            off = off + 2.0 ** -23 * want.abs()
    assert_within(got, want, HALF_BF16 * (want.abs() + off) + off + 1e-37, what)


@pytest.mark.parametrize("tokens", [1, 7, 24])
def test_a_block_that_serves_many_requests(tokens):
    d, experts, inner, top, adapters, rank = 512, 8, 320, 2, 5, 16
    x, stream = normal(tokens, d, seed=1), normal(tokens, d, seed=2)
    n1, b1, n2, b2 = (normal(d, seed=s, std=0.2, shift=1.0 if s % 2 else 0.0) for s in (3, 4, 5, 6))
    w, bias = normal(d, d, seed=7, std=d ** -0.5), normal(d, seed=8, std=0.1)
    a, b = normal(adapters, rank, d, seed=9, std=d ** -0.5), normal(adapters, d, rank, seed=10, std=0.2)
    scale = torch.rand(adapters, device=DEV) + 0.5
    router = normal(experts, d, seed=11, std=2 * d ** -0.5)
    w1, w3 = normal(experts, inner, d, seed=12, std=d ** -0.5), normal(experts, inner, d, seed=13, std=d ** -0.5)
    w2 = normal(experts, d, inner, seed=14, std=inner ** -0.5)
    ids = (torch.arange(tokens, device=DEV) % (adapters + 1) - 1).to(torch.int32)

    def block():
        y1, h1, _, _ = gb.add_layer_norm(x, n1, b1, stream)
        p = gb.linear(y1, w, bias, R=gb.lora(y1, a, b, ids, scale, R=h1), split_k="auto")
        y2, h2, _, _ = gb.add_layer_norm(p, n2, b2)
        out, chosen, weights = gb.moe_ffn_gated(y2, router, w1, w3, w2, top, R=h2)
        return y1, h1, p, y2, h2, out, chosen, weights

    def check(got):
        y1, h1, p, y2, h2, out, chosen, weights = got
        want = more_ref.layer_norm(x, stream, n1, b1, 1e-5)
        assert_within(y1, *want["y"])
        assert_within(h1, *want["h"])
        delta, tol = more_ref.lora(y1, a, b, ids, scale, h1)
        base = y1.double() @ w.double().T + bias.double()
        off = tol + (d + 8) * 2.0 ** -23 * (y1.double().abs() @ w.double().abs().T) + 2.0 ** -22 * base.abs()
        assert_within(p, base + delta, off + HALF_BF16 * ((base + delta).abs() + off) + 1e-37, "projection")
        assert h2 is p or torch.equal(h2, p)
        assert_within(y2, *more_ref.layer_norm(p, None, n2, b2, 1e-5)["y"])
        want_ids, want_w = more_ref.routing(y2, router, top, True)
        assert torch.equal(chosen.long(), want_ids)
        moved, tol = more_ref.moe(y2, w1, w3, w2, h2, want_ids, want_w)
        assert_within(out, moved, tol + 2.0 ** -15 * (moved - h2.double()).abs(), "experts")
    check(block())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = block()
    for seed in (20, 21):  # other tokens of other requests
        x.copy_(normal(tokens, d, seed=seed))
        ids.copy_(ids.roll(1))
        graph.replay()
        torch.cuda.synchronize()
        check(captured)
    gb.device_status()


def test_a_training_step_of_a_biased_gelu_block():
    m, d, inner = 300, 264, 520
    x, r = normal(m, d, seed=1), normal(m, d, seed=2, shift=0.2)
    n, b = normal(d, seed=3, std=0.2, shift=1.0), normal(d, seed=4, std=0.2)
    w1, c1 = normal(inner, d, seed=5, std=d ** -0.5), normal(inner, seed=6, std=0.1)
    w2 = normal(d, inner, seed=7, std=inner ** -0.5)
    y, h, mean, rstd = gb.add_layer_norm(x, n, b, r)
    act, z = gb.linear_preact(y, w1, c1, act="gelu_tanh")
    out = gb.linear(act, w2, R=h)
    linear_within(out, act, w2, None, h, "output")

    dout = normal(m, d, seed=8)
    dz = gb.linear_dact(dout, w2, z, act="gelu_tanh")
    dy = gb.matmul(dz, w1)
    dx, dr, dn, db = gb.add_layer_norm_backward(dy, h, n, mean, rstd, dH=dout)
    want_r, want_n, want_b = more_ref.layer_norm_gradient(dy, h, n, mean, rstd, dout)
    e_r, e_n, e_b = more_ref.layer_norm_gradient_tolerances(dy, h, n, mean, rstd, dout, want_r)
    assert dx is dr or torch.equal(dx, dr)
    assert_within(dr, want_r, HALF_BF16 * (want_r.abs() + e_r) + e_r + 1e-37, "dR")
    assert_within(dn, want_n, e_n, "dweight")
    assert_within(db, want_b, e_b, "dbias")

    # The whole step against differences of the block in 64 bits, along one direction of all that it depends on.
    # Roundings to bf16 stand between (Y, Z and the activation; dZ, dY and dX): each is 2^-8 of its vector at most and
    # acts on the slope as the vector itself does, six of them.
    t = [v.double() for v in (x, r, n, b)]
    move = [torch.randn(v.shape, generator=torch.Generator(device=DEV).manual_seed(30 + i), device=DEV, dtype=torch.float64)
            for i, v in enumerate(t)]

    def loss(s):
        x_, r_, n_, b_ = (v + s * u for v, u in zip(t, move))
        h_ = x_ + r_
        off = h_ - h_.mean(dim=1, keepdim=True)
        y_ = off * (off.square().mean(dim=1, keepdim=True) + 1e-5).rsqrt() * n_ + b_
        a_ = ref.act(y_ @ w1.double().T + c1.double(), "gelu_tanh")
        return ((a_ @ w2.double().T + h_) * dout.double()).sum()
    slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
    parts = [(g.double() * u).sum() for g, u in zip((dx, dr, dn, db), move)]
    size = sum((g.double().norm() * u.norm() / max(u.numel(), 1) ** 0.5) for g, u in zip((dx, dr, dn, db), move))
    assert abs(sum(parts) - slope) < 6 * HALF_BF16 * size, (sum(parts).item(), slope.item(), size.item())
