"""Experts and adapters on whole numbers, where a sum has no rounding: long sums, each term of which shows in the result
(test_exact_data.py leaves them out one step after the other)."""
import pytest
import torch

import dense_bf16_gemm_persistent_gb300 as gb
from tests import exact_data as exact
from tests import more_ref
from tests.block_ref import assert_within

pytestmark = pytest.mark.gpu

DEV, BF16 = "cuda", torch.bfloat16


@pytest.mark.parametrize("d,inner", [(2056, 1416), (4099, 515), (4096, 48), (48, 4096), (264, 1000), (1000, 264), (31, 33), (40, 17)])
@pytest.mark.parametrize("t,experts,top_k", [(1, 4, 2), (11, 6, 2), (64, 4, 2), (130, 3, 2), (17, 40, 6)])
def test_experts(d, inner, t, experts, top_k):
    q = exact.moe_problem(t, d, inner, experts, d + inner + t, DEV)
    out, ids, weights = gb.moe_ffn_gated(**q, top_k=top_k)
    want_ids, want_w = more_ref.routing(q["X"], q["router"], top_k, True)
    assert torch.equal(ids.long(), want_ids)
    # exp to 2 ulp of its value and 2^-24 of its argument (below 64 here), a tree of sums, a quotient
    assert_within(weights, want_w, want_w * 2.0 ** -17 + 1e-38, "weights")
    assert_within(out, *exact.moe(q, want_ids, weights), "D")  # (with the weights that were given, which are looked at above)


def test_experts_far_into_a_long_stack():
    """Offsets of experts pass 2^31 elements: D is, bit for bit, what a copy of the two chosen experts gives."""
    experts, inner, d = 72, 3840, 8192
    x = normal(5, d, seed=1)
    x[:, 0] = 1.0
    router = torch.zeros((experts, d), dtype=BF16, device=DEV)
    router[70, 0], router[71, 0] = 3.0, 4.0  # (logits that are exact, in any order of their sum)
    w = {}
    for name, shape in (("W1", (experts, inner, d)), ("W3", (experts, inner, d)), ("W2", (experts, d, inner))):
        w[name] = torch.randn(shape, dtype=BF16, device=DEV, generator=torch.Generator(device=DEV).manual_seed(len(w))) * shape[2] ** -0.5
        assert w[name][:70].numel() > 2 ** 31
    out, ids, weights = gb.moe_ffn_gated(x, router, **w, top_k=2)
    assert torch.equal(ids, torch.tensor([[71, 70]] * 5, dtype=torch.int32, device=DEV))
    some = lambda *which: gb.moe_ffn_gated(x, router[70:], **{k: v[list(which)] for k, v in w.items()}, top_k=2)  # noqa: E731
    alone = some(70, 71)
    assert torch.equal(weights, alone[2]) and torch.equal(out, alone[0])
    # what other experts, the same two in the other's place, or none would give is another D
    for other in (some(71, 70)[0], some(68, 69)[0], some(0, 1)[0], torch.zeros_like(out)):
        assert ((out - other).float().abs() > 0.02 * out.float().abs()).float().mean() > 0.9


def normal(*shape, seed):
    return torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(BF16)


@pytest.mark.parametrize("k", [4104, 14336, 14337])
@pytest.mark.parametrize("r", [16, 40, 64])
@pytest.mark.parametrize("m,adapters", [(1, 2), (20, 3), (48, 3), (48, 60), (130, 5), (1000, 5)])
def test_adapters(m, adapters, k, r):
    for n in (264, 333):
        q = exact.lora_problem(m, n, k, r, adapters, m + r + k, DEV)
        assert torch.equal(gb.lora(**q), exact.lora(q))
    q["ids"].fill_(adapters - 1)  # one request's
    assert torch.equal(gb.lora(**q), exact.lora(q))


@pytest.mark.parametrize("m", [200, 1000])
@pytest.mark.parametrize("n", [333, 1000])
@pytest.mark.parametrize("r", [16, 64])
@pytest.mark.parametrize("extra,offset", [(0, 0), (8, 0), (3, 1), (0, 5)])
def test_adapters_in_place_with_rows_in_any_order(m, n, r, extra, offset):
    """A block's rows lie anywhere in the matrix, beside rows that other blocks write at the time."""
    q = exact.lora_problem(m, n, 264, r, 7, m + n + r, DEV)
    want = exact.lora(q)
    assert torch.equal(gb.lora(**q), want)
    room = torch.full((offset + m * (n + extra) + 16,), 9.0, dtype=BF16, device=DEV)
    rows = room[offset:offset + m * (n + extra)].view(m, n + extra)
    for _ in range(3):
        rows[:, :n] = q["R"]
        gb.lora(**dict(q, R=rows[:, :n]), out=rows[:, :n])
        assert torch.equal(rows[:, :n], want)
        assert (rows[:, n:] == 9).all() and (room[:offset] == 9).all() and (room[offset + m * (n + extra):] == 9).all()


@pytest.mark.parametrize("d,extra,offset", [(264, 0, 0), (136, 3, 1)])
def test_experts_in_place_over_several_passes(d, extra, offset):
    q = exact.moe_problem(130, d, 72, 12, d, DEV)
    want, ids, weights = gb.moe_ffn_gated(**q, top_k=4)
    assert_within(want, *exact.moe(q, ids.long(), weights), "D")
    rows = torch.full((130 * (d + extra) + offset,), 9.0, dtype=BF16, device=DEV)[offset:].view(130, d + extra)
    rows[:, :d] = q["R"]
    gb.moe_ffn_gated(**dict(q, R=rows[:, :d]), top_k=4, out=rows[:, :d])
    assert torch.equal(rows[:, :d], want) and (rows[:, d:] == 9).all()
