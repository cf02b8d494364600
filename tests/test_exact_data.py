"""What the exact cases of the adapters and the experts tell apart, on the CPU: each step of a long sum."""
import pytest
import torch

from tests import exact_data as exact
from tests import more_ref

LORA = [(k, r) for k in (4104, 14336, 14337) for r in (16, 64)]
MOE = [(2056, 1416), (4099, 515), (4096, 48), (48, 4096), (264, 1000), (1000, 264), (31, 33), (40, 17)]


@pytest.mark.parametrize("k,r", LORA)
def test_a_step_of_the_adapters_that_is_left_out_shows_in_every_row(k, r):
    q = exact.lora_problem(9, 64, k, r, 3, k + r, "cpu")
    want = exact.lora(q)
    live = q["ids"] >= 0
    assert live.any() and torch.equal(want[~live], q["R"][~live])
    for span in exact.spans(k):
        assert ((exact.lora(q, span) != want).any(dim=1) == live).all(), span


@pytest.mark.parametrize("k,r", LORA)
def test_the_adapters_exact_result_is_the_definitions(k, r):
    q = exact.lora_problem(20, 40, k, r, 3, k + r, "cpu")
    want, tol = more_ref.lora(q["X"], q["A"], q["B"], q["ids"], q["scale"], q["R"])
    assert torch.equal(want.float().to(torch.bfloat16), exact.lora(q))


def outside(got, want, tol):
    """The tokens of which a value is out of tolerance."""
    return ((got - want).abs() > tol).any(dim=1)


@pytest.mark.parametrize("d,inner", MOE)
def test_a_step_of_the_experts_that_is_left_out_is_out_of_tolerance(d, inner):
    q = exact.moe_problem(3, d, inner, 4, d + inner, "cpu")
    ids, weights = more_ref.routing(q["X"], q["router"], 2, True)
    want, tol = exact.moe(q, ids, weights)
    assert outside(q["R"].double(), want, tol).all() and outside(exact.moe(q, ids.flip(1), weights)[0], want, tol).all()
    assert outside(exact.moe(q, (ids + 1) % 4, weights)[0], want, tol).all()  # the neighbour's matrices
    for span in exact.spans(d):
        assert outside(exact.moe(q, ids, weights, without=span)[0], want, tol).all(), span
        assert outside(exact.moe(q, ids, weights, without=span, only_gate=True)[0], want, tol).any(), span
    for span in exact.spans(inner):
        assert outside(exact.moe(q, ids, weights, without_inner=span)[0], want, tol).any(), span


@pytest.mark.parametrize("d,inner", MOE)
def test_the_experts_exact_result_is_the_definitions(d, inner):
    q = exact.moe_problem(3, d, inner, 4, d + inner, "cpu")
    ids, weights = more_ref.routing(q["X"], q["router"], 2, False)
    got, tol = exact.moe(q, ids, weights)
    want, loose = more_ref.moe(q["X"], q["W1"], q["W3"], q["W2"], q["R"], ids, weights)
    assert (got - want).abs().max() < 1e-12 * want.abs().max() and (tol < loose + 1e-9).all()
