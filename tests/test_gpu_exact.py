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
