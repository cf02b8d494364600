"""Sums on the tensor cores over thousands of terms of one sign, on whole numbers (times powers of two) whose result is known.
R takes the result away, so that D shows the error and not its own rounding.  127 times 129 is 2^14 - 1: what an adder cuts
off of a sum of such products is nearly a whole unit each time."""
import pytest
import torch

import dense_bf16_gemm_persistent_gb300 as gb
from tests.block_ref import HALF_BF16

pytestmark = pytest.mark.gpu

DEV, BF16 = "cuda", torch.bfloat16

# An mma's adder may cut off what is below its sum: 2^-23 of it each time, always towards zero.  A chain of 64 of them, the
# fp32 sums of up to 256 chains, and of the 64 warps' parts that a result has at most.  (Of the adapters 32 chains, and 32
# mma of the second product.)
SUM = 64 * 2.0 ** -23 + (256 + 64) * 2.0 ** -24
TERMS = 2.0 ** -17 + 2.0 ** -23  # two bf16 terms, each rounded to nearest


def error(d, want, r):
    """The largest error of D - R as a share of `want`; D's own rounding counted in is at most (what R leaves) 2^-8."""
    left = want + r.double()
    assert (left.abs() <= HALF_BF16 * abs(want)).all()
    return ((d.double() - left).abs() / abs(want)).max().item() - HALF_BF16 * (left.abs() / abs(want)).max().item()


@pytest.mark.parametrize("t", [1, 9, 32])
def test_experts_of_a_long_inner_dimension(t):
    """D = 14336 times 45045 from each of eight experts: a warp's part of the second products is a whole expert's."""
    d, inner, experts = 2560, 14336, 8
    w1, w3 = (torch.zeros((experts, inner, d), dtype=BF16, device=DEV) for _ in range(2))
    w1[:, :, :45] = 1.0                           # silu(45) is 45 to 2^-60
    w3[:, :, 100:115], w3[:, :, 120] = 64.0, 41.0  # 1001
    want = inner * 45045.0
    r = torch.full((t, d), -want, device=DEV).to(BF16)
    out, _, weights = gb.moe_ffn_gated(torch.ones((t, d), dtype=BF16, device=DEV), torch.zeros((experts, d), dtype=BF16, device=DEV),
                                       w1, w3, torch.ones((experts, d, inner), dtype=BF16, device=DEV), experts, R=r)
    assert (weights == 1 / 8).all()
    # (the activation to 2^-20; 45045 has 16 bits)
    assert error(out, want, r) <= SUM + 2.0 ** -20


@pytest.mark.parametrize("t", [1, 9, 32])
def test_experts_of_long_rows(t):
    d, inner = 262144, 16
    x, w = torch.full((t, d), 127 / 128, device=DEV).to(BF16), torch.full((1, inner, d), 129 / 512, device=DEV).to(BF16)
    w2 = torch.zeros((1, d, inner), dtype=BF16, device=DEV)
    w2[:, :, 3] = 1.0
    want = (d * (127 / 128) * (129 / 512)) ** 2
    r = torch.full((t, d), -want, device=DEV).to(BF16)
    out, _, _ = gb.moe_ffn_gated(x, torch.zeros((1, d), dtype=BF16, device=DEV), w, w, w2, 1, R=r)
    assert error(out, want, r) <= 2 * SUM + TERMS + 2.0 ** -20


@pytest.mark.parametrize("m,r", [(8192, 256), (8192, 16), (16, 64)])
def test_adapters_of_long_rows(m, r):
    """With 256 ranks and a tile for each CTA a warp has all of a row's columns."""
    k, n = 32768, 40
    x, a = torch.full((m, k), 127 / 128, device=DEV).to(BF16), torch.full((1, r, k), 129 / 128, device=DEV).to(BF16)
    b = torch.zeros((1, n, r), dtype=BF16, device=DEV)
    b[:, torch.arange(n), torch.arange(n) % r] = 1.0
    want = k * (127 / 128) * (129 / 128)
    residual = torch.full((m, n), -want, device=DEV).to(BF16)
    out = gb.lora(x, a, b, torch.zeros(m, dtype=torch.int32, device=DEV), R=residual)
    assert error(out, want, residual) <= SUM + TERMS
