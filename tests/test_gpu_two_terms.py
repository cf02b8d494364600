"""What the two bf16 terms keep that stand between two products."""
import pytest
import torch

import dense_bf16_gemm_persistent_gb300 as gb
from tests.block_ref import HALF_BF16

pytestmark = pytest.mark.gpu

DEV, BF16 = "cuda", torch.bfloat16


@pytest.mark.parametrize("m", [1, 50])
def test_seventeen_bits_between_the_adapters_products(m):
    """(v) - (v - 1) for v of 17 bits: X's powers of two and A's bits make them, B takes one from the other."""
    v = torch.randint(2 ** 15, 2 ** 16, (300,), generator=torch.Generator().manual_seed(1)) * 2 + 1
    bits = lambda u: (u[:, None] >> torch.arange(24) & 1).to(BF16)  # noqa: E731
    a = torch.stack([bits(v), bits(v - 1)], dim=1).to(DEV)
    x = (2.0 ** torch.arange(24)).to(BF16).to(DEV).expand(m, 24).contiguous()
    b = torch.zeros((300, 16, 8), dtype=BF16, device=DEV)[:, :, :2]
    b[:, :, 0], b[:, :, 1] = 1.0, -1.0
    for first in range(0, 300, m):
        ids = (torch.arange(m, device=DEV) + first).to(torch.int32)
        assert (gb.lora(x, a, b, ids)[ids < 300] == 1).all()


def test_the_largest_values_between_two_products_stay_finite():
    """What rounds up past bf16's largest value is cut off instead: its two terms are its value to 2^-16."""
    top = 3.4e38  # (bf16's largest is 3.3895e38)
    a = torch.zeros((1, 1, 8), dtype=BF16, device=DEV)
    a[0, 0, :2] = torch.tensor([3.3895e38, 2.0 ** 118])
    low = a.double().sum().item()
    assert 3.3895e38 < low < top
    b = torch.full((1, 4, 8), 2.0 ** -30, dtype=BF16, device=DEV)[:, :, :1]
    d = gb.lora(torch.ones((2, 8), dtype=BF16, device=DEV), a, b, torch.zeros(2, dtype=torch.int32, device=DEV))
    assert ((d.double() - low * 2.0 ** -30).abs() <= HALF_BF16 * low * 2.0 ** -30).all()
