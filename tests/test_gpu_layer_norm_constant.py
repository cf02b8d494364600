"""Rows of one value: nothing is left of them but the bias, whatever the value and the width."""
import pytest
import torch

import dense_bf16_gemm_persistent_gb300 as gb

pytestmark = pytest.mark.gpu

DEV, BF16 = "cuda", torch.bfloat16


@pytest.mark.parametrize("d", [1, 7, 33, 100, 777, 1000, 4096, 4099, 10000, 12288, 16383, 16384])
def test_a_row_of_one_value_gives_the_bias(d):
    """A sum of up to 2^14 equal values of 8 bits is exact, so that its mean is the value."""
    values = torch.tensor([3.0, 1000.0, -30000.0, 0.7109375, 1e-3, 255.0, -1e20, 0.0]).to(BF16).to(DEV)
    x = values[:, None].expand(-1, d).contiguous()
    w = torch.full((d,), 1.5, dtype=BF16, device=DEV)
    b = torch.randn(d, generator=torch.Generator(device=DEV).manual_seed(d), device=DEV).to(BF16)
    y, _, mean, rstd = gb.add_layer_norm(x, w, b)
    assert torch.equal(mean, values.float())
    assert torch.equal(y, b.expand_as(y))
    # 1 / sqrt(eps): the root and the quotient are rounded, and eps was
    assert ((rstd.double() - 1e-5 ** -0.5).abs() <= 4 * 2.0 ** -24 * 1e-5 ** -0.5).all()
