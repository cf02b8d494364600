"""Calls around the products that were once answered wrongly, refused or unsafe, each against its definition in
64 bits (block_ref.py)."""
import pytest
import torch

import dense_bf16_gemm_persistent_gb300 as gb
from tests import block_ref as ref
from tests.block_ref import HALF_BF16, TINY, assert_within
from tests.test_gpu_block import BF16, DEV, check_linear_result, normal, w4_input, w4_weights

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------------- scales of 8-bit rows

def test_w4_row_scales_in_one_dimension():
    """[M] scales, contiguous and with a stride, are the [M,1] ones."""
    m, n, k, group = 9, 70, 288, 64
    q, s, z = w4_weights(n, k, group, True, 1)
    x, xs = w4_input(m, k, "row", 2)
    xs = xs * torch.arange(1, m + 1, device=DEV)[:, None]  # (each row's own)
    want = gb.linear_w4(x, q, s, zeros=z, group=group, x_scale=xs)
    check_linear_result(want, x, xs, q, s, z, None, None, "none", group)
    apart = torch.full((m, 3), float("nan"), device=DEV)
    apart[:, 1] = xs[:, 0]
    for scale in (xs[:, 0], xs.reshape(m).clone(), apart[:, 1]):
        assert scale.dim() == 1
        assert torch.equal(gb.linear_w4(x, q, s, zeros=z, group=group, x_scale=scale), want)
    one = gb.linear_w4(x[:1], q, s, zeros=z, group=group, x_scale=xs[0].expand(1))
    assert torch.equal(one, gb.linear_w4(x[:1], q, s, zeros=z, group=group, x_scale=xs[:1]))


def test_w4_refuses_a_scale_expanded_over_the_rows():
    """One element of storage for all rows: no row but the first has a scale in memory."""
    m, k = 4, 64
    q, s, z = w4_weights(8, k, 64, False, 1)
    x, xs = w4_input(m, k, "row", 2)
    for scale in (xs[0].expand(m), xs[:1].expand(m, 1)):
        with pytest.raises((ValueError, gb.GBError), match="x_scale|ldxs"):
            gb.linear_w4(x, q, s, group=64, x_scale=scale)
        with pytest.raises((ValueError, gb.GBError), match="x_scale|ldxs"):
            gb.ffn_gated_w4(x, q, s, q, s, group=64, x_scale=scale)
