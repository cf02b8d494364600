"""Calls around the products that were once accepted or answered wrongly, as far as the CPU shows it."""
import pytest

from tests.test_block_abi import GB_ERR_UNSUPPORTED, L, drop  # noqa: F401


@pytest.mark.parametrize("n", [(1 << 31) - 15, (1 << 31) - 8, (1 << 31) - 1])
def test_dropout_refuses_rows_whose_last_chunk_ends_past_32_bits(L, n):  # noqa: F811
    """A chunk's first column + 8 has to be a signed 32-bit number: above, the last one would be moved as a whole
    word past the row's end."""
    assert drop(L, N=n, ldx=n, ldd=n) == GB_ERR_UNSUPPORTED
    assert "2^31 - 16" in L.gb_last_error().decode()
    assert drop(L, X=None, D=None, N=n, M=0) == GB_ERR_UNSUPPORTED


def test_last_chunks_columns_are_32_bit_numbers():
    """The row kernels' index arithmetic at the largest width, for every shift of a row."""
    cols = (1 << 31) - 16
    for shift in range(8):
        chunks = -(-(cols + (7 if shift else 0)) // 8)
        for j in (0, 1, chunks - 2, chunks - 1):
            assert 8 * j < 1 << 31 and 8 * j - shift + 8 < 1 << 31
