"""Adapters whose rank is no multiple of eight, on the CPU: rows of B that begin on 16 bytes are what the C ABI takes."""
import pytest

from tests.test_more_abi import GB_ERR_UNSUPPORTED, L, lora  # noqa: F401  (L: the library, a fixture)


@pytest.mark.parametrize("r", [1, 2, 4, 12, 20])
def test_rows_of_b_without_gaps_are_refused(L, r):  # noqa: F811
    assert lora(L, r=r, ldb=r, aa=-(-r // 8) * 512, ab=32 * -(-r // 8) * 8) == GB_ERR_UNSUPPORTED
    assert "B: base address and rows" in L.gb_last_error().decode()
