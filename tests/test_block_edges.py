"""Calls around the products that were once accepted or answered wrongly, as far as the CPU shows it."""
import ctypes
from concurrent.futures import ThreadPoolExecutor

import pytest

from tests.test_block_abi import GB_ERR_UNSUPPORTED, GB_OK, L, bwd, drop, norm, norm_q8, w4  # noqa: F401


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


def test_a_call_without_work_says_so_in_its_plan(L):  # noqa: F811
    def after(call):  # (in a thread of its own: the plan is the calling thread's)
        def run():
            buf = ctypes.create_string_buffer(256)
            assert call() == GB_OK and L.gb_last_plan(buf, 256) == GB_OK
            return buf.value.decode()
        with ThreadPoolExecutor(1) as pool:
            return pool.submit(run).result()
    for call in (lambda: w4(L, X=None, W=None, s=None, D=None, M=0), lambda: drop(L, X=None, D=None, N=0),
                 lambda: norm(L, X=None, Y=None, w=None, M=0), lambda: norm_q8(L, X=None, Q=None, scale=None, D=0),
                 lambda: bwd(L, dY=None, H=None, w=None, rstd=None, dR=None, dw=None, D=0)):
        assert after(call) == "empty (no launch)"


def test_binding_is_compiled_again_for_another_torch(tmp_path, monkeypatch):
    """Its source is older than it, but what it was compiled for is not what is installed."""
    from dense_bf16_gemm_persistent_gb300 import _build
    made = []

    class Done:
        returncode, stderr = 0, ""

    def compiler(command, **kwargs):
        made.append(command)
        open(command[command.index("-o") + 1], "w").close()
        return Done
    monkeypatch.setattr(_build, "BINDING", str(tmp_path / "binding.so"))
    monkeypatch.setattr(_build, "LOG_DIR", str(tmp_path / "log"))
    monkeypatch.setattr(_build.subprocess, "run", compiler)
    for expected in (1, 1):  # (the second time there is nothing to do)
        _build.build_binding()
        assert len(made) == expected
    monkeypatch.setattr("torch.__version__", "0.0")
    _build.build_binding()
    assert len(made) == 2
    monkeypatch.setenv("CXX", "another-compiler")
    _build.build_binding()
    assert len(made) == 3 and made[-1][0] == "another-compiler"
