"""The layer norm's outputs in the places of its inputs, where the header allows it: the same bits as elsewhere."""
import pytest
import torch

import dense_bf16_gemm_persistent_gb300 as gb

pytestmark = pytest.mark.gpu

DEV, BF16 = "cuda", torch.bfloat16
SIZES = [(1, 4096), (3, 7), (33, 4096), (19, 1000), (700, 1031), (40, 4099), (9, 16384), (7, 16383), (2000, 64), (1300, 33)]
LAYOUTS = [(0, 0), (5, 3), (8, 0)]  # columns between rows, elements before the first


class Matrix:
    """m rows of d columns in a buffer that has more columns and begins elsewhere."""

    def __init__(self, values, extra, offset):
        m, d = values.shape
        self.room = torch.full((offset + m * (d + extra) + 8,), 9.0, dtype=BF16, device=DEV)
        self.all = self.room[offset:offset + m * (d + extra)].view(m, d + extra)
        self.rows, self.rest = self.all[:, :d], self.all[:, d:]
        self.rows.copy_(values)
        self.arg = (self.rows.data_ptr(), d + extra)


def normal(*shape, seed, shift=0.0):
    return (torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV) + shift).to(BF16)


def run(status):
    assert status == 0, gb.lib().gb_last_error().decode()


@pytest.mark.parametrize("m,d", SIZES)
@pytest.mark.parametrize("extra,offset", LAYOUTS)
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_forward(m, d, extra, offset, p):
    x, r, w, b = normal(m, d, seed=1), normal(m, d, seed=2, shift=0.5), normal(d, seed=3, shift=1.0), normal(d, seed=4)
    stream = torch.cuda.current_stream().cuda_stream

    def call(y, h):
        """Y and H in the place of X, of R, or in their own."""
        at = {"x": Matrix(x, extra, offset), "r": Matrix(r, extra, offset)}
        for name in (y, h):
            at.setdefault(name, Matrix(torch.zeros_like(x), extra, offset))
        stats = torch.empty((2, m), device=DEV)
        run(gb.lib().gb_add_layer_norm(*at["x"].arg, *at["r"].arg, w.data_ptr(), b.data_ptr(), 1e-5, p, 7, 11, None, *at[h].arg,
                                       *at[y].arg, stats[0].data_ptr(), stats[1].data_ptr(), m, d, stream))
        assert all((a.rest == 9).all() and (a.room[:offset] == 9).all() and (a.room[-8:] == 9).all() for a in at.values())
        for name, was in (("x", x), ("r", r)):
            assert name in (y, h) or torch.equal(at[name].rows, was)
        return at[y].rows, at[h].rows, stats
    want = call("y", "h")
    for y, h in (("x", "h"), ("r", "h"), ("y", "x"), ("y", "r"), ("x", "r"), ("r", "x")):
        for a, c in zip(call(y, h), want):
            assert torch.equal(a, c), (y, h)


@pytest.mark.parametrize("m,d", SIZES)
@pytest.mark.parametrize("extra,offset", LAYOUTS)
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_backward(m, d, extra, offset, p):
    dy, h, dh, w = normal(m, d, seed=1), normal(m, d, seed=2, shift=0.5), normal(m, d, seed=5), normal(d, seed=3, shift=1.0)
    _, _, mean, rstd = gb.add_layer_norm(h, w)
    need = gb.add_layer_norm_backward_workspace_bytes(m, d)
    stream = torch.cuda.current_stream().cuda_stream

    def call(dr):
        """dR in the place of dY, of dH, or in its own."""
        at = {"dy": Matrix(dy, extra, offset), "dh": Matrix(dh, extra, offset), "h": Matrix(h, extra, offset),
              "dx": Matrix(torch.zeros_like(h), extra, offset)}
        at.setdefault(dr, Matrix(torch.zeros_like(h), extra, offset))
        sums = torch.empty((2, d), device=DEV)
        workspace = torch.empty(need, dtype=torch.uint8, device=DEV)
        run(gb.lib().gb_add_layer_norm_backward(*at["dy"].arg, *at["h"].arg, w.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                                                *at["dh"].arg, p, 7, 11, None, *at[dr].arg, *at["dx"].arg, sums[0].data_ptr(),
                                                sums[1].data_ptr(), workspace.data_ptr(), need, m, d, stream))
        assert all((a.rest == 9).all() and (a.room[:offset] == 9).all() and (a.room[-8:] == 9).all() for a in at.values())
        for name, was in (("dy", dy), ("dh", dh), ("h", h)):
            assert name == dr or torch.equal(at[name].rows, was)
        return at[dr].rows, at["dx"].rows, sums
    want = call("dr")
    for dr in ("dy", "dh"):
        for a, c in zip(call(dr), want):
            assert torch.equal(a, c), dr
