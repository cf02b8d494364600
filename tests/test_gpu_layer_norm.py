"""Layer norm and its gradient on the GPU against their definitions in 64 bits, at the sizes, layouts and values
where they can go wrong.  Tolerances come from the arithmetic (more_ref.py)."""
import pytest
import torch

import dense_bf16_gemm_persistent_gb300 as gb
from tests import block_ref as ref
from tests import more_ref
from tests.block_ref import HALF_BF16, TINY, assert_within

pytestmark = pytest.mark.gpu

DEV, BF16 = "cuda", torch.bfloat16


def normal(*shape, seed, std=1.0, shift=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * std + shift).to(BF16)


def padded(t, extra, offset=0):
    """The same values in a buffer with `extra` more columns a row, `offset` elements after its start."""
    rows, cols = t.shape
    buf = torch.full((rows * (cols + extra) + offset + 8,), 7.0, dtype=t.dtype, device=t.device)
    view = buf[offset:offset + rows * (cols + extra)].view(rows, cols + extra)[:, :cols]
    view.copy_(t)
    return view


def check_forward(x, w, b, r, eps=1e-5, p=0.0, seed=3, offset=5, **kw):
    y, h, mean, rstd = gb.add_layer_norm(x, w, b, r, eps=eps, p=p, seed=seed, offset=offset, **kw)
    want = more_ref.layer_norm(x, r, w, b, eps, p, seed, offset)
    for name, got in (("y", y), ("h", h), ("mean", mean), ("rstd", rstd)):
        assert_within(got, *want[name], name)
    return y, h, mean, rstd


def check_backward(dy, h, w, mean, rstd, dh, p=0.0, seed=3, offset=5, **kw):
    dx, dr, dw, db = gb.add_layer_norm_backward(dy, h, w, mean, rstd, dH=dh, p=p, seed=seed, offset=offset, **kw)
    want_r, want_w, want_b = more_ref.layer_norm_gradient(dy, h, w, mean, rstd, dh)
    e_r, e_w, e_b = more_ref.layer_norm_gradient_tolerances(dy, h, w, mean, rstd, dh, want_r)
    assert_within(dr, want_r, HALF_BF16 * want_r.abs() + e_r * (1 + HALF_BF16) + TINY, "dR")
    want_x = ref.dropped(want_r, p, seed, offset)
    e_x = e_r / (1 - p) + 4 * more_ref.U * want_x.abs()
    assert_within(dx, want_x, HALF_BF16 * want_x.abs() + e_x * (1 + HALF_BF16) + TINY, "dX")
    assert_within(dw, want_w, e_w, "dweight")
    assert_within(db, want_b, e_b, "dbias")
    return dx, dr, dw, db


SIZES = [(1, 1), (1, 7), (3, 8), (2, 9), (5, 64), (17, 129), (9, 512), (3, 513), (40, 777), (1, 4096), (33, 4096),
         (700, 1000), (3, 4099), (2, 8192), (2, 8193), (5, 12288), (3, 16383), (9, 16384), (2000, 64), (5000, 33)]


@pytest.mark.parametrize("m,d", SIZES)
@pytest.mark.parametrize("residual,bias", [(True, True), (False, False)])
def test_forward_sizes(m, d, residual, bias):
    x = normal(m, d, seed=m + d)
    r = normal(m, d, seed=m + d + 1, shift=0.5) if residual else None
    w, b = normal(d, seed=2, std=0.3, shift=1.0), normal(d, seed=3) if bias else None
    _, h, _, _ = check_forward(x, w, b, r)
    assert residual or h is x


@pytest.mark.parametrize("m,d", SIZES)
def test_backward_sizes(m, d):
    h = normal(m, d, seed=m + d, shift=0.3)
    w = normal(d, seed=2, std=0.3, shift=1.0)
    _, _, mean, rstd = gb.add_layer_norm(h, w)
    check_backward(normal(m, d, seed=4), h, w, mean, rstd, normal(m, d, seed=5) if m % 2 else None)


@pytest.mark.parametrize("p", [0.1, 0.5])
@pytest.mark.parametrize("m,d", [(3, 40), (65, 4096), (7, 1001), (3, 16384)])
def test_dropout_in_both_passes(m, d, p):
    x, r = normal(m, d, seed=1), normal(m, d, seed=2)
    w, b = normal(d, seed=3, shift=1.0), normal(d, seed=4)
    state = torch.tensor([3, 5], dtype=torch.int64, device=DEV)
    y, h, mean, rstd = check_forward(x, w, b, r, p=p)
    for a, c in zip((y, h, mean, rstd), gb.add_layer_norm(x, w, b, r, p=p, seed=state)):
        assert torch.equal(a, c)
    dy, dh = normal(m, d, seed=5), normal(m, d, seed=6)
    got = check_backward(dy, h, w, mean, rstd, dh, p=p)
    for a, c in zip(got, gb.add_layer_norm_backward(dy, h, w, mean, rstd, dH=dh, p=p, seed=state)):
        assert torch.equal(a, c)


@pytest.mark.parametrize("extra,offset", [(8, 0), (3, 0), (0, 1), (5, 3), (1, 7)])
@pytest.mark.parametrize("m,d", [(6, 96), (19, 1000), (5, 4097)])
def test_strides_and_offsets(m, d, extra, offset):
    x, r = padded(normal(m, d, seed=1), extra, offset), padded(normal(m, d, seed=2), extra, offset)
    w, b = padded(normal(1, d, seed=3, shift=1.0), 0, offset)[0], padded(normal(1, d, seed=4), 0, 1)[0]
    y, h, mean, rstd = check_forward(x, w, b, r)
    check_backward(padded(normal(m, d, seed=5), extra, offset), padded(h, extra, offset), w, mean, rstd,
                   padded(normal(m, d, seed=6), 2 * extra, offset))


def test_outputs_that_are_given_are_written_within_their_rows():
    m, d = 13, 203
    out, h = (torch.full((m, d + 5), 9.0, dtype=BF16, device=DEV) for _ in range(2))
    x, r, w = normal(m, d, seed=1), normal(m, d, seed=2), normal(d, seed=3)
    check_forward(x, w, None, r, out=out[:, :d], h=h[:, :d])
    assert (out[:, d:] == 9.0).all() and (h[:, d:] == 9.0).all()
    here = r.clone()  # the residual stream in its own place
    check = gb.add_layer_norm(x, w, None, r)
    got = gb.add_layer_norm(x, w, None, here, h=here)
    assert torch.equal(here, check[1]) and torch.equal(got[0], check[0])


@pytest.mark.parametrize("d", [64, 4096, 10000])
def test_a_mean_far_from_zero_costs_no_bits(d):
    """The mean is 4096 times the deviation: a difference of sums of squares would leave nothing of it."""
    x = normal(6, d, seed=1, std=0.25) + torch.full((6, 1), 64.0, device=DEV, dtype=BF16)  # (steps of a half)
    w = torch.ones(d, device=DEV, dtype=BF16)
    r = torch.full((6, d), 1024.0, device=DEV, dtype=BF16)
    check_forward(x.to(BF16), w, None, r)
    check_forward(torch.full((2, d), 3.0, dtype=BF16, device=DEV), w, None, None)  # no deviation at all: zeros


def test_infinities_and_nan_stay_in_their_rows():
    m, d = 9, 520
    x, w, b = normal(m, d, seed=1), normal(d, seed=2), normal(d, seed=3)
    x[2, 5], x[4, 500], x[7, 0] = float("nan"), float("inf"), -float("inf")
    y, h, mean, rstd = gb.add_layer_norm(x, w, b)
    good = [0, 1, 3, 5, 6, 8]
    want = more_ref.layer_norm(x[good], None, w, b, 1e-5)
    assert_within(y[good], *want["y"])
    assert torch.isnan(y[[2, 4, 7]]).all() and torch.isnan(rstd[[2, 4, 7]]).all()
    dy = normal(m, d, seed=4)
    dx, dr, dw, db = gb.add_layer_norm_backward(dy, h, w, mean, rstd)
    assert torch.isnan(dr[[2, 4, 7]]).all() and torch.isfinite(dr[good].float()).all() and torch.isfinite(db).all()


def test_the_largest_values_and_a_row_of_zeros():
    x = torch.zeros((4, 300), dtype=BF16, device=DEV)
    x[1, ::2], x[2], x[3, 7] = 1e30, 1e-30, 1.0
    w, b = normal(300, seed=1), normal(300, seed=2)
    y, _, mean, rstd = gb.add_layer_norm(x, w, b, eps=1e-5)
    assert torch.equal(y[0], b) and torch.equal(y[1], b) and rstd[1] == 0  # (1e60 passes fp32's range)
    want = more_ref.layer_norm(x[2:], None, w, b, 1e-5)
    assert_within(y[2:], *want["y"])


def test_no_rows():
    w = normal(40, seed=1)
    x = torch.empty((0, 40), dtype=BF16, device=DEV)
    y, h, mean, rstd = gb.add_layer_norm(x, w, w)
    assert y.shape == (0, 40) and mean.shape == rstd.shape == (0,)
    dx, dr, dw, db = gb.add_layer_norm_backward(x, x, w, mean, rstd)
    assert dx.shape == (0, 40) and not dw.any() and not db.any() and dw.shape == db.shape == (40,)


def test_results_repeat_also_in_a_graph_on_another_stream():
    m, d = 300, 1031
    x, r, w, b = normal(m, d, seed=1), normal(m, d, seed=2), normal(d, seed=3), normal(d, seed=4)
    dy = normal(m, d, seed=5)

    def both():
        y, h, mean, rstd = gb.add_layer_norm(x, w, b, r, p=0.2, seed=9)
        return (y, h, mean, rstd, *gb.add_layer_norm_backward(dy, h, w, mean, rstd, dH=dy, p=0.2, seed=9))
    first = [t.clone() for t in both()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = both()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b_, c in zip(first, again, captured):
        assert torch.equal(a, b_) and torch.equal(a, c)
    side.synchronize()
    y = gb.add_layer_norm(x, w, b, r, p=0.2, seed=9, stream=side)[0]
    side.synchronize()
    assert torch.equal(y, first[0])


def test_the_workspace_is_checked_and_any_contents_do():
    m, d = 77, 640
    h, w, dy = normal(m, d, seed=1), normal(d, seed=2), normal(m, d, seed=3)
    _, _, mean, rstd = gb.add_layer_norm(h, w)
    need = gb.add_layer_norm_backward_workspace_bytes(m, d)
    check_backward(dy, h, w, mean, rstd, None, workspace=torch.full((need,), 255, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="workspace"):
        gb.add_layer_norm_backward(dy, h, w, mean, rstd, workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("m,d", [(9, 64), (20, 4096), (3, 16384), (40, 4099)])
def test_a_workspace_that_begins_anywhere_is_refused_or_does(m, d):
    h, w, dy = normal(m, d, seed=1), normal(d, seed=2), normal(m, d, seed=3)
    _, _, mean, rstd = gb.add_layer_norm(h, w)
    need = gb.add_layer_norm_backward_workspace_bytes(m, d)
    room = torch.empty(need + 16, dtype=torch.uint8, device=DEV)
    check_backward(dy, h, w, mean, rstd, None, workspace=room[16:])
    with pytest.raises(gb.GBError, match="16-byte"):
        check_backward(dy, h, w, mean, rstd, None, workspace=room[4:])


@pytest.mark.parametrize("m,d", [(700, 600), (700, 4099), (1300, 1031), (40, 16383)])
def test_many_blocks_with_shifts_of_their_own(m, d):
    """The gradients' parts lie as each block's rows do."""
    h, w, dy = padded(normal(m, d, seed=1), 5, 3), normal(d, seed=2), padded(normal(m, d, seed=3), 5, 3)
    _, _, mean, rstd = gb.add_layer_norm(h, w)
    check_backward(dy, h, w, mean, rstd, padded(normal(m, d, seed=4), 5, 3))


def test_wrong_tensors_are_refused():
    x, w = normal(4, 64, seed=1), normal(64, seed=2)
    f = torch.ones(4, device=DEV)
    for call, error, what in (
            (lambda: gb.add_layer_norm(x.float(), w), TypeError, "X"),
            (lambda: gb.add_layer_norm(x, w[:32]), ValueError, "weight"),
            (lambda: gb.add_layer_norm(x, w, w.float()), TypeError, "bias"),
            (lambda: gb.add_layer_norm(x, w, None, x[:2]), ValueError, "R"),
            (lambda: gb.add_layer_norm(x.t(), w[:4]), ValueError, "X"),
            (lambda: gb.add_layer_norm(x, w, eps=float("nan")), gb.GBError, "eps"),
            (lambda: gb.add_layer_norm(x, w, p=1.5), gb.GBError, "probability"),
            (lambda: gb.add_layer_norm(normal(1, 16385, seed=1), normal(16385, seed=1)), gb.GBError, "16384"),
            (lambda: gb.add_layer_norm_backward(x, x, w, f[:2], f), ValueError, "mean"),
            (lambda: gb.add_layer_norm_backward(x, x, w, f, f.double()), TypeError, "rstd")):
        with pytest.raises(error, match=what):
            call()
