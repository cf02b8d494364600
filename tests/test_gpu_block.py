"""The operators around the products on the GPU against their definitions in 64 bits: 4-bit
layers for a few tokens, the norm and its gradient, dropout; at the sizes, layouts and values
where they can go wrong.  Tolerances come from the arithmetic (block_ref.py)."""
import numpy as np
import pytest
import torch

import dense_bf16_gemm_persistent_gb300 as gb
from tests import block_ref as ref
from tests.block_ref import HALF_BF16, TINY, assert_within

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16 = torch.bfloat16


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(*shape, seed, std=1.0):
    return (torch.randn(shape, generator=gen(seed), device=DEV) * std).to(BF16)


def padded(t, extra, offset=0):
    """The same values in a buffer with `extra` more columns a row, `offset` elements after its start."""
    rows, cols = t.shape
    buf = torch.full((rows * (cols + extra) + offset + 8,), 0, dtype=t.dtype, device=t.device)
    view = buf[offset:offset + rows * (cols + extra)].view(rows, cols + extra)[:, :cols]
    view.copy_(t)
    return view


# ---------------------------------------------------------------------------------- 4-bit layers

def w4_weights(n, k, group, zeros, seed):
    groups = -(-k // group)
    q = torch.randint(0, 256, (n, k // 2), generator=gen(seed), device=DEV).to(torch.uint8)
    s = ((torch.rand((n, groups), generator=gen(seed + 1), device=DEV) + 0.5) * 0.01).to(BF16)
    z = torch.randint(0, 16, (n, groups), generator=gen(seed + 2), device=DEV).to(torch.uint8) if zeros else None
    return q, s, z


def w4_input(m, k, x8, seed):
    x = torch.randn((m, k), generator=gen(seed), device=DEV)
    if x8 == "no":
        return x.to(BF16), None
    width = 128 if x8 == "group" else k
    s = torch.stack([p.abs().amax(dim=1) for p in x.split(width, dim=1)], dim=1) / 448
    return (x / s.repeat_interleave(width, dim=1)[:, :k]).to(torch.float8_e4m3fn), s.contiguous()


def check_linear_w4(m, n, k, group, zeros=False, x8="no", act="none", bias=False, residual=False, seed=0):
    q, s, z = w4_weights(n, k, group, zeros, seed)
    x, xs = w4_input(m, k, x8, seed + 3)
    b = normal(n, seed=seed + 4) if bias else None
    r = normal(m, n, seed=seed + 5) if residual else None
    d = gb.linear_w4(x, q, s, b, r, act=act, zeros=z, group=group, x_scale=xs)
    check_linear_result(d, x, xs, q, s, z, b, r, act, group)
    return d


def check_linear_result(d, x, xs, q, s, z, b, r, act, group, what=""):
    v, off = ref.w4_products(x, xs, ref.unpack_w4(q, s, z, group, x.shape[1]))
    if b is not None:
        v = v + b.double()
    want = ref.act(v, act)
    # the activations' slopes are at most 1.13; they are computed to 2^-20 of their argument
    tol = 1.13 * (off + 2.0 ** -23 * v.abs()) + (2.0 ** -20 * v.abs() if act in ("gelu_tanh", "silu") else 0)
    if r is not None:
        want = want + r.double()
    assert_within(d, want, tol + (HALF_BF16 + 2.0 ** -23) * want.abs() + HALF_BF16 * tol + TINY, what)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("x8", ["no", "row", "group"])
@pytest.mark.parametrize("m", [1, 5, 8, 9, 17, 32, 33, 70])
def test_linear_w4_tokens(m, x8, group):
    check_linear_w4(m, 144, 1184, group, zeros=True, x8=x8, residual=True, seed=m)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,k", [(1, 32), (7, 64), (16, 96), (17, 128), (33, 160), (96, 480), (96, 512), (100, 544),
                                 (250, 2048), (4099, 4128), (96, 16384), (64, 40000), (3, 65536), (20000, 512)])
def test_linear_w4_sizes(n, k, group):
    check_linear_w4(3, n, k, group, zeros=True, seed=n + k)


@pytest.mark.parametrize("act", ["none", "gelu_tanh", "silu", "relu"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("residual", [False, True])
def test_linear_w4_epilogue(act, bias, residual):
    check_linear_w4(4, 130, 640, 64, act=act, bias=bias, residual=residual, seed=3)


@pytest.mark.parametrize("m,k", [(32, 16384), (32, 65536), (9, 131072)])
def test_linear_w4_long_rows(m, k):
    """x does not fit the shared memory in one slice: split over a cluster, fewer tokens a pass."""
    check_linear_w4(m, 40, k, 128, x8="group", seed=k)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("x8", ["no", "row", "group"])
@pytest.mark.parametrize("m,n,k", [(1, 8, 32), (1, 1000, 1024), (6, 333, 4096), (12, 17, 672), (32, 515, 2208),
                                   (40, 96, 512)])
def test_ffn_gated_w4(m, n, k, x8, group):
    q1, s1, z1 = w4_weights(n, k, group, True, 10 + k)
    q3, s3, _ = w4_weights(n, k, group, False, 20 + k)
    x, xs = w4_input(m, k, x8, m)
    d = gb.ffn_gated_w4(x, q1, s1, q3, s3, zeros1=z1, group=group, x_scale=xs)
    a, off_a = ref.w4_products(x, xs, ref.unpack_w4(q1, s1, z1, group, k))
    b, off_b = ref.w4_products(x, xs, ref.unpack_w4(q3, s3, None, group, k))
    gate = ref.act(a, "silu")
    tol = (1.13 * off_a + 2.0 ** -20 * a.abs()) * (b.abs() + off_b) + gate.abs() * off_b
    assert_within(d, gate * b, tol * (1 + HALF_BF16) + HALF_BF16 * (gate * b).abs() + TINY)


def test_w4_exact_integers():
    """Small integers: every product and sum is exact, so each output is the integer itself."""
    m, n, k = 11, 200, 1120
    q, _, z = w4_weights(n, k, 32, True, 1)
    s = torch.full((n, k // 32), 0.25, dtype=BF16, device=DEV)
    x = torch.randint(-1, 2, (m, k), generator=gen(2), device=DEV).to(BF16)
    v = x.double() @ ref.unpack_w4(q, s, z, 32, k).T
    assert torch.equal(gb.linear_w4(x, q, s, zeros=z, group=32), v.to(torch.float32).to(BF16))


def test_w4_strides_and_outputs_in_place():
    m, n, k, group = 6, 70, 288, 64
    q, s, z = w4_weights(n, k, group, True, 7)
    x, r, b = normal(m, k, seed=8), normal(m, n, seed=9), normal(n, seed=10)
    want = gb.linear_w4(x, q, s, b, r, zeros=z, group=group)
    qp, sp, zp = padded(q, 16, 32), padded(s, 3, 1), padded(z, 5, 3)
    xp, out = padded(x, 7, 3), padded(r, 5, 1)
    got = gb.linear_w4(xp, qp, sp, b, out, zeros=zp, group=group, out=out)
    assert got is out and torch.equal(out, want)
    # the columns next to the output are as they were
    assert out._base[:1].eq(0).all() and (out._base[1:1 + m * (n + 5)].view(m, n + 5)[:, n:] == 0).all()
    x8, xs = w4_input(m, k, "group", 11)
    want = gb.linear_w4(x8, q, s, zeros=z, group=group, x_scale=xs)
    assert torch.equal(gb.linear_w4(padded(x8, 5, 3), qp, sp, zeros=zp, group=group, x_scale=padded(xs, 2, 1)), want)


def test_w4_weights_past_32_bit_offsets():
    """Rows 2 GiB apart: byte offsets of the weights do not fit 32 bits."""
    n, k, ld = 3, 128, (1 << 31) + 64
    buf = torch.empty(2 * ld + k // 2, dtype=torch.uint8, device=DEV)
    wide = buf.as_strided((n, k // 2), (ld, 1))
    q, s, _ = w4_weights(n, k, 128, False, 5)
    wide.copy_(q)
    x = normal(2, k, seed=6)
    assert torch.equal(gb.linear_w4(x, wide, s), gb.linear_w4(x, q, s))


def test_w4_nan_and_infinity_stay_in_their_rows():
    q, s, _ = w4_weights(40, 256, 128, False, 5)
    q[:, 0] = 0x99  # q - 8 = 1 in the first two columns
    x = normal(4, 256, seed=6)
    want = gb.linear_w4(x, q, s)
    x[1, 0], x[2, 1] = float("nan"), float("inf")
    got = gb.linear_w4(x, q, s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[3], want[3])
    assert got[1].isnan().all() and (got[2] == float("inf")).all()


def test_w4_empty():
    q, s, _ = w4_weights(8, 64, 64, False, 1)
    assert gb.linear_w4(torch.empty(0, 64, dtype=BF16, device=DEV), q, s, group=64).shape == (0, 8)
    b, r = normal(8, seed=2), normal(3, 8, seed=3)
    empty = torch.empty(3, 0, dtype=BF16, device=DEV)
    d = gb.linear_w4(empty, torch.empty(8, 0, dtype=torch.uint8, device=DEV), torch.empty(8, 0, dtype=BF16, device=DEV),
                     b, r, act="relu")
    assert torch.equal(d, (b.float().clamp_min(0) + r.float()).to(BF16))


def test_w4_same_bits_on_every_run_and_stream():
    q, s, z = w4_weights(500, 8192, 64, True, 5)
    x = normal(7, 8192, seed=6)
    first = gb.linear_w4(x, q, s, zeros=z, group=64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(first)
    gb.linear_w4(x, q, s, zeros=z, group=64, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, first)
    for _ in range(3):
        assert torch.equal(gb.linear_w4(x, q, s, zeros=z, group=64), first)


# ---------------------------------------------------------------------------------- dropout

def check_dropout(d, x, r, p, seed, offset):
    v = ref.dropped(x, p, seed, offset)
    want = v + r.double() if r is not None else v
    size = v.abs() + (r.double().abs() if r is not None else 0)
    tol = HALF_BF16 * want.abs() + 2.0 ** -22 * size.nan_to_num(0, 0, 0) + TINY
    assert_within(d, want, tol)


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.999, 1.0])
@pytest.mark.parametrize("m,n", [(1, 1), (3, 7), (5, 8), (33, 64), (17, 4099), (200, 1000), (1, 100000)])
def test_dropout(m, n, p):
    x, r = normal(m, n, seed=m), normal(m, n, seed=n)
    check_dropout(gb.dropout(x, p, 123456789012345, 77), x, None, p, 123456789012345, 77)
    check_dropout(gb.dropout(x, p, 5, 1 << 40, R=r), x, r, p, 5, 1 << 40)


@pytest.mark.parametrize("offset", range(8))
def test_dropout_layouts(offset):
    """Rows that start anywhere in a 16-byte word, alike in every matrix or not."""
    x, r = normal(9, 203, seed=1), normal(9, 203, seed=2)
    want = gb.dropout(x, 0.3, 9, 4, R=r)
    for extra in (0, 1, 5, 13):
        alike = padded(torch.zeros_like(x), extra, offset)
        got = gb.dropout(padded(x, extra, offset), 0.3, 9, 4, R=padded(r, extra, offset), out=alike)
        assert torch.equal(got, want)
        assert not alike._base[:offset].any() and not alike._base[offset:][:9 * (203 + extra)].view(9, -1)[:, 203:].any()
        assert torch.equal(gb.dropout(padded(x, extra, offset), 0.3, 9, 4, R=padded(r, 3, 1)), want)


def test_dropout_drops_nan_and_infinity():
    x = normal(64, 96, seed=3)
    keep = ref.keep_mask(64, 96, 0.5, 21, 3).to(DEV)
    x[~keep] = float("nan")
    x[0][~keep[0]] = float("inf")
    check_dropout(gb.dropout(x, 0.5, 21, 3), torch.where(keep, x, torch.zeros_like(x)), None, 0.5, 21, 3)


def test_dropout_gradient_is_the_same_call():
    """<dropout(x), dy> = <x, dropout(dy)> element by element: the same mask, drawn twice."""
    x, dy = normal(50, 333, seed=1).abs() + 1, normal(50, 333, seed=2).abs() + 1
    assert torch.equal(gb.dropout(x, 0.4, 8, 2) != 0, gb.dropout(dy, 0.4, 8, 2) != 0)
    assert not torch.equal(gb.dropout(x, 0.4, 8, 2), gb.dropout(x, 0.4, 8, 3))
    assert not torch.equal(gb.dropout(x, 0.4, 8, 2), gb.dropout(x, 0.4, 9, 2))


def test_dropout_in_place_and_rows_past_32_bit_offsets():
    x = normal(3, 100, seed=1)
    want = gb.dropout(x, 0.2, 6, 6)
    y = x.clone()
    assert gb.dropout(y, 0.2, 6, 6, out=y) is y and torch.equal(y, want)
    y = x.clone()
    gb.dropout(x, 0.2, 6, 6, R=y, out=y)
    check_dropout(y, x, x, 0.2, 6, 6)
    far = torch.empty((1 << 32) + 256, dtype=BF16, device=DEV).as_strided((3, 100), ((1 << 31) + 8, 1))
    far.copy_(x)
    assert torch.equal(gb.dropout(far, 0.2, 6, 6), want)


def test_dropout_seed_read_when_a_graph_runs():
    x = normal(40, 88, seed=1)
    state = torch.tensor([11, 0], dtype=torch.int64, device=DEV)
    out = gb.dropout(x, 0.5, state)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gb.dropout(x, 0.5, state, out=out)
    for offset in (3, 4):
        state[1] = offset
        graph.replay()
        assert torch.equal(out, gb.dropout(x, 0.5, 11, offset))


# ---------------------------------------------------------------------------------- norm

def norm_reference(x, r, w, eps, p, seed, offset):
    h = ref.dropped(x, p, seed, offset)
    size = h.abs()
    if r is not None:
        h, size = h + r.double(), size + r.double().abs()
    rstd = (h.square().mean(dim=1) + eps).rsqrt()
    y = h * rstd[:, None] * w.double()
    # h: a product and a sum (2^-22 of their sizes, which rstd takes over); the sum of squares 64 terms deep at
    # most in any thread and join; a few roundings more
    slack = 2.0 ** -22 * size * rstd[:, None] * w.double().abs() + 2.0 ** -17 * y.abs()
    return h, size, rstd, y, slack


SIZES = [(1, 1), (2, 7), (3, 8), (9, 64), (33, 255), (8, 256), (5, 512), (7, 1000), (4, 1024), (3, 1025), (6, 1032),
         (5, 2047), (16, 4096), (9, 4099), (2, 8192), (3, 8193), (2, 12288), (1, 16383), (3, 16384)]


@pytest.mark.parametrize("m,d", SIZES)
@pytest.mark.parametrize("p", [0.0, 0.3])
@pytest.mark.parametrize("residual", [False, True])
def test_add_rms_norm(m, d, p, residual):
    x, w = normal(m, d, seed=d), normal(d, seed=d + 1)
    r = normal(m, d, seed=d + 2, std=3.0) if residual else None
    y, h, rstd = gb.add_rms_norm(x, w, r, eps=1e-5, p=p, seed=99, offset=d)
    hw, size, rw, yw, slack = norm_reference(x, r, w, 1e-5, p, 99, d)
    assert_within(h, hw, HALF_BF16 * hw.abs() + 2.0 ** -22 * size + TINY, "H")
    # dropped terms cancel nowhere: rstd moves by the relative error of the squares
    assert_within(rstd, rw, rw * 2.0 ** -17, "rstd")
    assert_within(y, yw, HALF_BF16 * yw.abs() + slack + TINY, "Y")
    if not residual and p == 0:
        assert h is x


@pytest.mark.parametrize("m,d", SIZES)
@pytest.mark.parametrize("group", [0, 128])
def test_add_rms_norm_q8(m, d, group):
    x, w, r = normal(m, d, seed=d), normal(d, seed=d + 1), normal(m, d, seed=d + 2)
    q, scale, h = gb.add_rms_norm_q8(x, w, r, eps=1e-5, scale_group=group)
    hw, size, _, yw, slack = norm_reference(x, r, w, 1e-5, 0.0, 0, 0)
    assert_within(h, hw, HALF_BF16 * hw.abs() + 2.0 ** -22 * size + TINY, "H")
    width = group or d
    top = torch.stack([t.abs().amax(dim=1) for t in yw.split(width, dim=1)], dim=1)
    top_slack = torch.stack([t.amax(dim=1) for t in slack.split(width, dim=1)], dim=1)
    assert scale.shape == top.shape
    assert_within(scale, (top / 448).clamp_min(2.0 ** -126), (top * 2.0 ** -22 + top_slack) / 448, "scale")
    s = scale.double().repeat_interleave(width, dim=1)[:, :d]
    # e4m3: half a unit is 2^-4 of a normal value, 2^-10 of the scale below 2^-6
    assert_within(q.double() * s, yw, (2.0 ** -4 * yw.abs()).clamp_min(2.0 ** -10 * s) + 2 * slack, "Q scale")


@pytest.mark.parametrize("offset", range(8))
@pytest.mark.parametrize("d", [203, 1027])
def test_norm_layouts(d, offset):
    m = 11
    x, r, w = normal(m, d, seed=1), normal(m, d, seed=2), normal(d, seed=3)
    y, h, _ = gb.add_rms_norm(x, w, r, p=0.25, seed=4, offset=1)
    q, scale, _ = gb.add_rms_norm_q8(x, w, r, scale_group=128)
    wide_w = padded(w[None], 0, offset)[0]
    # the order of a row's sum goes with where its words start: 2^-18 of rstd at most, then one rounding each
    near = lambda a, b: assert_within(a, b.double(), 2 * HALF_BF16 * b.double().abs() + TINY)  # noqa: E731
    for extra in (0, 1, 5):
        xs, rs = padded(x, extra, offset), padded(r, extra, offset)
        out, hh = padded(torch.zeros_like(x), extra, offset), padded(torch.zeros_like(x), extra, offset)
        y2, h2, _ = gb.add_rms_norm(xs, wide_w, rs, p=0.25, seed=4, offset=1, out=out, h=hh)
        near(y2, y)
        assert torch.equal(h2, h)
        assert not out._base[:offset].any() and not out._base[offset:][:m * (d + extra)].view(m, -1)[:, d:].any()
        y2, h2, _ = gb.add_rms_norm(xs, wide_w, padded(r, 2, 3), p=0.25, seed=4, offset=1)
        near(y2, y)
        assert torch.equal(h2, h)
        q2, scale2, _ = gb.add_rms_norm_q8(xs, wide_w, rs, scale_group=128,
                                           out=padded(torch.zeros_like(q).view(torch.uint8), extra, offset).view(q.dtype))
        assert_within(scale2, scale.double(), scale.double() * 2.0 ** -17)
        assert_within(q2.float(), q.double(), q.double().abs() * 2.0 ** -3 + 2.0 ** -9)


def test_norm_in_place_on_the_residual_stream():
    x, r, w = normal(20, 1500, seed=1), normal(20, 1500, seed=2), normal(1500, seed=3)
    y, h, _ = gb.add_rms_norm(x, w, r)
    r2, x2 = r.clone(), x.clone()
    y2, h2, _ = gb.add_rms_norm(x2, w, r2, h=r2, out=x2)
    assert h2 is r2 and torch.equal(r2, h) and torch.equal(x2, y)


def test_norm_rows_of_zeros_and_extremes():
    d = 640
    x, w = torch.zeros(6, d, dtype=BF16, device=DEV), normal(d, seed=1)
    x[1] = normal(1, d, seed=2)[0]
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] = 1e-20
    x[5] = torch.finfo(BF16).tiny
    y, _, rstd = gb.add_rms_norm(x, w, eps=1e-6)
    assert not y[0].any() and abs(rstd[0].item() - 1000.0) < 1e-3
    assert y[2].isnan().all()
    assert y[3, 7].isnan() and not y[3, :7].any() and rstd[3] == 0
    _, _, rw, yw, slack = norm_reference(x[4:], None, w, 1e-6, 0.0, 0, 0)
    assert_within(y[4:], yw, HALF_BF16 * yw.abs() + slack + TINY)
    q, scale, _ = gb.add_rms_norm_q8(x, w, eps=1e-6)
    assert scale[0].item() == 2.0 ** -126 and not q[0].float().any()
    assert scale[2].isnan() and q[2].float().isnan().all()
    q, scale, _ = gb.add_rms_norm_q8(x, w, eps=1e-6, scale_group=128)
    assert (scale[0] == 2.0 ** -126).all() and scale[3, 0].isnan() and (scale[3, 1:] == 2.0 ** -126).all()


def test_norm_all_dropped():
    """p = 1: the branch leaves nothing, not even its NaN."""
    x, r, w = torch.full((4, 96), float("nan"), dtype=BF16, device=DEV), normal(4, 96, seed=1), normal(96, seed=2)
    y, h, _ = gb.add_rms_norm(x, w, r, p=1.0)
    assert torch.equal(h, r) and torch.equal(y, gb.add_rms_norm(r, w)[0])
    y, h, rstd = gb.add_rms_norm(x, w, p=1.0, eps=1e-6)
    assert not h.any() and not y.any()


@pytest.mark.parametrize("m,d", SIZES + [(1000, 96), (700, 1500), (5000, 520), (313, 9000), (2500, 33)])
@pytest.mark.parametrize("p", [0.0, 0.3])
@pytest.mark.parametrize("with_dh", [False, True])
def test_add_rms_norm_backward(m, d, p, with_dh):
    dy, h, w = normal(m, d, seed=d), normal(m, d, seed=d + 1, std=2.0), normal(d, seed=d + 2)
    dh = normal(m, d, seed=d + 3) if with_dh else None
    rstd = (h.float().square().mean(dim=1) + 1e-6).rsqrt()
    dx, dr, dw = gb.add_rms_norm_backward(dy, h, w, rstd, dh, p=p, seed=31, offset=d)
    want, dw_want = ref.norm_gradient(dy, h, w, dh, 1e-6, rstd)
    xhat, g = h.double() * rstd.double()[:, None], dy.double() * w.double()
    # the two terms may cancel: fp32 errors go with their sizes (64 terms deep at most in the row's sum)
    size = rstd.double()[:, None] * (g.abs() + xhat.abs() * (g * xhat).abs().mean(dim=1, keepdim=True))
    slack = 2.0 ** -17 * size + (2.0 ** -22 * dh.double().abs() if with_dh else 0)
    assert_within(dr, want, HALF_BF16 * want.abs() + slack * (1 + HALF_BF16) + TINY, "dR")
    if p == 0:
        assert dx is dr
    else:
        scale = torch.where(ref.keep_mask(m, d, p, 31, d).to(DEV), 1 / (1 - p), 0.0).double()
        assert_within(dx, want * scale, (HALF_BF16 * want.abs() + slack * (1 + HALF_BF16)) * scale + TINY, "dX")
        assert not dx[scale == 0].any()
    # dweight: a thread's rows one after the other (at least 8 blocks share them), then the blocks' parts
    terms = m / 8 + 64 + 8
    assert dw.dtype == torch.float32
    assert_within(dw, dw_want, terms * 2.0 ** -24 * (dy.double() * xhat).abs().sum(dim=0) + TINY, "dweight")


def test_norm_gradient_against_differences():
    """The kernels' gradients along a direction against central differences of the 64-bit forward pass."""
    m, d = 6, 777
    h, w, dy, dh = normal(m, d, seed=1), normal(d, seed=2), normal(m, d, seed=3), normal(m, d, seed=4)
    rstd = (h.float().square().mean(dim=1) + 1e-6).rsqrt()
    _, dr, dw = gb.add_rms_norm_backward(dy, h, w, rstd, dh)

    def loss(h_, w_):
        y = h_ * (h_.square().mean(dim=1, keepdim=True) + 1e-6).rsqrt() * w_
        return (dy.double() * y).sum() + (dh.double() * h_).sum()
    for grad, at, f, half in ((dr, h.double(), lambda t: loss(t, w.double()), HALF_BF16),
                              (dw, w.double(), lambda t: loss(h.double(), t), 2.0 ** -19)):
        v = torch.randn(at.shape, generator=gen(9), device=DEV).double()
        diff = (f(at + 1e-5 * v) - f(at - 1e-5 * v)) / 2e-5
        # the gradient's own rounding, term by term, and the difference's (1e-10 h''' and 1e-16 / 1e-5 of the loss)
        assert abs(diff - (grad.double() * v).sum()) < half * (grad.double() * v).abs().sum() + 1e-5


@pytest.mark.parametrize("offset", range(0, 8, 3))
@pytest.mark.parametrize("m,d", [(40, 203), (620, 1027), (300, 9001)])
def test_norm_backward_layouts(m, d, offset):
    dy, h, w, dh = normal(m, d, seed=1), normal(m, d, seed=2), normal(d, seed=3), normal(m, d, seed=4)
    rstd = (h.float().square().mean(dim=1) + 1e-6).rsqrt()
    dx, dr, dw = gb.add_rms_norm_backward(dy, h, w, rstd, dh, p=0.2, seed=1)
    size = (dy.double() * h.double() * rstd.double()[:, None]).abs().sum(dim=0)
    for extra, other in ((1, 1), (5, 5), (1, 2)):
        dx2, dr2, dw2 = gb.add_rms_norm_backward(padded(dy, extra, offset), padded(h, other, offset),
                                                 padded(w[None], 0, offset)[0], rstd, padded(dh, extra, offset), p=0.2,
                                                 seed=1)
        for a, b in ((dx2, dx), (dr2, dr)):
            # the mean's sum in another order: below 2^-17 of the terms (here of order 1), then a rounding each
            assert_within(a, b.double(), 2 * HALF_BF16 * b.double().abs() + 2.0 ** -13)
        assert_within(dw2, dw.double(), (m / 8 + 72) * 2.0 ** -23 * size + TINY)


def test_norm_backward_workspace_same_bits_and_empty():
    m, d = 900, 2100
    dy, h, w = normal(m, d, seed=1), normal(m, d, seed=2), normal(d, seed=3)
    rstd = (h.float().square().mean(dim=1) + 1e-6).rsqrt()
    first = gb.add_rms_norm_backward(dy, h, w, rstd, p=0.1, seed=5)
    need = gb.add_rms_norm_backward_workspace_bytes(m, d)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(gb.add_rms_norm_backward(dy, h, w, rstd, p=0.1, seed=5,
                                                                             workspace=ws), first))
    with pytest.raises(ValueError, match="workspace"):
        gb.add_rms_norm_backward(dy, h, w, rstd, workspace=ws[:-1])
    _, dr, dw = gb.add_rms_norm_backward(dy[:0], h[:0], w, rstd[:0])
    assert dr.shape == (0, d) and not dw.any()


def test_norm_on_another_stream_and_in_a_graph():
    x, r, w = normal(300, 4096, seed=1), normal(300, 4096, seed=2), normal(4096, seed=3)
    y, h, rstd = gb.add_rms_norm(x, w, r, p=0.1, seed=7, offset=1)
    state = torch.tensor([7, 0], dtype=torch.int64, device=DEV)
    out, hh = torch.empty_like(y), torch.empty_like(h)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gb.add_rms_norm(x, w, r, p=0.1, seed=state, out=out, h=hh)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            gb.add_rms_norm(x, w, r, p=0.1, seed=state, out=out, h=hh)
    torch.cuda.synchronize()
    state[1] = 1
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, y) and torch.equal(hh, h)


def test_plans_are_described():
    gb.dropout(normal(4, 8, seed=1), 0.1, 1)
    assert "kernel=dropout" in gb.last_plan()
    gb.add_rms_norm(normal(4, 8, seed=1), normal(8, seed=2))
    assert "kernel=add_rms_norm" in gb.last_plan()
    q, s, _ = w4_weights(8, 128, 128, False, 1)
    gb.linear_w4(normal(4, 128, seed=1), q, s)
    assert "kernel=w4" in gb.last_plan()
    gb.linear(normal(8, 64, seed=1), normal(8, 64, seed=2))
    assert "kernel=w4" not in gb.last_plan()


@pytest.mark.parametrize("seed", range(12))
def test_norm_feeds_the_products(seed):
    """A block's serving path: norm with 8-bit output, the gated pair, the down projection onto the residual."""
    rng = np.random.default_rng(seed)
    m, d, f, group = int(rng.integers(1, 34)), 32 * int(rng.integers(1, 40)), 32 * int(rng.integers(1, 60)), 64
    x, r, w = normal(m, d, seed=seed), normal(m, d, seed=seed + 1), normal(d, seed=seed + 2)
    q, scale, h = gb.add_rms_norm_q8(x, w, r, scale_group=128 if seed % 2 else 0)
    w1, w3, w2 = (w4_weights(n, k, group, True, 50 + i) for i, (n, k) in enumerate(((f, d), (f, d), (d, f))))
    act = gb.ffn_gated_w4(q, w1[0], w1[1], w3[0], w3[1], zeros1=w1[2], zeros3=w3[2], group=group, x_scale=scale)
    out = gb.linear_w4(act, w2[0], w2[1], R=h, zeros=w2[2], group=group)
    a = ref.w4_products(q, scale, ref.unpack_w4(*w1, group, d))[0]
    b = ref.w4_products(q, scale, ref.unpack_w4(*w3, group, d))[0]
    want = ref.act(a, "silu") * b
    # the pair's error is bounded in test_ffn_gated_w4; here 2^-16 of the largest covers its fp32 part
    assert_within(act, want, HALF_BF16 * want.abs() + 2.0 ** -16 * want.abs().max() + TINY)
    check_linear_result(out, act, None, w2[0], w2[1], w2[2], None, h, "none", group)


# ---------------------------------------------------------------------------------- plans

@pytest.fixture
def config():
    yield gb.set_config
    gb.set_config(None)


@pytest.mark.parametrize("m", [1, 3, 8, 16])
@pytest.mark.parametrize("gated", [False, True])
def test_w4_every_plan_gives_the_result(config, m, gated):
    """Columns over 1, 2, 4 and 8 CTAs and any number of a CTA's warps: rows, tokens and columns end inside."""
    n, k, group = 77, 2400, 32
    q, s, z = w4_weights(n, k, group, True, 3)
    q3, s3, z3 = w4_weights(n, k, group, True, 7)
    x, r = normal(m, k, seed=4), normal(m, n, seed=5)
    plans = set()
    for cluster in (1, 2, 4, 8):
        for k_warps in (1, 2, 4, 8, 16):
            config(f"w4_cluster={cluster},w4_k_warps={k_warps}")
            try:
                if gated:
                    d = gb.ffn_gated_w4(x, q, s, q3, s3, zeros1=z, zeros3=z3, group=group)
                else:
                    d = gb.linear_w4(x, q, s, R=r, zeros=z, group=group)
            except gb.GBError as e:
                assert e.status == 2 and "w4_cluster" in str(e)
                continue
            plans.add(gb.last_plan())
            if gated:
                a, off_a = ref.w4_products(x, None, ref.unpack_w4(q, s, z, group, k))
                b, off_b = ref.w4_products(x, None, ref.unpack_w4(q3, s3, z3, group, k))
                gate = ref.act(a, "silu")
                tol = (1.13 * off_a + 2.0 ** -20 * a.abs()) * (b.abs() + off_b) + gate.abs() * off_b
                assert_within(d, gate * b, tol * (1 + HALF_BF16) + HALF_BF16 * (gate * b).abs() + TINY, gb.last_plan())
            else:
                check_linear_result(d, x, None, q, s, z, None, r, "none", group, gb.last_plan())
    assert len(plans) >= 12


def test_w4_columns_that_end_before_the_last_cta(config):
    """CTAs of a cluster without any columns add nothing, whatever an earlier kernel left in shared memory."""
    config("w4_cluster=8,w4_k_warps=2")
    m, n, group = 4, 100, 64
    long_q, long_s, _ = w4_weights(n, 4096, group, False, 1)
    x8, xs = w4_input(m, 4096, "row", 2)
    for k in (2304, 256, 0):
        q, s, z = w4_weights(n, k, group, True, 3)
        x, r = normal(m, k, seed=4), normal(m, n, seed=5)
        assert gb.linear_w4(x8, long_q, long_s, group=group, x_scale=xs * float("nan")).isnan().all()
        d = gb.linear_w4(x, q, s, R=r, zeros=z, group=group)
        check_linear_result(d, x, None, q, s, z, None, r, "none", group, str(k))


def test_w4_config_refuses_what_no_plan_has(config):
    q, s, _ = w4_weights(8, 128, 128, False, 1)
    for bad in ("w4_cluster=3", "w4_k_warps=17", "w4_cluster=16"):
        with pytest.raises(gb.GBError):
            config(bad)
    config("w4_k_warps=5")
    with pytest.raises(gb.GBError, match="w4_k_warps"):
        gb.linear_w4(normal(1, 128, seed=1), q, s)


def test_w4_weights_at_their_zero_point_leave_nothing():
    """q = z = 8 everywhere: every output is exactly its residual, whatever x is."""
    q = torch.full((50, 1024), 0x88, dtype=torch.uint8, device=DEV)
    for group in (32, 64, 128):
        s = torch.full((50, 2048 // group), 3.0, dtype=BF16, device=DEV)
        for m in (1, 7, 16):
            assert not gb.linear_w4(normal(m, 2048, seed=m, std=100.0), q, s, group=group).any()


@pytest.mark.parametrize("m", [2, 12])
def test_w4_wide_range_of_x(m):
    """Channels of very different size, values at bf16's ends, rows of zeros."""
    q, s, z = w4_weights(64, 1024, 64, True, 5)
    x = normal(m, 1024, seed=6)
    x[0] = 0
    x[1, ::7] *= 2.0 ** 20
    x[1, ::11] *= 2.0 ** -60
    if m > 2:
        x[2] *= 2.0 ** -120
        x[3] *= 2.0 ** 110
        x[4] = torch.finfo(BF16).tiny
    d = gb.linear_w4(x, q, s, zeros=z, group=64)
    check_linear_result(d, x, None, q, s, z, None, None, "none", 64)


@pytest.mark.parametrize("m,n,k", [(3, 40, 700), (16, 33, 2048), (1, 5, 64)])
def test_w4_infinities_and_nan_anywhere(m, n, k):
    """Several a row, in every part of the columns; a weight at its zero point makes NaN of an infinity."""
    k = k // 32 * 32
    q, s, z = w4_weights(n, k, 32, True, 5)
    x = normal(m, k, seed=6)
    x[0, 0], x[0, k - 1] = float("inf"), float("inf")
    x[m // 2, k // 2] = float("-inf")
    x[m - 1, k // 3] = float("nan")
    d = gb.linear_w4(x, q, s, zeros=z, group=32)
    w = ref.unpack_w4(q, s, z, 32, k)
    fine = torch.isfinite(x)
    v, off = ref.w4_products(torch.where(fine, x, torch.zeros_like(x)), None, w)
    odd = torch.zeros_like(v)
    for i, j in (~fine).nonzero().tolist():
        odd[i] += x[i, j].double() * w[:, j]
    want = v + odd
    assert_within(d, want, torch.where(torch.isfinite(want), 1.0 * off + HALF_BF16 * want.abs() * 1.01 + TINY,
                                       torch.zeros_like(want)))


# ---------------------------------------------------------------------------------- calls one after another

def test_calls_back_to_back_see_each_other():
    """Kernels are set up while the one before runs: a chain of calls through the same buffers gives what the
    same calls give with a wait after each."""
    d = 512
    w = normal(d, seed=1)
    ws = [w4_weights(d, d, 64, True, 10 + i) for i in range(3)]

    def chain(wait):
        x, r = normal(4, d, seed=2), normal(4, d, seed=3)
        q8 = torch.empty(4, d, dtype=torch.float8_e4m3fn, device=DEV)
        for i in range(60):
            q, scale, r = gb.add_rms_norm_q8(x, w, r, out=q8, h=r)
            wait()
            gb.linear_w4(q, *ws[i % 3][:2], R=r, zeros=ws[i % 3][2], group=64, x_scale=scale, out=x, act="silu")
            wait()
            gb.dropout(x, 0.2, 5, i, out=x)
            wait()
            y, _, rstd = gb.add_rms_norm(x, w)
            wait()
            dx, _, dw = gb.add_rms_norm_backward(y, x, w, rstd, p=0.1, seed=i)
            wait()
            x = gb.dropout(dx, 0.0, 0, R=x)
            wait()
        return x, r, dw
    fast = chain(lambda: None)
    for a, b in zip(fast, chain(torch.cuda.synchronize)):
        assert torch.equal(a, b)


def test_binding_refuses_wrong_tensors():
    x, w = normal(4, 64, seed=1), normal(64, seed=2)
    q, s, z = w4_weights(8, 64, 64, True, 1)
    for error, call in (
            (TypeError, lambda: gb.linear_w4(x, q.float(), s, group=64)),
            (TypeError, lambda: gb.linear_w4(x, q, s.float(), group=64)),
            (TypeError, lambda: gb.linear_w4(x, q.cpu(), s, group=64)),
            (ValueError, lambda: gb.linear_w4(x[:, :32], q, s, group=64)),
            (ValueError, lambda: gb.linear_w4(x, q, s, group=32)),
            (ValueError, lambda: gb.linear_w4(x, q, s, group=64, zeros=z[:4])),
            (ValueError, lambda: gb.linear_w4(x, q, s, group=64, R=x)),
            (ValueError, lambda: gb.linear_w4(x, q.t().contiguous().t(), s, group=64)),
            (TypeError, lambda: gb.linear_w4(x.tolist(), q, s, group=64)),
            (ValueError, lambda: gb.dropout(x[0], 0.1, 1)),
            (ValueError, lambda: gb.dropout(x.t(), 0.1, 1)),
            (TypeError, lambda: gb.dropout(x, 0.1, 1.5)),
            (TypeError, lambda: gb.dropout(x, 0.1, torch.zeros(2, device=DEV))),
            (ValueError, lambda: gb.dropout(x, 0.1, torch.zeros(3, dtype=torch.int64, device=DEV))),
            (gb.GBError, lambda: gb.dropout(x, 1.5, 1)),
            (ValueError, lambda: gb.add_rms_norm(x, w[:32])),
            (TypeError, lambda: gb.add_rms_norm(x.float(), w)),
            (gb.GBError, lambda: gb.add_rms_norm(x, w, eps=-1.0)),
            (gb.GBError, lambda: gb.add_rms_norm_q8(x, w, scale_group=64)),
            (gb.GBError, lambda: gb.add_rms_norm(normal(1, 16400, seed=1), normal(16400, seed=2))),
            (ValueError, lambda: gb.add_rms_norm_backward(x, x, w, torch.ones(3, device=DEV))),
            (TypeError, lambda: gb.add_rms_norm_backward(x, x, w, torch.ones(4, device=DEV), workspace=x.cpu()))):
        with pytest.raises(error):
            call()
    gb.device_status()
