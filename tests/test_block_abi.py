"""The operators around the products on the CPU: the generator's published vectors, and the calls
that the C ABI and the Python entry points refuse before they touch a GPU."""
import ctypes

import numpy as np
import pytest
import torch

from tests import block_ref as ref

GB_OK, GB_ERR_INVALID_ARG, GB_ERR_UNSUPPORTED = 0, 1, 2
P16, P4, P2, P1 = 0x10000, 0x10004, 0x10002, 0x10001  # never dereferenced


@pytest.fixture(scope="module")
def L():
    from dense_bf16_gemm_persistent_gb300 import _build
    _build.build()
    import dense_bf16_gemm_persistent_gb300 as gb
    return gb.lib()


@pytest.mark.parametrize("counter,key,out", [
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_reference_generator_has_the_published_vectors(counter, key, out):
    assert tuple(int(w) for w in ref.philox(counter, key)) == out


def test_reference_mask_keeps_the_share_it_should():
    mask = ref.keep_mask(512, 1024, 0.1, seed=3, offset=9)
    # 524288 draws: five standard deviations are 5 sqrt(0.09 / 524288)
    assert abs(mask.double().mean().item() - 0.9) < 5 * (0.09 / 524288) ** 0.5
    assert ref.keep_mask(4, 9, 0.0, 1, 1).all() and not ref.keep_mask(4, 9, 1.0, 1, 1).any()


def w4(L, X=P16, ldx=64, xt=0, xs=None, ldxs=0, W=P16, ldq=32, s=P2, lds=1, z=None, ldz=0, group=128, bias=None,
       R=None, ldr=0, act=0, D=P16, ldd=32, M=4, N=32, K=64):
    return L.gb_gemm_linear_w4(X, ldx, xt, xs, ldxs, W, ldq, s, lds, z, ldz, group, bias, R, ldr, act, D, ldd, M, N, K,
                               None)


@pytest.mark.parametrize("kwargs,status,needle", [
    (dict(X=None), GB_ERR_INVALID_ARG, "X is null"),
    (dict(W=None), GB_ERR_INVALID_ARG, "W is null"),
    (dict(s=None), GB_ERR_INVALID_ARG, "scales is null"),
    (dict(D=None), GB_ERR_INVALID_ARG, "D is null"),
    (dict(M=-1), GB_ERR_INVALID_ARG, "negative"),
    (dict(ldx=32), GB_ERR_INVALID_ARG, "ldx"),
    (dict(ldq=16), GB_ERR_INVALID_ARG, "leading dimension"),
    (dict(lds=0), GB_ERR_INVALID_ARG, "groups"),
    (dict(z=P1, ldz=0), GB_ERR_INVALID_ARG, "groups"),
    (dict(ldd=31), GB_ERR_INVALID_ARG, "ldd"),
    (dict(R=P16, ldr=31), GB_ERR_INVALID_ARG, "ldr"),
    (dict(group=16), GB_ERR_INVALID_ARG, "group"),
    (dict(act=4), GB_ERR_INVALID_ARG, "activation"),
    (dict(xt=3), GB_ERR_INVALID_ARG, "type of X"),
    (dict(xt=1), GB_ERR_INVALID_ARG, "x_scale is null"),
    (dict(xt=2, xs=P4, ldxs=0), GB_ERR_INVALID_ARG, "ldxs"),
    (dict(xt=1, xs=P2, ldxs=1), GB_ERR_UNSUPPORTED, "x_scale"),
    (dict(K=48), GB_ERR_UNSUPPORTED, "multiple of 32"),
    (dict(W=P4), GB_ERR_UNSUPPORTED, "16 bytes"),
    (dict(ldq=40), GB_ERR_UNSUPPORTED, "16 bytes"),
    (dict(s=P1), GB_ERR_UNSUPPORTED, "2-byte"),
    (dict(D=P1), GB_ERR_UNSUPPORTED, "2-byte"),
    (dict(X=P1), GB_ERR_UNSUPPORTED, "2-byte"),
    (dict(N=1 << 31), GB_ERR_UNSUPPORTED, "2^31"),
])
def test_linear_w4_rejects(L, kwargs, status, needle):
    assert w4(L, **kwargs) == status
    assert needle in L.gb_last_error().decode()


def test_ffn_gated_w4_names_the_matrix_it_rejects(L):
    a = [P16, 64, 0, None, 0, P16, 32, P2, 1, None, 0, P16, 32, P2, 1, None, 0, 128, P16, 32, 4, 32, 64, None]
    for at, value, needle in ((11, None, "W3 is null"), (5, P4, "W1"), (12, 8, "W3"), (17, 96, "group")):
        b = list(a)
        b[at] = value
        assert L.gb_gemm_ffn_gated_w4(*b) != GB_OK
        assert needle in L.gb_last_error().decode()


def drop(L, X=P16, ldx=32, R=None, ldr=0, p=0.1, D=P16, ldd=32, M=4, N=32, state=None):
    return L.gb_dropout(X, ldx, R, ldr, p, 1, 2, state, D, ldd, M, N, None)


@pytest.mark.parametrize("kwargs,status,needle", [
    (dict(X=None), GB_ERR_INVALID_ARG, "X is null"),
    (dict(D=None), GB_ERR_INVALID_ARG, "D is null"),
    (dict(p=-0.1), GB_ERR_INVALID_ARG, "probability"),
    (dict(p=1.5), GB_ERR_INVALID_ARG, "probability"),
    (dict(p=float("nan")), GB_ERR_INVALID_ARG, "probability"),
    (dict(ldx=31), GB_ERR_INVALID_ARG, "of X"),
    (dict(R=P16, ldr=8), GB_ERR_INVALID_ARG, "of R"),
    (dict(M=-2), GB_ERR_INVALID_ARG, "negative"),
    (dict(X=P1), GB_ERR_UNSUPPORTED, "2-byte"),
    (dict(state=P4), GB_ERR_UNSUPPORTED, "8-byte"),
    (dict(N=1 << 31, ldx=1 << 31, ldd=1 << 31), GB_ERR_UNSUPPORTED, "2^31"),
])
def test_dropout_rejects(L, kwargs, status, needle):
    assert drop(L, **kwargs) == status
    assert needle in L.gb_last_error().decode()


def norm(L, X=P16, ldx=32, R=None, ldr=0, w=P16, eps=1e-6, p=0.0, H=None, ldh=0, Y=P16, ldy=32, rstd=None, M=4, D=32):
    return L.gb_add_rms_norm(X, ldx, R, ldr, w, eps, p, 1, 2, None, H, ldh, Y, ldy, rstd, M, D, None)


@pytest.mark.parametrize("kwargs,status,needle", [
    (dict(X=None), GB_ERR_INVALID_ARG, "X is null"),
    (dict(Y=None), GB_ERR_INVALID_ARG, "Y is null"),
    (dict(w=None), GB_ERR_INVALID_ARG, "weight is null"),
    (dict(eps=-1.0), GB_ERR_INVALID_ARG, "eps"),
    (dict(eps=float("inf")), GB_ERR_INVALID_ARG, "eps"),
    (dict(p=2.0), GB_ERR_INVALID_ARG, "probability"),
    (dict(R=P16, ldr=31), GB_ERR_INVALID_ARG, "of R"),
    (dict(H=P16, ldh=31), GB_ERR_INVALID_ARG, "of H"),
    (dict(rstd=P2), GB_ERR_UNSUPPORTED, "rstd"),
    (dict(w=P1), GB_ERR_UNSUPPORTED, "weight"),
    (dict(D=16385, ldx=16385, ldy=16385), GB_ERR_UNSUPPORTED, "16384"),
])
def test_add_rms_norm_rejects(L, kwargs, status, needle):
    assert norm(L, **kwargs) == status
    assert needle in L.gb_last_error().decode()


def norm_q8(L, group=0, Q=P16, ldq=256, scale=P16, lds=2, M=4, D=256, X=P16):
    return L.gb_add_rms_norm_q8(X, 256, None, 0, P16, 1e-6, group, None, 0, Q, ldq, scale, lds, M, D, None)


@pytest.mark.parametrize("kwargs,status,needle", [
    (dict(group=64), GB_ERR_INVALID_ARG, "scale_group"),
    (dict(Q=None), GB_ERR_INVALID_ARG, "Q is null"),
    (dict(scale=None), GB_ERR_INVALID_ARG, "scale is null"),
    (dict(group=128, lds=1), GB_ERR_INVALID_ARG, "of scale"),
    (dict(ldq=255), GB_ERR_INVALID_ARG, "of Q"),
    (dict(scale=P2), GB_ERR_UNSUPPORTED, "scale"),
])
def test_add_rms_norm_q8_rejects(L, kwargs, status, needle):
    assert norm_q8(L, **kwargs) == status
    assert needle in L.gb_last_error().decode()


def bwd(L, dY=P16, H=P16, w=P16, rstd=P16, dH=None, p=0.0, dR=P16, dX=None, dw=P16, D=32, M=4, ld=32):
    return L.gb_add_rms_norm_backward(dY, ld, H, ld, w, rstd, dH, ld, p, 1, 2, None, dR, ld, dX, ld, dw, P16, 1 << 30, M,
                                      D, None)


@pytest.mark.parametrize("kwargs,status,needle", [
    (dict(dY=None), GB_ERR_INVALID_ARG, "dY is null"),
    (dict(H=None), GB_ERR_INVALID_ARG, "H is null"),
    (dict(dR=None), GB_ERR_INVALID_ARG, "dR is null"),
    (dict(p=0.5), GB_ERR_INVALID_ARG, "dX is null"),
    (dict(dw=None), GB_ERR_INVALID_ARG, "dweight is null"),
    (dict(rstd=None), GB_ERR_INVALID_ARG, "rstd is null"),
    (dict(w=None), GB_ERR_INVALID_ARG, "weight is null"),
    (dict(ld=16), GB_ERR_INVALID_ARG, "leading dimension"),
    (dict(dH=P1), GB_ERR_UNSUPPORTED, "dH"),
    (dict(D=20000, ld=20000), GB_ERR_UNSUPPORTED, "16384"),
])
def test_add_rms_norm_backward_rejects(L, kwargs, status, needle):
    assert bwd(L, **kwargs) == status
    assert needle in L.gb_last_error().decode()


def test_empty_calls_are_noops_without_a_device(L):
    assert w4(L, X=None, W=None, s=None, D=None, M=0) == GB_OK
    assert w4(L, X=None, W=None, s=None, D=None, N=0) == GB_OK
    assert drop(L, X=None, D=None, M=0) == GB_OK and drop(L, X=None, D=None, N=0) == GB_OK
    assert norm(L, X=None, Y=None, w=None, M=0) == GB_OK
    assert norm_q8(L, X=None, Q=None, scale=None, D=0) == GB_OK
    assert bwd(L, dY=None, H=None, w=None, rstd=None, dR=None, dw=None, D=0) == GB_OK
    n = ctypes.c_size_t(7)
    assert L.gb_add_rms_norm_backward_workspace_bytes(0, 5, ctypes.byref(n)) == GB_OK and n.value == 0
    assert L.gb_add_rms_norm_backward_workspace_bytes(-1, 5, ctypes.byref(n)) == GB_ERR_INVALID_ARG
    assert L.gb_add_rms_norm_backward_workspace_bytes(4, 5, None) == GB_ERR_INVALID_ARG


def test_python_entry_points_refuse_host_tensors_and_wrong_arguments():
    import dense_bf16_gemm_persistent_gb300 as gb
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(32, 32, dtype=torch.uint8)
    s = torch.zeros(32, 1, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="X"):
        gb.linear_w4(x, w, s)
    with pytest.raises(ValueError, match="group"):
        gb.linear_w4(x, w, s, group=256)
    with pytest.raises(ValueError, match="act"):
        gb.linear_w4(x, w, s, act="tanh")
    with pytest.raises(ValueError, match="x_scale"):
        gb.linear_w4(x, w, s, x_scale=torch.ones(2, 1))
    with pytest.raises(ValueError, match="x_scale"):
        gb.linear_w4(x.to(torch.float8_e4m3fn), w, s)
    with pytest.raises(TypeError, match="X"):
        gb.dropout(x, 0.1, 1)
    with pytest.raises(TypeError, match="X"):
        gb.add_rms_norm(x, s[:, 0])
    with pytest.raises(TypeError, match="dY"):
        gb.add_rms_norm_backward(x, x, s[:, 0], torch.ones(2))


def test_reference_norm_gradient_is_the_forward_difference():
    """The formula that the GPU's gradients are held to, against central differences in 64 bits."""
    g = torch.Generator().manual_seed(5)
    h, dy, dh = (torch.randn(3, 17, generator=g, dtype=torch.float64) for _ in range(3))
    w = torch.rand(17, generator=g, dtype=torch.float64) + 0.5
    dr, dw = ref.norm_gradient(dy, h, w, dh, 1e-6)

    def loss(h_, w_):
        rstd = (h_.square().mean(dim=1, keepdim=True) + 1e-6).rsqrt()
        return (dy * h_ * rstd * w_).sum() + (dh * h_).sum()
    for grad, at, f in ((dr, h, lambda t: loss(t, w)), (dw, w, lambda t: loss(h, t))):
        v = torch.from_numpy(np.random.default_rng(1).standard_normal(tuple(at.shape)))
        # a central difference is off by step^2 times a third derivative (of order 10), and 1e-16 / step
        assert abs((f(at + 1e-5 * v) - f(at - 1e-5 * v)) / 2e-5 - (grad * v).sum()) < 1e-7
