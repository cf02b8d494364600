"""Layer norm, low-rank adapters and the mixture of experts on the CPU: what the C ABI and the Python entry points
refuse before they touch a GPU, and the formulas of the gradients against differences."""
import ctypes

import numpy as np
import pytest
import torch

from tests import more_ref

GB_OK, GB_ERR_INVALID_ARG, GB_ERR_UNSUPPORTED = 0, 1, 2
P16, P4, P2, P1 = 0x10000, 0x10004, 0x10002, 0x10001  # never dereferenced


@pytest.fixture(scope="module")
def L():
    from dense_bf16_gemm_persistent_gb300 import _build
    _build.build()
    import dense_bf16_gemm_persistent_gb300 as gb
    return gb.lib()


# ---------------------------------------------------------------------------------- layer norm

def norm(L, X=P16, ldx=32, R=None, ldr=0, w=P16, b=None, eps=1e-5, p=0.0, H=None, ldh=0, Y=P16, ldy=32, mean=None,
         rstd=None, M=4, D=32, state=None):
    return L.gb_add_layer_norm(X, ldx, R, ldr, w, b, eps, p, 1, 2, state, H, ldh, Y, ldy, mean, rstd, M, D, None)


@pytest.mark.parametrize("kwargs,status,needle", [
    (dict(X=None), GB_ERR_INVALID_ARG, "X is null"),
    (dict(Y=None), GB_ERR_INVALID_ARG, "Y is null"),
    (dict(w=None), GB_ERR_INVALID_ARG, "weight is null"),
    (dict(M=-1), GB_ERR_INVALID_ARG, "negative"),
    (dict(eps=-1.0), GB_ERR_INVALID_ARG, "eps"),
    (dict(eps=float("nan")), GB_ERR_INVALID_ARG, "eps"),
    (dict(p=2.0), GB_ERR_INVALID_ARG, "probability"),
    (dict(ldx=31), GB_ERR_INVALID_ARG, "of X"),
    (dict(R=P16, ldr=31), GB_ERR_INVALID_ARG, "of R"),
    (dict(H=P16, ldh=31), GB_ERR_INVALID_ARG, "of H"),
    (dict(b=P1), GB_ERR_UNSUPPORTED, "bias"),
    (dict(mean=P2), GB_ERR_UNSUPPORTED, "mean"),
    (dict(rstd=P2), GB_ERR_UNSUPPORTED, "rstd"),
    (dict(state=P4), GB_ERR_UNSUPPORTED, "rng_state"),
    (dict(D=16385, ldx=16385, ldy=16385), GB_ERR_UNSUPPORTED, "16384"),
])
def test_add_layer_norm_rejects(L, kwargs, status, needle):
    assert norm(L, **kwargs) == status
    assert needle in L.gb_last_error().decode()


def bwd(L, dY=P16, H=P16, w=P16, mean=P16, rstd=P16, dH=None, p=0.0, dR=P16, dX=None, dw=P16, db=P16, D=32, M=4, ld=32):
    return L.gb_add_layer_norm_backward(dY, ld, H, ld, w, mean, rstd, dH, ld, p, 1, 2, None, dR, ld, dX, ld, dw, db, P16,
                                        1 << 30, M, D, None)


@pytest.mark.parametrize("kwargs,status,needle", [
    (dict(dY=None), GB_ERR_INVALID_ARG, "dY is null"),
    (dict(H=None), GB_ERR_INVALID_ARG, "H is null"),
    (dict(dR=None), GB_ERR_INVALID_ARG, "dR is null"),
    (dict(p=0.5), GB_ERR_INVALID_ARG, "dX is null"),
    (dict(dw=None), GB_ERR_INVALID_ARG, "dweight is null"),
    (dict(db=None), GB_ERR_INVALID_ARG, "dbias is null"),
    (dict(mean=None), GB_ERR_INVALID_ARG, "mean is null"),
    (dict(rstd=P2), GB_ERR_UNSUPPORTED, "rstd"),
    (dict(w=None), GB_ERR_INVALID_ARG, "weight is null"),
    (dict(ld=16), GB_ERR_INVALID_ARG, "leading dimension"),
    (dict(D=20000, ld=20000), GB_ERR_UNSUPPORTED, "16384"),
])
def test_add_layer_norm_backward_rejects(L, kwargs, status, needle):
    assert bwd(L, **kwargs) == status
    assert needle in L.gb_last_error().decode()


def test_empty_layer_norms_are_noops_without_a_device(L):
    assert norm(L, X=None, Y=None, w=None, M=0) == GB_OK and norm(L, X=None, Y=None, w=None, D=0) == GB_OK
    assert bwd(L, dY=None, H=None, w=None, mean=None, rstd=None, dR=None, dw=None, db=None, D=0) == GB_OK
    n = ctypes.c_size_t(7)
    assert L.gb_add_layer_norm_backward_workspace_bytes(0, 5, ctypes.byref(n)) == GB_OK and n.value == 0
    assert L.gb_add_layer_norm_backward_workspace_bytes(4, 5, None) == GB_ERR_INVALID_ARG


def test_python_layer_norm_refuses_host_tensors():
    import dense_bf16_gemm_persistent_gb300 as gb
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="X"):
        gb.add_layer_norm(x, w)
    with pytest.raises(TypeError, match="dY"):
        gb.add_layer_norm_backward(x, x, w, torch.ones(2), torch.ones(2))


def test_reference_layer_norm_gradient_is_the_forward_difference():
    """The formula that the GPU's gradients are held to, against central differences in 64 bits."""
    g = torch.Generator().manual_seed(5)
    h, dy, dh = (torch.randn(3, 17, generator=g, dtype=torch.float64) for _ in range(3))
    w, b = torch.rand(17, generator=g, dtype=torch.float64) + 0.5, torch.zeros(17, dtype=torch.float64)
    rstd = (h.var(dim=1, unbiased=False) + 1e-5).rsqrt()
    dr, dw, db = more_ref.layer_norm_gradient(dy, h, w, h.mean(dim=1), rstd, dh)

    def loss(h_, w_, b_):
        off = h_ - h_.mean(dim=1, keepdim=True)
        return (dy * (off * (off.square().mean(dim=1, keepdim=True) + 1e-5).rsqrt() * w_ + b_)).sum() + (dh * h_).sum()
    for grad, at, f in ((dr, h, lambda t: loss(t, w, b)), (dw, w, lambda t: loss(h, t, b)), (db, b, lambda t: loss(h, w, t))):
        v = torch.from_numpy(np.random.default_rng(1).standard_normal(tuple(at.shape)))
        # a central difference is off by step^2 times a third derivative (of order 10), and 1e-16 / step
        assert abs((f(at + 1e-5 * v) - f(at - 1e-5 * v)) / 2e-5 - (grad * v).sum()) < 1e-7


# ---------------------------------------------------------------------------------- mixture of experts

def moe(L, X=P16, ldx=64, router=P16, ldrouter=64, W1=P16, ld1=64, e1=2048, W3=P16, ld3=64, e3=2048, W2=P16, ld2=32, e2=2048,
        R=None, ldr=0, top=2, D=P16, ldd=64, ids=P16, weights=P16, ws=P16, wsb=1 << 30, T=3, d=64, inner=32, experts=4):
    return L.gb_moe_ffn_gated(X, ldx, router, ldrouter, W1, ld1, e1, W3, ld3, e3, W2, ld2, e2, R, ldr, top, 1, D, ldd, ids,
                              weights, ws, wsb, T, d, inner, experts, None)


@pytest.mark.parametrize("kwargs,status,needle", [
    (dict(X=None), GB_ERR_INVALID_ARG, "X is null"),
    (dict(router=None), GB_ERR_INVALID_ARG, "router is null"),
    (dict(W1=None), GB_ERR_INVALID_ARG, "W1 is null"),
    (dict(W3=None), GB_ERR_INVALID_ARG, "W3 is null"),
    (dict(W2=None), GB_ERR_INVALID_ARG, "W2 is null"),
    (dict(D=None), GB_ERR_INVALID_ARG, "D is null"),
    (dict(ids=None), GB_ERR_INVALID_ARG, "ids is null"),
    (dict(weights=None), GB_ERR_INVALID_ARG, "weights is null"),
    (dict(ws=None), GB_ERR_INVALID_ARG, "workspace"),
    (dict(wsb=100), GB_ERR_INVALID_ARG, "workspace"),
    (dict(ws=P4), GB_ERR_INVALID_ARG, "16-byte"),
    (dict(T=-1), GB_ERR_INVALID_ARG, "negative"),
    (dict(T=1 << 31), GB_ERR_UNSUPPORTED, "2^31"),
    (dict(inner=0), GB_ERR_INVALID_ARG, "experts of"),
    (dict(top=0), GB_ERR_INVALID_ARG, "top_k"),
    (dict(top=5), GB_ERR_INVALID_ARG, "top_k"),
    (dict(experts=1025), GB_ERR_UNSUPPORTED, "1024"),
    (dict(experts=64, top=17), GB_ERR_UNSUPPORTED, "top_k"),
    (dict(ldx=63), GB_ERR_INVALID_ARG, "of X"),
    (dict(ldx=68), GB_ERR_UNSUPPORTED, "X"),
    (dict(W1=P4), GB_ERR_UNSUPPORTED, "W1"),
    (dict(ld2=31), GB_ERR_INVALID_ARG, "of W2"),
    (dict(e1=2040), GB_ERR_INVALID_ARG, "W1"),
    (dict(e3=2052), GB_ERR_UNSUPPORTED, "W3"),
    (dict(e2=0), GB_ERR_INVALID_ARG, "W2"),
    (dict(ldd=63), GB_ERR_INVALID_ARG, "of D"),
    (dict(R=P16, ldr=63), GB_ERR_INVALID_ARG, "of R"),
    (dict(D=P1), GB_ERR_UNSUPPORTED, "2-byte"),
    (dict(weights=P2), GB_ERR_UNSUPPORTED, "4-byte"),
])
def test_moe_ffn_gated_rejects(L, kwargs, status, needle):
    assert moe(L, **kwargs) == status
    assert needle in L.gb_last_error().decode()


# A row of so many columns is within 32 bits, but not what the router counts ahead in it (2048 columns a turn).
@pytest.mark.parametrize("kwargs", [dict(d=2**31 - 1000), dict(inner=2**31 - 1000), dict(d=2**31 - 65535)])
def test_moe_ffn_gated_rejects_rows_that_are_counted_past_32_bits(L, kwargs):
    assert moe(L, **kwargs) == GB_ERR_UNSUPPORTED
    assert "65536" in L.gb_last_error().decode()


def test_empty_moe_is_a_noop_and_its_workspace_is_counted(L):
    assert moe(L, X=None, D=None, T=0) == GB_OK
    n = ctypes.c_size_t(7)
    # two terms of two bytes for each pair of a token and an expert, rows of whole 16 bytes; a pass has 64 tokens
    for t, tokens in ((0, 0), (3, 3), (64, 64), (1000, 64)):
        assert L.gb_moe_ffn_gated_workspace_bytes(t, 33, 8, 2, ctypes.byref(n)) == GB_OK and n.value == tokens * 2 * 40 * 4
    assert L.gb_moe_ffn_gated_workspace_bytes(3, 33, 8, 9, ctypes.byref(n)) == GB_ERR_INVALID_ARG
    assert L.gb_moe_ffn_gated_workspace_bytes(3, 33, 8, 2, None) == GB_ERR_INVALID_ARG


def test_python_moe_refuses_host_tensors():
    import dense_bf16_gemm_persistent_gb300 as gb
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(4, 64, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="X"):
        gb.moe_ffn_gated(x, x, w, w, w, 2)


# ---------------------------------------------------------------------------------- low-rank adapters

def lora(L, X=P16, ldx=64, A=P16, lda=64, aa=512, B=P16, ldb=8, ab=256, ids=P16, scale=None, R=None, ldr=0, act=0, D=P16,
         ldd=32, ws=P16, wsb=1 << 30, M=3, N=32, K=64, r=8, adapters=4):
    return L.gb_lora(X, ldx, A, lda, aa, B, ldb, ab, ids, scale, R, ldr, act, D, ldd, ws, wsb, M, N, K, r, adapters, None)


@pytest.mark.parametrize("kwargs,status,needle", [
    (dict(X=None), GB_ERR_INVALID_ARG, "X is null"),
    (dict(A=None), GB_ERR_INVALID_ARG, "A is null"),
    (dict(B=None), GB_ERR_INVALID_ARG, "B is null"),
    (dict(D=None), GB_ERR_INVALID_ARG, "D is null"),
    (dict(ids=None), GB_ERR_INVALID_ARG, "ids is null"),
    (dict(M=-1), GB_ERR_INVALID_ARG, "negative"),
    (dict(N=1 << 31), GB_ERR_UNSUPPORTED, "2^31"),
    (dict(r=257, ldb=264), GB_ERR_UNSUPPORTED, "rank"),
    (dict(act=4), GB_ERR_INVALID_ARG, "activation"),
    (dict(ldx=63), GB_ERR_INVALID_ARG, "of X"),
    (dict(ldx=65), GB_ERR_UNSUPPORTED, "X"),
    (dict(lda=60), GB_ERR_INVALID_ARG, "of A"),
    (dict(B=P4), GB_ERR_UNSUPPORTED, "B"),
    (dict(ldb=12), GB_ERR_UNSUPPORTED, "B"),
    (dict(ldb=1 << 26, ab=1 << 34), GB_ERR_UNSUPPORTED, "2^26"),
    (dict(lda=1 << 30, aa=1 << 34), GB_ERR_UNSUPPORTED, "2^31 elements"),
    (dict(aa=504), GB_ERR_INVALID_ARG, "A"),
    (dict(ab=260), GB_ERR_UNSUPPORTED, "B"),
    (dict(ldd=31), GB_ERR_INVALID_ARG, "of D"),
    (dict(R=P16, ldr=31), GB_ERR_INVALID_ARG, "of R"),
    (dict(R=P1, ldr=32), GB_ERR_UNSUPPORTED, "2-byte"),
    (dict(ids=P2), GB_ERR_UNSUPPORTED, "4-byte"),
    (dict(scale=P2), GB_ERR_UNSUPPORTED, "4-byte"),
])
def test_lora_rejects(L, kwargs, status, needle):
    assert lora(L, **kwargs) == status
    assert needle in L.gb_last_error().decode()


def test_empty_lora_is_a_noop(L):
    assert lora(L, X=None, A=None, B=None, D=None, ids=None, M=0) == GB_OK
    assert lora(L, X=None, A=None, B=None, D=None, ids=None, N=0) == GB_OK
    n = ctypes.c_size_t(7)
    assert L.gb_lora_workspace_bytes(0, 8, 8, 8, ctypes.byref(n)) == GB_OK and n.value == 0
    # two terms of two bytes for each row and rank, in whole steps of 16 or 32; of more than 128 rows their order too
    for m, r, want in ((3, 5, 3 * 16 * 4), (128, 40, 128 * 64 * 4), (129, 16, 129 * 16 * 4 + 130 * 16 + 129 * 4)):
        assert L.gb_lora_workspace_bytes(m, 8, 8, r, ctypes.byref(n)) == GB_OK and n.value == want
    assert L.gb_lora_workspace_bytes(8, 8, 8, 300, ctypes.byref(n)) == GB_ERR_UNSUPPORTED
    assert L.gb_lora_workspace_bytes(8, 8, 8, 8, None) == GB_ERR_INVALID_ARG


def test_python_lora_refuses_host_tensors():
    import dense_bf16_gemm_persistent_gb300 as gb
    x, a = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(4, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="X"):
        gb.lora(x, a, a.transpose(1, 2).contiguous(), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="act"):
        gb.lora(x, a, a, torch.zeros(2, dtype=torch.int32), act="tanh")
