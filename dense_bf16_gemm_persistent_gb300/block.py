"""The operators around the products: 4-bit layers for a few tokens, the norm, dropout.

    linear_w4(X, Wq, scales, bias, R, act)       ->  bf16(act(X @ W.T + bias) + R), W = (q - z) * s
    ffn_gated_w4(X, W1q, s1, W3q, s3)            ->  bf16(silu(X @ W1.T) * (X @ W3.T))
    add_rms_norm(X, weight, R, p, seed, offset)  ->  (Y, H, rstd): H = dropout(X) + R, Y = H / rms(H) * weight
    add_rms_norm_q8(X, weight, R)                ->  (Q, scale, H): the same in e4m3 with scales
    add_rms_norm_backward(dY, H, weight, rstd)   ->  (dX, dR, dweight)
    dropout(X, p, seed, offset, R)               ->  bf16(keep * X / (1 - p) + R)

Argument marshalling only, like the package's module; ``include/gbgemm.h`` has the definitions.
"""
from __future__ import annotations

import ctypes

import torch

from . import ACT, _check, _mat, _stream, lib

_BF16, _E4M3, _F32, _U8 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.uint8


def _tensor(t: torch.Tensor, name: str, dtype, shape: tuple):
    """(pointer, leading dimension in elements) of a CUDA tensor of this type and shape (1-D or 2-D, its
    last dimension contiguous)."""
    if t.dtype != dtype or not t.is_cuda:
        raise TypeError(f"{name}: expected a CUDA {dtype} tensor, got {t.dtype} on {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")
    stride, width = t.stride(), shape[-1]
    if width > 1 and stride[-1] != 1:
        raise ValueError(f"{name}: expected a contiguous last dimension")
    if len(shape) == 1:
        return t.data_ptr(), width
    # (one row's stride is arbitrary: at least its width)
    return t.data_ptr(), stride[0] if shape[0] > 1 else max(stride[0], width, 1)


def _rng(seed, offset):
    """(seed, offset, state pointer): two numbers, or a CUDA int64 tensor {seed, offset} as `seed`."""
    if isinstance(seed, torch.Tensor):
        return 0, 0, _tensor(seed, "seed", torch.int64, (2,))[0]
    return seed & 0xFFFFFFFFFFFFFFFF, offset & 0xFFFFFFFFFFFFFFFF, None


def _activations(X: torch.Tensor, x_scale, M: int, K: int):
    """(pointer, ld, gb_x_type_t, scales' pointer, their ld) of a product's X."""
    if X.dtype == _E4M3:
        if x_scale is None:
            raise ValueError("x_scale: float8_e4m3fn X needs its scales")
        px, ldx = _tensor(X, "X", _E4M3, (M, K))
        groups = -(-K // 128)
        if x_scale.dim() == 1:
            x_scale = x_scale[:, None]
        by_group = x_scale.dim() == 2 and x_scale.shape[1] == groups and groups > 1
        ps, lds = _tensor(x_scale, "x_scale", _F32, (M, groups if by_group else 1))
        return px, ldx, 2 if by_group else 1, ps, lds
    if x_scale is not None:
        raise ValueError("x_scale: only float8_e4m3fn X has scales")
    px, ldx = _mat(X, "X", M, K)
    return px, ldx, 0, None, 0


def _weights(Wq, scales, zeros, names, N: int, K: int, groups: int):
    pq, ldq = _tensor(Wq, names[0], _U8, (N, K // 2))
    ps, lds = _tensor(scales, names[1], _BF16, (N, groups))
    pz, ldz = _tensor(zeros, names[2], _U8, (N, groups)) if zeros is not None else (None, 0)
    return pq, ldq, ps, lds, pz, ldz


def _group(group: int, K: int) -> int:
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    return -(-K // group)


def linear_w4(X: torch.Tensor, Wq: torch.Tensor, scales: torch.Tensor, bias: torch.Tensor | None = None,
              R: torch.Tensor | None = None, act: str = "none", zeros: torch.Tensor | None = None, group: int = 128,
              x_scale: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """D = bf16(act(X @ W.T + bias) + R) for a few tokens, W[n,k] = (q[n,k] - z[n,k//group]) * scales[n,k//group].

    X [M,K] bf16, or float8_e4m3fn with x_scale ([M] or [M,1]: a row's; [M,ceil(K/128)]: of 128 columns); Wq
    [N,K/2] uint8 (the low nibble is the even column); scales [N,ceil(K/group)] bf16; zeros uint8 of the same
    shape (None: 8); bias [N], R [M,N] as in linear()."""
    M, K = X.shape
    N = Wq.shape[0]
    if act not in ACT:
        raise ValueError(f"act must be one of {sorted(ACT)}")
    groups = _group(group, K)
    x = _activations(X, x_scale, M, K)
    w = _weights(Wq, scales, zeros, ("Wq", "scales", "zeros"), N, K, groups)
    pb = _tensor(bias, "bias", _BF16, (N,))[0] if bias is not None else None
    pr, ldr = _mat(R, "R", M, N)
    if out is None:
        out = torch.empty((M, N), dtype=_BF16, device=X.device)
    pd, ldd = _mat(out, "out", M, N)
    _check(lib().gb_gemm_linear_w4(*x, *w, group, pb, pr, ldr, ACT[act], pd, ldd, M, N, K, _stream(stream)))
    return out


def ffn_gated_w4(X: torch.Tensor, W1q: torch.Tensor, scales1: torch.Tensor, W3q: torch.Tensor, scales3: torch.Tensor,
                 zeros1: torch.Tensor | None = None, zeros3: torch.Tensor | None = None, group: int = 128,
                 x_scale: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """D = bf16(silu(X @ W1.T) * (X @ W3.T)) for a few tokens, the weights as in linear_w4()."""
    M, K = X.shape
    N = W1q.shape[0]
    groups = _group(group, K)
    x = _activations(X, x_scale, M, K)
    w1 = _weights(W1q, scales1, zeros1, ("W1q", "scales1", "zeros1"), N, K, groups)
    w3 = _weights(W3q, scales3, zeros3, ("W3q", "scales3", "zeros3"), N, K, groups)
    if out is None:
        out = torch.empty((M, N), dtype=_BF16, device=X.device)
    pd, ldd = _mat(out, "out", M, N)
    _check(lib().gb_gemm_ffn_gated_w4(*x, *w1, *w3, group, pd, ldd, M, N, K, _stream(stream)))
    return out


def dropout(X: torch.Tensor, p: float, seed, offset: int = 0, R: torch.Tensor | None = None,
            out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """D = bf16(keep * X / (1 - p) + R); keep is drawn from (seed, offset) and the element's place alone, so the
    gradient of X is dropout(dD, p, seed, offset).  `seed`: a number, or a CUDA int64 tensor {seed, offset} that
    is read when the kernel runs (a replayed graph then draws what the tensor holds)."""
    M, N = X.shape
    px, ldx = _mat(X, "X", M, N)
    pr, ldr = _mat(R, "R", M, N)
    if out is None:
        out = torch.empty((M, N), dtype=_BF16, device=X.device)
    pd, ldd = _mat(out, "out", M, N)
    seed, offset, state = _rng(seed, offset)
    _check(lib().gb_dropout(px, ldx, pr, ldr, p, seed, offset, state, pd, ldd, M, N, _stream(stream)))
    return out


def add_rms_norm(X: torch.Tensor, weight: torch.Tensor, R: torch.Tensor | None = None, eps: float = 1e-6,
                 p: float = 0.0, seed=0, offset: int = 0, out: torch.Tensor | None = None,
                 h: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(Y, H, rstd): H = dropout(X) + R (p, seed, offset as in dropout()), rstd = 1 / sqrt(mean(H^2) + eps) of
    each row, Y = H * rstd * weight from H before its rounding.  Without R and dropout H is X itself."""
    M, D = X.shape
    px, ldx = _mat(X, "X", M, D)
    pr, ldr = _mat(R, "R", M, D)
    pw = _tensor(weight, "weight", _BF16, (D,))[0]
    if out is None:
        out = torch.empty((M, D), dtype=_BF16, device=X.device)
    py, ldy = _mat(out, "out", M, D)
    ph, ldh = None, 0
    if h is None and R is None and p == 0:
        h = X
    else:
        if h is None:
            h = torch.empty((M, D), dtype=_BF16, device=X.device)
        ph, ldh = _mat(h, "h", M, D)
    rstd = torch.empty(M, dtype=_F32, device=X.device)
    seed, offset, state = _rng(seed, offset)
    _check(lib().gb_add_rms_norm(px, ldx, pr, ldr, pw, eps, p, seed, offset, state, ph, ldh, py, ldy,
                                 rstd.data_ptr(), M, D, _stream(stream)))
    return out, h, rstd


def add_rms_norm_q8(X: torch.Tensor, weight: torch.Tensor, R: torch.Tensor | None = None, eps: float = 1e-6,
                    scale_group: int = 0, out: torch.Tensor | None = None, h: torch.Tensor | None = None,
                    stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(Q, scale, H): the norm's output in float8_e4m3fn, Q * scale = Y.  scale is [M,1] (scale_group = 0) or
    [M,ceil(D/128)] (scale_group = 128), as linear_w4() and ffn_gated_w4() take it."""
    M, D = X.shape
    px, ldx = _mat(X, "X", M, D)
    pr, ldr = _mat(R, "R", M, D)
    pw = _tensor(weight, "weight", _BF16, (D,))[0]
    if out is None:
        out = torch.empty((M, D), dtype=_E4M3, device=X.device)
    pq, ldq = _tensor(out, "out", _E4M3, (M, D))
    ph, ldh = None, 0
    if h is None and R is None:
        h = X
    else:
        if h is None:
            h = torch.empty((M, D), dtype=_BF16, device=X.device)
        ph, ldh = _mat(h, "h", M, D)
    scale = torch.empty((M, -(-D // scale_group) if scale_group > 0 else 1), dtype=_F32, device=X.device)
    _check(lib().gb_add_rms_norm_q8(px, ldx, pr, ldr, pw, eps, scale_group, ph, ldh, pq, ldq, scale.data_ptr(),
                                    max(scale.shape[1], 1), M, D, _stream(stream)))
    return out, scale, h


def add_rms_norm_backward_workspace_bytes(M: int, D: int) -> int:
    """Bytes of workspace add_rms_norm_backward() needs on the current device."""
    n = ctypes.c_size_t(0)
    _check(lib().gb_add_rms_norm_backward_workspace_bytes(M, D, ctypes.byref(n)))
    return int(n.value)


def add_rms_norm_backward(dY: torch.Tensor, H: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                          dH: torch.Tensor | None = None, p: float = 0.0, seed=0, offset: int = 0,
                          workspace: torch.Tensor | None = None,
                          stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(dX, dR, dweight) of add_rms_norm() from the gradient dY of Y and (optionally) dH of H, with H and rstd as
    it returned them and the same p, seed and offset.  Without dropout dX is dR; dweight [D] is fp32."""
    M, D = dY.shape
    py, ldy = _mat(dY, "dY", M, D)
    ph, ldh = _mat(H, "H", M, D)
    pw = _tensor(weight, "weight", _BF16, (D,))[0]
    ps = _tensor(rstd, "rstd", _F32, (M,))[0]
    pg, ldg = _mat(dH, "dH", M, D)
    dR = torch.empty((M, D), dtype=_BF16, device=dY.device)
    dX = torch.empty((M, D), dtype=_BF16, device=dY.device) if p > 0 else dR
    dweight = torch.empty(D, dtype=_F32, device=dY.device)
    need = add_rms_norm_backward_workspace_bytes(M, D)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=_U8, device=dY.device)
    elif workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace holds {workspace.numel() * workspace.element_size()} bytes, {need} needed")
    seed, offset, state = _rng(seed, offset)
    ld = max(D, 1)
    _check(lib().gb_add_rms_norm_backward(py, ldy, ph, ldh, pw, ps, pg, ldg, p, seed, offset, state, dR.data_ptr(), ld,
                                          dX.data_ptr(), ld, dweight.data_ptr(), workspace.data_ptr(),
                                          workspace.numel() * workspace.element_size(), M, D, _stream(stream)))
    return dX, dR, dweight
