"""The operators around the products: 4-bit layers for a few tokens, norms, dropout, adapters, experts.

    linear_w4(X, Wq, scales, bias, R, act)       ->  bf16(act(X @ W.T + bias) + R), W = (q - z) * s
    ffn_gated_w4(X, W1q, s1, W3q, s3)            ->  bf16(silu(X @ W1.T) * (X @ W3.T))
    add_rms_norm(X, weight, R, p, seed, offset)  ->  (Y, H, rstd): H = dropout(X) + R, Y = H / rms(H) * weight
    add_rms_norm_q8(X, weight, R)                ->  (Q, scale, H): the same in e4m3 with scales
    add_rms_norm_backward(dY, H, weight, rstd)   ->  (dX, dR, dweight)
    add_layer_norm(X, weight, bias, R, p, seed)  ->  (Y, H, mean, rstd): Y = (H - mean) * rstd * weight + bias
    add_layer_norm_backward(dY, H, weight, mean, rstd)  ->  (dX, dR, dweight, dbias)
    lora(X, A, B, ids, scale, R, act)            ->  bf16(act(R + scale * (X @ A[id].T) @ B[id].T)), id = ids[row]
    moe_ffn_gated(X, router, W1, W3, W2, top_k)  ->  (D, ids, weights): the top experts' gated layers, weighted
    dropout(X, p, seed, offset, R)               ->  bf16(keep * X / (1 - p) + R)

Tensors are on the current device.  Argument marshalling only, like the package's module, here by the compiled
``_gbgemm_torch.so`` (``csrc/binding.cpp``): these calls take microseconds on the GPU.  There is no fallback; a
call raises if it is not built.  ``include/gbgemm.h`` has the definitions.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

import torch

from . import _PKG, ACT, GBError, _check, _lock, _on, _raw_stream, lib

_module = None


def _bind(m, L, device=torch._C._cuda_getDevice) -> None:
    stream = _raw_stream or (lambda number: torch.cuda.current_stream(number).cuda_stream)
    m.bind(GBError, device, stream, *[ctypes.cast(getattr(L, name), ctypes.c_void_p).value for name in (
        "gb_gemm_linear_w4", "gb_gemm_ffn_gated_w4", "gb_dropout", "gb_add_rms_norm", "gb_add_rms_norm_q8",
        "gb_add_rms_norm_backward", "gb_add_rms_norm_backward_workspace_bytes", "gb_add_layer_norm",
        "gb_add_layer_norm_backward", "gb_add_layer_norm_backward_workspace_bytes",
        "gb_moe_ffn_gated", "gb_moe_ffn_gated_workspace_bytes", "gb_lora", "gb_lora_workspace_bytes", "gb_last_error")])


def binding():
    """The compiled binding, loaded and given the C library's functions."""
    global _module
    path = os.path.join(_PKG, "_gbgemm_torch.so")
    if not os.path.exists(path):
        raise RuntimeError(f"the binding {path} is not built; run "
                           "`python -c 'import __graft_entry__ as g; g.build()'` first")
    L = lib()
    with _lock:
        if _module is None:
            loader = importlib.machinery.ExtensionFileLoader("_gbgemm_torch", path)
            m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_gbgemm_torch", loader))
            loader.exec_module(m)
            _bind(m, L)
            _module = m
        return _module


def linear_w4(X: torch.Tensor, Wq: torch.Tensor, scales: torch.Tensor, bias: torch.Tensor | None = None,
              R: torch.Tensor | None = None, act: str = "none", zeros: torch.Tensor | None = None, group: int = 128,
              x_scale: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """D = bf16(act(X @ W.T + bias) + R) for a few tokens, W[n,k] = (q[n,k] - z[n,k//group]) * scales[n,k//group].

    X [M,K] bf16, or float8_e4m3fn with x_scale ([M] or [M,1]: a row's; [M,ceil(K/128)]: of 128 columns); Wq
    [N,K/2] uint8 (the low nibble is the even column); scales [N,ceil(K/group)] bf16; zeros uint8 of the same
    shape, their low four bits (None: 8); bias [N], R [M,N] as in linear()."""
    if stream is not None:
        return _on(stream, linear_w4, X, Wq, scales, bias, R, act, zeros, group, x_scale, out)
    if act not in ACT:
        raise ValueError(f"act must be one of {sorted(ACT)}")
    return (_module or binding()).linear_w4(X, Wq, scales, bias, R, ACT[act], zeros, group, x_scale, out)


def ffn_gated_w4(X: torch.Tensor, W1q: torch.Tensor, scales1: torch.Tensor, W3q: torch.Tensor, scales3: torch.Tensor,
                 zeros1: torch.Tensor | None = None, zeros3: torch.Tensor | None = None, group: int = 128,
                 x_scale: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """D = bf16(silu(X @ W1.T) * (X @ W3.T)) for a few tokens, the weights as in linear_w4()."""
    if stream is not None:
        return _on(stream, ffn_gated_w4, X, W1q, scales1, W3q, scales3, zeros1, zeros3, group, x_scale, out)
    return (_module or binding()).ffn_gated_w4(X, W1q, scales1, W3q, scales3, zeros1, zeros3, group, x_scale, out)


def dropout(X: torch.Tensor, p: float, seed, offset: int = 0, R: torch.Tensor | None = None,
            out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """D = bf16(keep * X / (1 - p) + R); keep is drawn from (seed, offset) and the element's place alone, so the
    gradient of X is dropout(dD, p, seed, offset).  `seed`: a number, or a CUDA int64 tensor {seed, offset} that
    is read when the kernel runs (a replayed graph then draws what the tensor holds)."""
    if stream is not None:
        return _on(stream, dropout, X, p, seed, offset, R, out)
    return (_module or binding()).dropout(X, p, seed, offset, R, out)


def add_rms_norm(X: torch.Tensor, weight: torch.Tensor, R: torch.Tensor | None = None, eps: float = 1e-6,
                 p: float = 0.0, seed=0, offset: int = 0, out: torch.Tensor | None = None,
                 h: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(Y, H, rstd): H = dropout(X) + R (p, seed, offset as in dropout()), rstd = 1 / sqrt(mean(H^2) + eps) of
    each row, Y = H * rstd * weight from H before its rounding.  Without R and dropout H is X itself."""
    if stream is not None:
        return _on(stream, add_rms_norm, X, weight, R, eps, p, seed, offset, out, h)
    return (_module or binding()).add_rms_norm(X, weight, R, eps, p, seed, offset, out, h)


def add_rms_norm_q8(X: torch.Tensor, weight: torch.Tensor, R: torch.Tensor | None = None, eps: float = 1e-6,
                    scale_group: int = 0, out: torch.Tensor | None = None, h: torch.Tensor | None = None,
                    stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(Q, scale, H): the norm's output in float8_e4m3fn, Q * scale = Y.  scale is [M,1] (scale_group = 0) or
    [M,ceil(D/128)] (scale_group = 128), as linear_w4() and ffn_gated_w4() take it."""
    if stream is not None:
        return _on(stream, add_rms_norm_q8, X, weight, R, eps, scale_group, out, h)
    return (_module or binding()).add_rms_norm_q8(X, weight, R, eps, scale_group, out, h)


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
    if stream is not None:
        return _on(stream, add_rms_norm_backward, dY, H, weight, rstd, dH, p, seed, offset, workspace)
    return (_module or binding()).add_rms_norm_backward(dY, H, weight, rstd, dH, p, seed, offset, workspace)


def add_layer_norm(X: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
                   R: torch.Tensor | None = None, eps: float = 1e-5, p: float = 0.0, seed=0, offset: int = 0,
                   out: torch.Tensor | None = None, h: torch.Tensor | None = None,
                   stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """(Y, H, mean, rstd): H = dropout(X) + R (p, seed, offset as in dropout()), the mean and
    rstd = 1 / sqrt(variance + eps) of each row, Y = (H - mean) * rstd * weight + bias from H before its rounding.
    Without R and dropout H is X itself."""
    if stream is not None:
        return _on(stream, add_layer_norm, X, weight, bias, R, eps, p, seed, offset, out, h)
    return (_module or binding()).add_layer_norm(X, weight, bias, R, eps, p, seed, offset, out, h)


def add_layer_norm_backward_workspace_bytes(M: int, D: int) -> int:
    """Bytes of workspace add_layer_norm_backward() needs on the current device."""
    n = ctypes.c_size_t(0)
    _check(lib().gb_add_layer_norm_backward_workspace_bytes(M, D, ctypes.byref(n)))
    return int(n.value)


def add_layer_norm_backward(dY: torch.Tensor, H: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor,
                            rstd: torch.Tensor, dH: torch.Tensor | None = None, p: float = 0.0, seed=0,
                            offset: int = 0, workspace: torch.Tensor | None = None,
                            stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """(dX, dR, dweight, dbias) of add_layer_norm() from the gradient dY of Y and (optionally) dH of H, with H, mean
    and rstd as it returned them and the same p, seed and offset.  Without dropout dX is dR; dweight and dbias
    [D] are fp32."""
    if stream is not None:
        return _on(stream, add_layer_norm_backward, dY, H, weight, mean, rstd, dH, p, seed, offset, workspace)
    return (_module or binding()).add_layer_norm_backward(dY, H, weight, mean, rstd, dH, p, seed, offset, workspace)


def moe_ffn_gated_workspace_bytes(T: int, I: int, E: int, top_k: int) -> int:  # noqa: E741
    """Bytes of workspace moe_ffn_gated() needs for T tokens, E experts and I inner columns."""
    n = ctypes.c_size_t(0)
    _check(lib().gb_moe_ffn_gated_workspace_bytes(T, I, E, top_k, ctypes.byref(n)))
    return int(n.value)


def moe_ffn_gated(X: torch.Tensor, router: torch.Tensor, W1: torch.Tensor, W3: torch.Tensor, W2: torch.Tensor,
                  top_k: int, R: torch.Tensor | None = None, renormalize: bool = True, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(D, ids, weights) of a mixture-of-experts layer for a few tokens: each row of X [T,D] goes to the top_k experts
    of the largest logits X @ router.T (router [E,D]; equal ones: the lower expert first), and
    D = bf16(R + sum_j weights[:,j] * (silu(X @ W1[e].T) * (X @ W3[e].T)) @ W2[e].T), e = ids[:,j], with W1 and W3
    [E,I,D] and W2 [E,D,I].  weights [T,top_k] fp32 are the logits' softmax, over the chosen experts (renormalize) or
    over all; ids [T,top_k] int32 are in falling order of the logits."""
    if stream is not None:
        return _on(stream, moe_ffn_gated, X, router, W1, W3, W2, top_k, R, renormalize, out, workspace)
    return (_module or binding()).moe_ffn_gated(X, router, W1, W3, W2, top_k, R, renormalize, out, workspace)


def lora_workspace_bytes(M: int, N: int, K: int, r: int) -> int:
    """Bytes of workspace lora() needs for M rows of K and N columns and a rank of r."""
    n = ctypes.c_size_t(0)
    _check(lib().gb_lora_workspace_bytes(M, N, K, r, ctypes.byref(n)))
    return int(n.value)


def lora(X: torch.Tensor, A: torch.Tensor, B: torch.Tensor, ids: torch.Tensor, scale: torch.Tensor | None = None,
         R: torch.Tensor | None = None, act: str = "none", out: torch.Tensor | None = None,
         workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """D = bf16(act(R + scale[id] * (X @ A[id].T) @ B[id].T)), id = ids[row]: low-rank adapters of many requests at once
    (X [M,K], A [adapters,r,K], B [adapters,N,r], ids [M] int32, scale [adapters] fp32 or None, R [M,N] or None).  A
    row whose id is outside 0 .. adapters - 1 has none: act(R).  Rows of X, A and B begin on 16 bytes: a B of a rank that
    is no multiple of 8 is refused unless its rows are padded (torch.zeros(adapters, N, 8, ...)[:, :, :r]).
    Beside a projection: linear(X, W, bias,
    R=lora(X, A, B, ids, scale)), or before its activation lora(..., R=linear(X, W, bias), act=...)."""
    if stream is not None:
        return _on(stream, lora, X, A, B, ids, scale, R, act, out, workspace)
    if act not in ACT:
        raise ValueError(f"act must be one of {sorted(ACT)}")
    return (_module or binding()).lora(X, A, B, ids, scale, R, ACT[act], out, workspace)
