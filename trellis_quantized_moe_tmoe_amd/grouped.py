"""Products grouped by expert over ragged rows, and their gradients: the experts of a layer that is trained, or served with
bf16 or fp16 weights.

Thin wrappers of tmoe_grouped_linear, tmoe_grouped_grad_x and tmoe_grouped_grad_w (include/tmoe.h holds the formulas).
Rows are sorted by expert: with the ids of `router.topk`,

    route = torch.sort(ids.flatten() + 1, stable=True).indices          # dropped routes (id -1) first
    offsets = torch.bincount(ids.flatten() + 1, minlength=E + 1).cumsum(0)   # [E + 1]
    y = grouped.linear(x[route // k], w, offsets)

expert e has the rows [offsets[e], offsets[e + 1]); rows outside every group give zeros. `linear` records a gradient where x
or w requires one (first derivatives only; tensors with a forward-mode tangent are refused); `grad_x` and `grad_w` are the
same gradients as explicit calls, for programs without autograd and for hipGraph capture. The 8-bit form is
`mxfp8.grouped_linear`."""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import native
from .layer import _fits, _in_forward_mode, _int32, _launch, _one_gpu, _refuse_duals, _require, _same_device
from .native import lib

_DTYPES = {torch.bfloat16: native.BF16, torch.float16: native.F16, torch.float32: native.F32}
_IDS = {torch.int32: native.IDS_I32, torch.int64: native.IDS_I64}


@functools.lru_cache(maxsize=512)
def _config(E: int, K: int, N: int, dtype, out_dtype, ids_dtype):
    _int32(E=E, K=K, N=N)
    return ctypes.byref(native.GroupedConfig(E, K, N, _DTYPES[dtype], _DTYPES[out_dtype], _IDS[ids_dtype]))


def _matrix(t, name: str, dim: int = 2):
    if not isinstance(t, torch.Tensor) or t.dim() != dim:
        raise ValueError(f"{name}: expected a tensor with {dim} dimensions")
    if t.dtype is not torch.bfloat16 and t.dtype is not torch.float16:
        raise ValueError(f"{name}: dtype {t.dtype}, expected torch.bfloat16 or torch.float16")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _check_offsets(offsets, E: Optional[int] = None) -> int:
    """Number of experts."""
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.dtype not in _IDS:
        raise ValueError("offsets: expected a 1-D tensor [E + 1] of torch.int32 or torch.int64")
    if not offsets.is_contiguous():
        raise ValueError("offsets: must be contiguous")
    n = offsets.shape[0] - 1
    if n < 1 or (E is not None and n != E):
        raise ValueError(f"offsets: {n + 1} values, expected E + 1" + (f" = {E + 1}" if E is not None else ""))
    return n


def _check_out(out_dtype, dtype):
    if out_dtype is None or out_dtype is dtype:
        return dtype
    if out_dtype is not torch.float32:
        raise ValueError(f"out_dtype: {out_dtype}, expected {dtype} or torch.float32")
    return out_dtype


def _same_dtype(a, name: str, b, other: str) -> None:
    if a.dtype is not b.dtype:
        raise ValueError(f"{name}: dtype {a.dtype}, {other} has {b.dtype}")


def _linear(x, w, offsets, out_dtype):
    _matrix(x, "x")
    _matrix(w, "w", 3)
    _same_dtype(w, "w", x, "x")
    (R, K), (E, N, Kw) = x.shape, w.shape
    if Kw != K:
        raise ValueError(f"w: rows of {Kw} values, x has {K}")
    _check_offsets(offsets, E)
    if R >= 2 ** 31:
        _int32(R=R)
    out = _check_out(out_dtype, x.dtype)
    if not _one_gpu(x, w, offsets):
        _same_device([("x", x), ("w", w), ("offsets", offsets)])
    dev = x.device
    y = torch.empty((R, N), dtype=out, device=dev)
    _launch(dev.index, lib.tmoe_grouped_linear, "tmoe_grouped_linear", _config(E, K, N, x.dtype, out, offsets.dtype),
            x.data_ptr(), w.data_ptr(), offsets.data_ptr(), R, y.data_ptr())
    return y


def grad_x(dy: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, out_dtype=None) -> torch.Tensor:
    """dx [R, K] of dy [R, N] and w [E, N, K]: dx_r = W_e^T dy_r, zeros in rows outside every group."""
    if _in_forward_mode():
        _refuse_duals(dy=dy, w=w)
    _matrix(dy, "dy")
    _matrix(w, "w", 3)
    _same_dtype(w, "w", dy, "dy")
    (R, N), (E, Nw, K) = dy.shape, w.shape
    if Nw != N:
        raise ValueError(f"w: {Nw} rows an expert, dy has {N} columns")
    _check_offsets(offsets, E)
    if R >= 2 ** 31:
        _int32(R=R)
    out = _check_out(out_dtype, dy.dtype)
    if not _one_gpu(dy, w, offsets):
        _same_device([("dy", dy), ("w", w), ("offsets", offsets)])
    dev = dy.device
    dx = torch.empty((R, K), dtype=out, device=dev)
    _launch(dev.index, lib.tmoe_grouped_grad_x, "tmoe_grouped_grad_x", _config(E, K, N, dy.dtype, out, offsets.dtype),
            dy.data_ptr(), w.data_ptr(), offsets.data_ptr(), R, dx.data_ptr())
    return dx


def grad_w(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor, out_dtype=None) -> torch.Tensor:
    """dw [E, N, K] of dy [R, N] and x [R, K]: the sum over an expert's rows of dy_r x_r^T, zeros for one without rows."""
    if _in_forward_mode():
        _refuse_duals(dy=dy, x=x)
    _matrix(dy, "dy")
    _matrix(x, "x")
    _same_dtype(dy, "dy", x, "x")
    (R, N), (Rx, K) = dy.shape, x.shape
    if Rx != R:
        raise ValueError(f"x: {Rx} rows, dy has {R}")
    E = _check_offsets(offsets)
    if R >= 2 ** 31:
        _int32(R=R)
    out = _check_out(out_dtype, x.dtype)
    if not _one_gpu(dy, x, offsets):
        _same_device([("dy", dy), ("x", x), ("offsets", offsets)])
    dev = dy.device
    dw = torch.empty((E, N, K), dtype=out, device=dev)
    _launch(dev.index, lib.tmoe_grouped_grad_w, "tmoe_grouped_grad_w", _config(E, K, N, x.dtype, out, offsets.dtype),
            dy.data_ptr(), x.data_ptr(), offsets.data_ptr(), R, dw.data_ptr())
    return dw


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets, out_dtype):
        y = _linear(x, w, offsets, out_dtype)
        ctx.save_for_backward(x, w, offsets)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        dy = dy.to(x.dtype).contiguous()          # an fp32 gradient is rounded once: the products take x's type
        dx = grad_x(dy, w, offsets) if ctx.needs_input_grad[0] else None
        dw = grad_w(dy, x, offsets) if ctx.needs_input_grad[1] else None
        return dx, dw, None, None


def linear(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, out_dtype=None) -> torch.Tensor:
    """y [R, N] of x [R, K] and w [E, N, K] (both bf16 or both fp16), offsets [E + 1]: y_r = W_e x_r for the rows of expert
    e, zeros in rows outside every group; in x's type or fp32 (out_dtype)."""
    if _in_forward_mode():
        _refuse_duals(x=x, w=w)
    if torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad for t in (x, w)):
        return _Linear.apply(x, w, offsets, out_dtype)
    return _linear(x, w, offsets, out_dtype)
