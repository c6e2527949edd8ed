"""Products grouped by expert over ragged rows, and their gradients: the experts of a layer that is trained, or served with
bf16 or fp16 weights.

Thin wrappers of tmoe_grouped_linear, tmoe_grouped_grad_x and tmoe_grouped_grad_w (include/tmoe.h holds the formulas).
Rows are sorted by expert: with the ids of `router.topk`,

    route = torch.sort(ids.flatten() + 1, stable=True).indices          # dropped routes (id -1) first
    offsets = torch.bincount(ids.flatten() + 1, minlength=E + 1).cumsum(0)   # [E + 1]
    y = grouped.linear(x[route // k], w, offsets)

expert e has the rows [offsets[e], offsets[e + 1]); rows outside every group give zeros. `linear` records a gradient where x
or w requires one (first derivatives only; tensors with a forward-mode tangent are refused; an fp32 gradient that arrives is
rounded to x's type, which the products take); `grad_x` and `grad_w` are the same gradients as explicit calls, for programs
without autograd and for hipGraph capture. The 8-bit form is `mxfp8.grouped_linear`."""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import native
from .layer import _in_forward_mode, _int32, _launch, _one_gpu, _refuse_duals, _same_device
from .native import check, lib

_DTYPES = {torch.bfloat16: native.BF16, torch.float16: native.F16, torch.float32: native.F32}
_IDS = {torch.int32: native.IDS_I32, torch.int64: native.IDS_I64}
_BITS16 = (torch.bfloat16, torch.float16)


@functools.lru_cache(maxsize=512)
def _config(E: int, K: int, N: int, dtype, out_dtype, ids_dtype):
    _int32(E=E, K=K, N=N)
    cfg = ctypes.byref(native.GroupedConfig(E, K, N, _DTYPES[dtype], _DTYPES[out_dtype], _IDS[ids_dtype]))   # kept alive
    # refused here, before a wrapper allocates outputs of these sizes: without rows nothing is launched
    check(lib.tmoe_grouped_linear(cfg, None, None, None, 0, None, None), "grouped configuration")
    return cfg


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


def _check(a, a_name: str, b, b_name: str, b_dim: int, offsets, out_dtype) -> None:
    """Raise ValueError for operands that do not fit: a [R, .], b [E, ., .] or [R, .], of one 16-bit type, contiguous."""
    for t, name, dim in ((a, a_name, 2), (b, b_name, b_dim)):
        if not isinstance(t, torch.Tensor) or t.dim() != dim:
            raise ValueError(f"{name}: expected a tensor with {dim} dimensions")
        if t.dtype is not torch.bfloat16 and t.dtype is not torch.float16:
            raise ValueError(f"{name}: dtype {t.dtype}, expected torch.bfloat16 or torch.float16")
        if not t.is_contiguous():
            raise ValueError(f"{name}: must be contiguous")
    if b.dtype is not a.dtype:
        raise ValueError(f"{b_name}: dtype {b.dtype}, {a_name} has {a.dtype}")
    if out_dtype is not None and out_dtype is not a.dtype and out_dtype is not torch.float32:
        raise ValueError(f"out_dtype: {out_dtype}, expected {a.dtype} or torch.float32")
    _check_offsets(offsets, b.shape[0] if b_dim == 3 else None)
    if a.shape[0] >= 2 ** 31:
        _int32(R=a.shape[0])


# What a call checks apart from the tensors' layout and device depends on these alone: once for each combination.
@functools.lru_cache(maxsize=512)
def _fitting(op: str, a_cols: int, a_dtype, b_shape, b_dtype, off_shape, off_dtype, out_dtype):
    """(configuration, columns or shape of the result, its type) of operands that fit, else None."""
    out = a_dtype if out_dtype is None else out_dtype
    if a_dtype not in _BITS16 or b_dtype is not a_dtype or off_dtype not in _IDS or len(off_shape) != 1 or \
            (out is not a_dtype and out is not torch.float32):
        return None
    E = off_shape[0] - 1
    if op == "grad_w":
        N, K, shape, fits = a_cols, b_shape[-1], (E, a_cols, b_shape[-1]), len(b_shape) == 1 and E >= 1
    elif len(b_shape) != 3:
        return None
    elif op == "linear":
        N, K, shape, fits = b_shape[1], b_shape[2], b_shape[1], b_shape[2] == a_cols and b_shape[0] == E and E >= 1
    else:
        N, K, shape, fits = b_shape[1], b_shape[2], b_shape[2], b_shape[1] == a_cols and b_shape[0] == E and E >= 1
    return (_config(E, K, N, a_dtype, out, off_dtype), shape, out) if fits else None


def _rows_by_weights(op: str, fn, where: str, a, a_name: str, w, offsets, out_dtype):
    """linear and grad_x: a [R, .] and w [E, N, K]."""
    plan = None
    if isinstance(a, torch.Tensor) and isinstance(w, torch.Tensor) and isinstance(offsets, torch.Tensor) and a.dim() == 2:
        plan = _fitting(op, a.shape[1], a.dtype, w.shape, w.dtype, offsets.shape, offsets.dtype, out_dtype)
    R = a.shape[0] if plan is not None else 0
    if plan is None or R >= 2 ** 31 or not (a.is_contiguous() and w.is_contiguous() and offsets.is_contiguous()
                                            and _one_gpu(a, w, offsets)):
        _check(a, a_name, w, "w", 3, offsets, out_dtype)
        if op == "linear" and w.shape[2] != a.shape[1]:
            raise ValueError(f"w: rows of {w.shape[2]} values, {a_name} has {a.shape[1]}")
        if op == "grad_x" and w.shape[1] != a.shape[1]:
            raise ValueError(f"w: {w.shape[1]} rows an expert, {a_name} has {a.shape[1]} columns")
        _same_device([(a_name, a), ("w", w), ("offsets", offsets)])
        raise ValueError("operands do not fit")
    cfg, cols, out = plan
    y = a.new_empty((R, cols), dtype=out)
    _launch(a.get_device(), fn, where, cfg, a.data_ptr(), w.data_ptr(), offsets.data_ptr(), R, y.data_ptr())
    return y


def _linear(x, w, offsets, out_dtype):
    return _rows_by_weights("linear", lib.tmoe_grouped_linear, "tmoe_grouped_linear", x, "x", w, offsets, out_dtype)


def grad_x(dy: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, out_dtype=None) -> torch.Tensor:
    """dx [R, K] of dy [R, N] and w [E, N, K]: dx_r = W_e^T dy_r, zeros in rows outside every group."""
    if _in_forward_mode():
        _refuse_duals(dy=dy, w=w)
    return _rows_by_weights("grad_x", lib.tmoe_grouped_grad_x, "tmoe_grouped_grad_x", dy, "dy", w, offsets, out_dtype)


def grad_w(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor, out_dtype=None) -> torch.Tensor:
    """dw [E, N, K] of dy [R, N] and x [R, K]: the sum over an expert's rows of dy_r x_r^T, zeros for one without rows."""
    if _in_forward_mode():
        _refuse_duals(dy=dy, x=x)
    plan = None
    if isinstance(dy, torch.Tensor) and isinstance(x, torch.Tensor) and isinstance(offsets, torch.Tensor) and \
            dy.dim() == 2 and x.dim() == 2 and dy.shape[0] == x.shape[0]:
        plan = _fitting("grad_w", dy.shape[1], dy.dtype, x.shape[1:], x.dtype, offsets.shape, offsets.dtype, out_dtype)
    R = x.shape[0] if plan is not None else 0
    if plan is None or R >= 2 ** 31 or not (dy.is_contiguous() and x.is_contiguous() and offsets.is_contiguous()
                                            and _one_gpu(dy, x, offsets)):
        _check(x, "x", dy, "dy", 2, offsets, out_dtype)
        if x.shape[0] != dy.shape[0]:
            raise ValueError(f"x: {x.shape[0]} rows, dy has {dy.shape[0]}")
        _same_device([("dy", dy), ("x", x), ("offsets", offsets)])
        raise ValueError("operands do not fit")
    cfg, shape, out = plan
    dw = x.new_empty(shape, dtype=out)
    _launch(x.get_device(), lib.tmoe_grouped_grad_w, "tmoe_grouped_grad_w", cfg, dy.data_ptr(), x.data_ptr(),
            offsets.data_ptr(), R, dw.data_ptr())
    return dw


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets, out_dtype):
        y = _linear(x, w, offsets, out_dtype)
        track_x, track_w = ctx.needs_input_grad[:2]
        ctx.save_for_backward(x if track_w else None, w if track_x else None, offsets)   # dw reads x, dx reads w
        ctx.dtype = x.dtype
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        dy = dy.to(ctx.dtype).contiguous()        # an fp32 gradient is rounded once: the products take x's type
        if dy.data_ptr() % 16:                    # a part of a larger gradient: the products copy from 16-byte addresses
            dy = dy.clone()
        dx = grad_x(dy, w, offsets) if ctx.needs_input_grad[0] else None
        dw = grad_w(dy, x, offsets) if ctx.needs_input_grad[1] else None
        return dx, dw, None, None


def linear(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, out_dtype=None) -> torch.Tensor:
    """y [R, N] of x [R, K] and w [E, N, K] (both bf16 or both fp16), offsets [E + 1]: y_r = W_e x_r for the rows of expert
    e, zeros in rows outside every group; in x's type or fp32 (out_dtype)."""
    if _in_forward_mode():
        _refuse_duals(x=x, w=w)
    if torch.is_grad_enabled() and (getattr(x, "requires_grad", False) or getattr(w, "requires_grad", False)):
        return _Linear.apply(x, w, offsets, out_dtype)
    return _linear(x, w, offsets, out_dtype)
