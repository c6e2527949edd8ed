"""RMS norm with the residual's addition, in the input's type or in MXFP8, and its gradients.

Thin wrappers of tmoe_rms_norm, tmoe_rms_norm_mxfp8 and tmoe_rms_norm_backward (include/tmoe.h holds the formulas).
`rms_norm` is what stands in front of the router and the experts; it records a gradient where an input requires one
(first derivatives only; tensors with a forward-mode tangent are refused). It flows from `y` and `h`; `rstd` is not
differentiable. `backward` is the same gradient as one explicit call, for programs without autograd and for hipGraph
capture. `rms_norm_mxfp8` gives the rows that `mxfp8.grouped_linear` takes; it is forward only."""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import native
from .layer import _fits, _in_forward_mode, _int32, _launch, _no_gradient, _one_gpu, _refuse_duals, _require, _same_device
from .native import check, lib

_ROWS = torch.contiguous_format                  # of outputs: empty_like takes half the time of empty with a shape
_DTYPES = {torch.float32: native.F32, torch.bfloat16: native.BF16, torch.float16: native.F16}


@functools.lru_cache(maxsize=256)
def _config(H: int, dtype, weight_dtype, eps: float):
    cfg = ctypes.byref(native.NormConfig(H, _DTYPES[dtype], _DTYPES[weight_dtype], eps))   # kept alive
    need = ctypes.c_size_t()
    # refused here, before a wrapper allocates outputs of these sizes
    check(lib.tmoe_rms_norm_backward_scratch(cfg, 0, ctypes.byref(need)), "norm configuration")
    return cfg


@functools.lru_cache(maxsize=256)
def _scratch_bytes(cfg, T: int) -> int:
    need = ctypes.c_size_t()
    check(lib.tmoe_rms_norm_backward_scratch(cfg, T, ctypes.byref(need)), "tmoe_rms_norm_backward_scratch")
    return need.value


def _rows(t, name: str, shape=None, dtype=None) -> int:
    """Row stride of a tensor [T, H] whose rows may be strided."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name}: expected a 2-D tensor [T, H]")
    if t.dtype not in _DTYPES or (dtype is not None and t.dtype is not dtype):
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype or [str(d) for d in _DTYPES]}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    (T, H), (row, step) = t.shape, t.stride()
    if T + H >= 2 ** 31:
        _int32(T=T, H=H)
    if T > 0 and ((H > 1 and step != 1) or (T > 1 and row < H)):
        raise ValueError(f"{name}: the values of a row must be adjacent and rows must not overlap")
    return row if T > 1 else H


def _inputs(x, weight, residual, eps):
    """(configuration, strides) of inputs that the library can take."""
    if isinstance(x, torch.Tensor) and isinstance(weight, torch.Tensor) and x.dim() == 2 and x.is_contiguous() and \
            weight.is_contiguous() and weight.get_device() == x.get_device() >= 0:
        T, H = x.shape                            # what most calls bring: one comparison
        if weight.shape == (H,) and (weight.dtype is x.dtype or weight.dtype is torch.float32) and T < 2 ** 31 and \
                H < 2 ** 31 and x.dtype in _DTYPES and (residual is None or (
                    _fits(residual, x.shape, x.dtype) and residual.get_device() == x.get_device())):
            return _config(H, x.dtype, weight.dtype, float(eps)), H, H
    stride = _rows(x, "x")
    H = x.shape[1]
    if not isinstance(weight, torch.Tensor) or weight.shape != (H,) or not weight.is_contiguous() or \
            (weight.dtype is not x.dtype and weight.dtype is not torch.float32):
        _require(weight, "weight", (H,), (x.dtype, torch.float32))
    res_stride = H
    if residual is not None:
        res_stride = _rows(residual, "residual", x.shape, x.dtype)
        if not _one_gpu(x, weight, residual):
            _same_device([("x", x), ("weight", weight), ("residual", residual)])
    elif not _one_gpu(x, weight):
        _same_device([("x", x), ("weight", weight)])
    return _config(H, x.dtype, weight.dtype, float(eps)), stride, res_stride


def _rms_norm(x, weight, residual, eps):
    cfg, stride, res_stride = _inputs(x, weight, residual, eps)
    T = x.shape[0]
    y = torch.empty_like(x, memory_format=_ROWS)
    rstd = x.new_empty(T, dtype=torch.float32)
    h, ph, pr = x, None, None
    if residual is not None:
        h = torch.empty_like(y)
        ph, pr = h.data_ptr(), residual.data_ptr()
    _launch(x.get_device(), lib.tmoe_rms_norm, "tmoe_rms_norm", cfg, x.data_ptr(), stride, pr, res_stride, weight.data_ptr(), T,
            y.data_ptr(), ph, rstd.data_ptr())
    return y, h, rstd


def backward(h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor, dy: torch.Tensor,
             dh: Optional[torch.Tensor] = None):
    """(dx [T, H] in h's type, dweight [H] in the weight's): dx is the gradient of x and of the residual alike. h and
    rstd as `rms_norm` returned them, dy [T, H] the gradient of y and dh that of h, both contiguous."""
    if _in_forward_mode():
        _refuse_duals(h=h, weight=weight, rstd=rstd, dy=dy, dh=dh)
    cfg, stride, _ = _inputs(h, weight, None, 0.0)
    shape, dtype = h.shape, h.dtype
    T = shape[0]
    if not _fits(rstd, (T,), torch.float32):
        _require(rstd, "rstd", (T,), (torch.float32,))
    if not _fits(dy, shape, dtype):
        _require(dy, "dy", shape, (dtype,))
    pdh, tensors = None, [weight, rstd, dy]
    if dh is not None:
        if not _fits(dh, shape, dtype):
            _require(dh, "dh", shape, (dtype,))
        pdh = dh.data_ptr()
        tensors.append(dh)
    if not _one_gpu(h, *tensors):
        _same_device([("h", h)] + list(zip(("weight", "rstd", "dy", "dh"), tensors)))
    dx = torch.empty_like(h, memory_format=_ROWS)
    dweight = torch.empty_like(weight)
    need = _scratch_bytes(cfg, T)
    scratch = h.new_empty(need, dtype=torch.uint8)
    _launch(h.get_device(), lib.tmoe_rms_norm_backward, "tmoe_rms_norm_backward", cfg, h.data_ptr(), stride, weight.data_ptr(),
            rstd.data_ptr(), dy.data_ptr(), pdh, T, dx.data_ptr(), dweight.data_ptr(), scratch.data_ptr(), need)
    return dx, dweight


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, h, rstd = _rms_norm(x, weight, residual, eps)
        track_x, _, track_residual = ctx.needs_input_grad[:3]
        if track_x or track_residual:
            ctx.save_for_backward(h, weight, rstd)
            ctx.mark_non_differentiable(rstd)
        else:                                     # dweight does not read the weight, which may change until then
            ctx.save_for_backward(h, None, rstd)
            ctx.weight = weight.detach()
            ctx.mark_non_differentiable(*([rstd] if residual is None else [rstd, h]))
        ctx.set_materialize_grads(False)
        return (y, rstd) if residual is None else (y, h, rstd)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, *rest):
        h, weight, rstd = ctx.saved_tensors
        if weight is None:
            weight = ctx.weight                   # for the size and type; dx is nobody's
        dh = rest[0] if len(rest) == 2 else None
        if dy is None:                            # only h was used
            return dh, None, dh, None
        dx, dweight = backward(h, weight, rstd, dy.contiguous(), None if dh is None else dh.contiguous())
        return dx, dweight, dx if len(rest) == 2 else None, None


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, eps: float = 1e-6):
    """(y [T, H], h [T, H], rstd fp32 [T]) of x [T, H] (fp32, bf16 or fp16; rows may be strided) and weight [H] (x's type
    or fp32): h = x + residual (x itself without one), y = h / sqrt(mean(h^2) + eps) * weight."""
    if _in_forward_mode():
        _refuse_duals(x=x, weight=weight, residual=residual)
    if torch.is_grad_enabled() and (getattr(x, "requires_grad", False) or getattr(weight, "requires_grad", False)
                                    or getattr(residual, "requires_grad", False)):
        out = _RmsNorm.apply(x, weight, residual, eps)
        return out if residual is not None else (out[0], x, out[1])
    return _rms_norm(x, weight, residual, eps)


def rms_norm_mxfp8(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, eps: float = 1e-6):
    """(codes uint8 [T, H], scales uint8 [T, H/32], h [T, H]): `rms_norm` with y rounded to MXFP8 straight from fp32.
    Forward only: tensors that require a gradient are refused."""
    _no_gradient(x=x, weight=weight, residual=residual)
    cfg, stride, res_stride = _inputs(x, weight, residual, eps)
    T, H = x.shape
    if H % 32:
        raise ValueError(f"x: rows of {H} values, expected a multiple of 32")
    codes = torch.empty_like(x, dtype=torch.uint8, memory_format=_ROWS)
    scales = x.new_empty((T, H // 32), dtype=torch.uint8)
    h, ph, pr = x, None, None
    if residual is not None:
        h = torch.empty_like(x, memory_format=_ROWS)
        ph, pr = h.data_ptr(), residual.data_ptr()
    _launch(x.get_device(), lib.tmoe_rms_norm_mxfp8, "tmoe_rms_norm_mxfp8", cfg, x.data_ptr(), stride, pr, res_stride,
            weight.data_ptr(), T, codes.data_ptr(), scales.data_ptr(), ph)
    return codes, scales, h
