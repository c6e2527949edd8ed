"""MXFP8 (E4M3 elements, one E8M0 scale per 32): quantisation and the product grouped by expert.

Thin wrappers of tmoe_mxfp8_quantize, tmoe_mxfp8_dequantize and tmoe_grouped_linear_mxfp8 (include/tmoe.h holds the format
and the formulas). Codes and scales are uint8 tensors [..., K] and [..., K/32]; weights are rows of output features,
quantised along their input features: `mxfp8.quantize(w)` with w [E, N, K]. `norm.rms_norm_mxfp8` gives rows in this form.

Forward only: no call here has a backward. Tensors that require a gradient are refused (detach them, or call under
torch.no_grad()), leaves among them; only a torch.nn.Parameter can be quantised as it is."""
from __future__ import annotations

import torch

from . import native
from .grouped import _check_offsets, _config
from .layer import _fits, _in_forward_mode, _int32, _launch, _no_gradient, _one_gpu, _refuse_duals, _require, _same_device
from .native import lib

_DTYPES = {torch.float32: native.F32, torch.bfloat16: native.BF16, torch.float16: native.F16}


def quantize(x: torch.Tensor):
    """(codes uint8 [..., K], scales uint8 [..., K/32]) of fp32, bf16 or fp16 values [..., K], K a multiple of 32."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x: expected a tensor [..., K]")
    if x.requires_grad and not (x.is_leaf and isinstance(x, torch.nn.Parameter)):   # a parameter, as a program loads it
        _no_gradient(x=x)
    elif _in_forward_mode():
        _refuse_duals(x=x)
    K = x.shape[-1]
    if x.dtype not in _DTYPES or not x.is_contiguous():
        _require(x, "x", x.shape, tuple(_DTYPES))
    if K == 0 or K % 32:
        raise ValueError(f"x: the last dimension is {K}, expected a multiple of 32")
    _int32(K=K)
    if not x.is_cuda:
        _same_device([("x", x)])
    codes = torch.empty_like(x, dtype=torch.uint8)
    scales = x.new_empty((*x.shape[:-1], K // 32), dtype=torch.uint8)
    _launch(x.get_device(), lib.tmoe_mxfp8_quantize, "tmoe_mxfp8_quantize", x.data_ptr(), _DTYPES[x.dtype], x.numel() // K, K,
            codes.data_ptr(), scales.data_ptr())
    return codes, scales


def _operand(codes, scales, name: str, dim=None) -> int:
    """K of an MXFP8 tensor, after checking its two parts against each other."""
    if not isinstance(codes, torch.Tensor) or codes.dim() < 1 or (dim is not None and codes.dim() != dim):
        raise ValueError(f"{name}: expected a tensor of codes" + (f" with {dim} dimensions" if dim else ""))
    shape = codes.shape
    K = shape[-1]
    if K == 0 or K % 32:
        raise ValueError(f"{name}: rows of {K} values, expected a multiple of 32")
    _int32(K=K)
    if not (codes.dtype is torch.uint8 and codes.is_contiguous()):
        _require(codes, f"{name} codes", shape, (torch.uint8,))
    if not _fits(scales, (*shape[:-1], K // 32), torch.uint8):
        _require(scales, f"{name} scales", (*shape[:-1], K // 32), (torch.uint8,))
    return K


def dequantize(codes: torch.Tensor, scales: torch.Tensor, dtype=torch.float32) -> torch.Tensor:
    """The values [..., K] of codes [..., K] and scales [..., K/32], rounded once to `dtype`."""
    K = _operand(codes, scales, "x")
    if dtype not in _DTYPES:
        raise ValueError(f"dtype: {dtype}, expected one of {[str(d) for d in _DTYPES]}")
    if not _one_gpu(codes, scales):
        _same_device([("codes", codes), ("scales", scales)])
    x = torch.empty_like(codes, dtype=dtype)
    _launch(codes.get_device(), lib.tmoe_mxfp8_dequantize, "tmoe_mxfp8_dequantize", codes.data_ptr(), scales.data_ptr(),
            x.numel() // K, K, _DTYPES[dtype], x.data_ptr())
    return x


def grouped_linear(x_codes: torch.Tensor, x_scales: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
                   offsets: torch.Tensor, out_dtype=torch.bfloat16) -> torch.Tensor:
    """y [R, N] of MXFP8 x [R, K] and w [E, N, K], offsets [E + 1]: `grouped.linear` with 8-bit operands, rounded once to
    out_dtype, bf16 or fp32. The 8-bit matrix unit adds 16 neighbouring products at a time, each cut 13 bits below the largest of
    them, and those sums in fp32: fp32 results are unrounded, not more exact than that (include/tmoe.h)."""
    K = _operand(x_codes, x_scales, "x", 2)
    if _operand(w_codes, w_scales, "w", 3) != K:
        raise ValueError(f"w: rows of {w_codes.shape[2]} values, x has {K}")
    if out_dtype is not torch.bfloat16 and out_dtype is not torch.float32:
        raise ValueError(f"out_dtype: {out_dtype}, expected torch.bfloat16 or torch.float32")
    R, (E, N, _) = x_codes.shape[0], w_codes.shape
    _check_offsets(offsets, E)
    if R >= 2 ** 31:
        _int32(R=R)
    if not _one_gpu(x_codes, x_scales, w_codes, w_scales, offsets):
        _same_device([("x codes", x_codes), ("x scales", x_scales), ("w codes", w_codes), ("w scales", w_scales),
                      ("offsets", offsets)])
    cfg = _config(E, K, N, torch.bfloat16, out_dtype, offsets.dtype)
    y = x_codes.new_empty((R, N), dtype=out_dtype)
    _launch(x_codes.get_device(), lib.tmoe_grouped_linear_mxfp8, "tmoe_grouped_linear_mxfp8", cfg, x_codes.data_ptr(),
            x_scales.data_ptr(), w_codes.data_ptr(), w_scales.data_ptr(), offsets.data_ptr(), R, y.data_ptr())
    return y
