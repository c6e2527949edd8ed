"""MXFP4 (E2M1 elements, one E8M0 scale per 32): quantisation, the dense product and the expert layer.

Thin wrappers of tmoe_mxfp4_quantize, tmoe_mxfp4_dequantize, tmoe_linear_mxfp4 and tmoe_forward_mxfp4
(include/tmoe.h holds the format and the formulas). Codes and scales are uint8 tensors [..., K/2] and
[..., K/32]; weights are rows of output features, quantised along their input features:
`ExpertWeights(*quantize(w1), *quantize(w2))` with w1 [E, 2I, H] (gate rows first) and w2 [E, H, I].

Forward only: no call here has a backward. Activations, weights of routes and outputs that require a gradient are
refused (detach them, or call under torch.no_grad()); a leaf parameter can be quantised as it is."""
from __future__ import annotations

import ctypes
from typing import Optional

import torch
from torch.autograd.graph import increment_version

from . import native
from .layer import _BITS16, _check_scratch, _fits, _in_forward_mode, _int32, _launch, _no_gradient, _one_gpu, \
    _refuse_duals, _require, _same_device
from .native import check, lib

_DTYPES = {torch.float32: native.F32, torch.bfloat16: native.BF16, torch.float16: native.F16}
_OUT = {torch.float32: native.F32, torch.bfloat16: native.BF16}


def _out_dtype(dtype) -> int:
    if dtype not in _OUT:
        raise ValueError(f"out_dtype: {dtype}, expected torch.float32 or torch.bfloat16")
    return _OUT[dtype]


def quantize(x: torch.Tensor):
    """(codes uint8 [..., K/2], scales uint8 [..., K/32]) of fp32, bf16 or fp16 values [..., K], K a multiple of 32."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x: expected a tensor [..., K]")
    if x.grad_fn is not None:                     # a parameter itself may be quantised: nothing lies behind it
        _no_gradient(x=x)
    elif _in_forward_mode():
        _refuse_duals(x=x)
    lead, K = x.shape[:-1], x.shape[-1]
    if x.dtype not in _DTYPES or not x.is_contiguous():
        _require(x, "x", x.shape, tuple(_DTYPES))
    if K == 0 or K % 32:
        raise ValueError(f"x: the last dimension is {K}, expected a multiple of 32")
    _int32(K=K)
    if not x.is_cuda:
        _same_device([("x", x)])
    dev = x.device
    codes = torch.empty((*lead, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((*lead, K // 32), dtype=torch.uint8, device=dev)
    _launch(dev.index, lib.tmoe_mxfp4_quantize, "tmoe_mxfp4_quantize", x.data_ptr(), _DTYPES[x.dtype], x.numel() // K,
            K, codes.data_ptr(), scales.data_ptr())
    return codes, scales


def _operand(codes, scales, name: str, dim: Optional[int] = None) -> int:
    """K of an MXFP4 tensor, after checking its two parts against each other."""
    if not isinstance(codes, torch.Tensor) or codes.dim() < 1 or (dim is not None and codes.dim() != dim):
        raise ValueError(f"{name}: expected a tensor of codes" + (f" with {dim} dimensions" if dim else ""))
    shape = codes.shape
    K = 2 * shape[-1]
    if K == 0 or K % 32:
        raise ValueError(f"{name}: rows of {K} values, expected a multiple of 32")
    if dim == 2:
        _int32(K=K, rows=shape[0])
    else:
        _int32(K=K)
    if not (codes.dtype is torch.uint8 and codes.is_contiguous()):
        _require(codes, f"{name} codes", shape, (torch.uint8,))
    if not _fits(scales, (*shape[:-1], K // 32), torch.uint8):
        _require(scales, f"{name} scales", (*shape[:-1], K // 32), (torch.uint8,))
    return K


def dequantize(codes: torch.Tensor, scales: torch.Tensor, dtype=torch.float32) -> torch.Tensor:
    """The values [..., K] of codes [..., K/2] and scales [..., K/32], rounded once to `dtype`."""
    K = _operand(codes, scales, "x")
    if dtype not in _DTYPES:
        raise ValueError(f"dtype: {dtype}, expected one of {[str(d) for d in _DTYPES]}")
    if not _one_gpu(codes, scales):
        _same_device([("codes", codes), ("scales", scales)])
    dev = codes.device
    x = torch.empty((*codes.shape[:-1], K), dtype=dtype, device=dev)
    _launch(dev.index, lib.tmoe_mxfp4_dequantize, "tmoe_mxfp4_dequantize", codes.data_ptr(), scales.data_ptr(),
            x.numel() // K, K, _DTYPES[dtype], x.data_ptr())
    return x


def linear(x_codes: torch.Tensor, x_scales: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
           out_dtype=torch.float32, y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [T, N] = X W^T of MXFP4 X [T, K] and W [N, K] (fp32 sums, rounded once to out_dtype)."""
    K = _operand(x_codes, x_scales, "x", 2)
    if _operand(w_codes, w_scales, "w", 2) != K:
        raise ValueError(f"w: rows of {2 * w_codes.shape[1]} values, x has {K}")
    T, N, out, dev = x_codes.shape[0], w_codes.shape[0], _out_dtype(out_dtype), x_codes.device
    given = y is not None
    if not given:
        y = torch.empty((T, N), dtype=out_dtype, device=dev)
    else:
        _no_gradient(y=y)
        if not _fits(y, (T, N), out_dtype):
            _require(y, "y", (T, N), (out_dtype,))
    if not _one_gpu(x_codes, x_scales, w_codes, w_scales, y):
        _same_device([("x codes", x_codes), ("x scales", x_scales), ("w codes", w_codes), ("w scales", w_scales),
                      ("y", y)])
    if given:
        increment_version(y)                      # a graph that saved y learns that it is written
    _launch(dev.index, lib.tmoe_linear_mxfp4, "tmoe_linear_mxfp4", x_codes.data_ptr(), x_scales.data_ptr(), T,
            w_codes.data_ptr(), w_scales.data_ptr(), K, N, out, y.data_ptr())
    return y


class ExpertWeights:
    """MXFP4 weights of E experts: w1 [E, 2I, H/2] and s1 [E, 2I, H/32] (gate rows first), w2 [E, H, I/2] and
    s2 [E, H, I/32], uint8 tensors on one GPU."""

    FIELDS = ("w1", "s1", "w2", "s2")

    def __init__(self, w1: torch.Tensor, s1: torch.Tensor, w2: torch.Tensor, s2: torch.Tensor):
        self.w1, self.s1, self.w2, self.s2 = w1, s1, w2, s2

    @property
    def c(self) -> native.Mxfp4Weights:
        return native.Mxfp4Weights(self.w1.data_ptr(), self.s1.data_ptr(), self.w2.data_ptr(), self.s2.data_ptr())


class ExpertPlan:
    """The routed expert layer with MXFP4 weights and activations (tmoe_forward_mxfp4)."""

    def __init__(self, hidden: int, inter: int, num_experts: int, top_k: int, max_tokens: int, ids_dtype=torch.int64,
                 out_dtype=torch.float32):
        if ids_dtype not in (torch.int32, torch.int64):
            raise ValueError(f"ids_dtype: {ids_dtype}, expected torch.int32 or torch.int64")
        _int32(hidden=hidden, inter=inter, num_experts=num_experts, top_k=top_k, max_tokens=max_tokens)
        self.config = native.Mxfp4Config(hidden, inter, num_experts, top_k, max_tokens,
                                         native.IDS_I64 if ids_dtype == torch.int64 else native.IDS_I32,
                                         _out_dtype(out_dtype))
        handle, sb = ctypes.c_void_p(), ctypes.c_size_t()
        check(lib.tmoe_mxfp4_plan(ctypes.byref(self.config), ctypes.byref(handle), ctypes.byref(sb)), "tmoe_mxfp4_plan")
        self.handle, self.scratch_bytes = handle, sb.value
        self.hidden, self.inter, self.num_experts, self.top_k = hidden, inter, num_experts, top_k
        self.max_tokens, self.ids_dtype, self.out_dtype = max_tokens, ids_dtype, out_dtype
        E, H, I = num_experts, hidden, inter
        self._weight_shapes = ((E, 2 * I, H // 2), (E, 2 * I, H // 32), (E, H, I // 2), (E, H, I // 32))

    def close(self):
        if getattr(self, "handle", None) and self.handle.value:
            lib.tmoe_mxfp4_plan_destroy(self.handle)
            self.handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def alloc_scratch(self, device="cuda") -> torch.Tensor:
        return torch.empty(self.scratch_bytes, dtype=torch.uint8, device=device)

    def forward(self, x: torch.Tensor, ids: torch.Tensor, w: torch.Tensor, weights: ExpertWeights,
                scratch: torch.Tensor, y: Optional[torch.Tensor] = None) -> torch.Tensor:
        """y [T, H] of x bf16 [T, H] (or its bit patterns), ids [T, k], w fp32 [T, k]."""
        _no_gradient(x=x, w=w, y=y)
        given = y is not None
        T = x.shape[0] if isinstance(x, torch.Tensor) and x.dim() == 2 else -1
        if not given and isinstance(x, torch.Tensor):
            y = torch.empty((max(T, 0), self.hidden), dtype=self.out_dtype, device=x.device)
        if not (0 <= T <= self.max_tokens and x.shape[1] == self.hidden and x.dtype in _BITS16 and x.is_contiguous()
                and _fits(ids, (T, self.top_k), self.ids_dtype) and _fits(w, (T, self.top_k), torch.float32)
                and _fits(y, (T, self.hidden), self.out_dtype) and isinstance(weights, ExpertWeights)
                and all(_fits(t, s, torch.uint8) for t, s in zip((weights.w1, weights.s1, weights.w2, weights.s2),
                                                                 self._weight_shapes))
                and isinstance(scratch, torch.Tensor) and scratch.dtype is torch.uint8 and scratch.dim() == 1
                and scratch.is_contiguous() and scratch.numel() >= self.scratch_bytes
                and _one_gpu(x, ids, w, y, scratch, weights.w1, weights.s1, weights.w2, weights.s2)):
            self.check_call(x, ids, w, weights, scratch, y)
        if given:
            increment_version(y)                  # a graph that saved y learns that it is written
        _launch(x.get_device(), lib.tmoe_forward_mxfp4, "tmoe_forward_mxfp4", self.handle, x.data_ptr(), ids.data_ptr(),
                w.data_ptr(), T, ctypes.byref(weights.c), y.data_ptr(), scratch.data_ptr(), scratch.numel())
        return y

    def check_call(self, x, ids, w, weights, scratch, y) -> None:
        """Raise ValueError unless the tensors match what the forward reads and writes, all contiguous and on
        one GPU device."""
        if not isinstance(x, torch.Tensor) or x.dim() != 2:
            raise ValueError("x: expected a 2-D tensor [T, H]")
        T = x.shape[0]
        if T > self.max_tokens:
            raise ValueError(f"x: {T} tokens, the plan holds at most {self.max_tokens}")
        H, k = self.hidden, self.top_k
        _require(x, "x", (T, H), _BITS16)
        _require(ids, "ids", (T, k), (self.ids_dtype,))
        _require(w, "w", (T, k), (torch.float32,))
        _require(y, "y", (T, H), (self.out_dtype,))
        if not isinstance(weights, ExpertWeights):
            raise ValueError("weights: expected ExpertWeights")
        for name, shape in zip(ExpertWeights.FIELDS, self._weight_shapes):
            _require(getattr(weights, name), name, shape, (torch.uint8,))
        _check_scratch(scratch, self.scratch_bytes)
        _same_device([("x", x), ("ids", ids), ("w", w), ("y", y), ("scratch", scratch)]
                     + [(n, getattr(weights, n)) for n in ExpertWeights.FIELDS])
