"""Trellis-quantized routed MoE layer for MI355X (gfx950): HIP kernels behind a C ABI.

Import `trellis_quantized_moe_tmoe_amd.layer` for the torch-facing wrapper (it loads libtmoe.so and
fails if the library is not built), `trellis_quantized_moe_tmoe_amd.router` for the ids and weights it takes
(top-k, balance loss, gradients), `trellis_quantized_moe_tmoe_amd.mxfp4` for MXFP4 quantisation, its dense product
and its expert layer, `norm` for the RMS norm with the residual's addition, `grouped` for bf16 and fp16 products grouped
by expert with their gradients, `mxfp8` for MXFP8 quantisation and the grouped product of such operands, and `trellis_quantized_moe_tmoe_amd.workloads` for seeded inputs.
"""
__all__ = ["grouped", "layer", "mxfp4", "mxfp8", "native", "norm", "router", "workloads"]
