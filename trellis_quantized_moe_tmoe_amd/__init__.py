"""Trellis-quantized routed MoE layer for MI355X (gfx950): HIP kernels behind a C ABI.

Import `trellis_quantized_moe_tmoe_amd.layer` for the torch-facing wrapper (it loads libtmoe.so and
fails if the library is not built), `trellis_quantized_moe_tmoe_amd.router` for the ids and weights it takes
(top-k, balance loss, gradients), `trellis_quantized_moe_tmoe_amd.mxfp4` for MXFP4 quantisation, its dense product
and its expert layer, and `trellis_quantized_moe_tmoe_amd.workloads` for seeded inputs.
"""
__all__ = ["layer", "mxfp4", "native", "router", "workloads"]
