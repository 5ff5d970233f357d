"""MI355X-native MoE layer hot path: layer or RMS norm -> gate -> routing
preprocessing -> dispatch-permute -> grouped SwiGLU MLP -> combine-unpermute.

Every step runs in the hand-written HIP kernels of ``libmoe_route.so``
(C ABI in ``include/moe_route.h``).  This package only marshals torch tensors
(device memory) and torch's current HIP stream into those calls.
"""
from ._abi import (BF16, F32, FP8E4M3_B128, INT4_G128, FLAG_BAD_EXPERT, FLAG_CAPACITY, FLAG_DUPLICATE, FLAG_OUT_ROWS,
                   ROUTE_DENSE_I16, ROUTE_DENSE_I32, ROUTE_SPARSE_BOOL, MoeError, lib)
from .api import (BufferRing, Dispatcher, RmsNorm, assert_no_overflow, capacity_from_rows, layer_norm,
                  layer_norm_backward, layer_norm_backward_scratch_bytes, out_rows_bound, rms_norm, rms_norm_backward,
                  rms_norm_backward_scratch_bytes, routing_bytes)

__all__ = ["BufferRing", "Dispatcher", "RmsNorm", "assert_no_overflow", "capacity_from_rows", "layer_norm",
           "layer_norm_backward", "layer_norm_backward_scratch_bytes", "out_rows_bound", "rms_norm",
           "rms_norm_backward", "rms_norm_backward_scratch_bytes", "routing_bytes", "MoeError", "lib", "BF16", "F32", "FP8E4M3_B128", "INT4_G128", "ROUTE_DENSE_I16", "ROUTE_DENSE_I32",
           "ROUTE_SPARSE_BOOL", "FLAG_CAPACITY", "FLAG_OUT_ROWS", "FLAG_BAD_EXPERT", "FLAG_DUPLICATE"]
