"""ExTernD greedy sequential ternary ALS on B200 (sm_100a).

The factorization runs in the CUDA library ``libexternd.so`` (C ABI in
include/externd.h); this package is its Python binding plus the seeded
synthetic workload generators.
"""
from .api import (ExterndError, Factors, Int4Weights, NOALLOC_SCRATCH_BYTES, STATUS, Trace, debug_component,  # noqa: F401
                  debug_halfstep, debug_start_trits, debug_wait_fault,
                  factor, factor_batched, factor_block, factor_noalloc, factor_weighted, inference_layout, last_stats, matvec, pack_mask_sign,
                  gated, gated_backward, gated_forward, int4_dequantize, int4_gated, int4_matvec, int4_quantize, int4_row_bytes, pack_int4, unpack_int4,
                  pack_trits, rank, reconstruct, strerror, transpose_trits, trit_bytes, unpack_trits)

__all__ = [
    "ExterndError", "Factors", "NOALLOC_SCRATCH_BYTES", "STATUS", "factor_noalloc", "debug_halfstep", "debug_start_trits", "debug_component", "debug_wait_fault", "Trace", "factor", "factor_batched", "factor_block",
    "last_stats", "pack_trits", "rank", "reconstruct", "strerror", "trit_bytes", "unpack_trits",
    "transpose_trits", "inference_layout", "matvec", "pack_mask_sign", "factor_weighted",
    "Int4Weights", "int4_quantize", "int4_dequantize", "int4_matvec", "int4_gated", "int4_row_bytes", "pack_int4",
    "unpack_int4", "gated", "gated_forward", "gated_backward",
]
