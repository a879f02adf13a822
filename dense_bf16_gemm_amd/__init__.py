"""MI355X-native bf16 GEMM: MatmulOp / LinearOp forms with fused epilogues,
and the decoder-layer operators beside them: RMS norm with the residual's
addition, and linear layers with 4-bit and 8-bit weights.

The operations run in hand-written HIP kernels for gfx950 behind the C ABI in
``include/mm.h`` (``libmm.so``); this package only marshals arguments to it.
The library is loaded on first use and its absence is an error.
"""
from .gemm import (bmm, ffn_glu, ffn_swiglu, linear, linear_batched, linear_preact, matmul,  # noqa: F401
                   release_workspaces)
from .decoder import linear_q8, linear_w4, pack_w4, rms_norm, rms_norm_backward, rms_norm_q8  # noqa: F401
from .binding import describe_config, set_config  # noqa: F401
