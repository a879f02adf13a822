"""MI355X-native bf16 GEMM: MatmulOp / LinearOp forms with fused epilogues,
and the decoder-layer operators beside them: RMS norm and layer norm with the
residual's addition, linear layers with 4-bit and 8-bit weights or with an adapter per
row, and the mixture-of-experts FFN.

The operations run in hand-written HIP kernels for gfx950 behind the C ABI in
``include/mm.h`` (``libmm.so``); this package only marshals arguments to it.
The library is loaded on first use and its absence is an error.
"""
from .gemm import (bmm, ffn_glu, ffn_swiglu, linear, linear_batched, linear_preact, matmul,  # noqa: F401
                   release_workspaces)
from .decoder import (layer_norm, layer_norm_backward, linear_lora, linear_q8, linear_w4, moe_ffn,  # noqa: F401
                      pack_w4, rms_norm, rms_norm_backward, rms_norm_q8)
from .binding import describe_config, set_config  # noqa: F401
