"""GB300 (sm_103a) weight-only quantized linear layer (W4A16, W4A8 and W8), and what
lies between its calls in a decode step: head norms with rotation, an 8-bit key /
value cache with its attention, and a mixture of experts on W4 weights.

The compute lives in libw4q.so (CUDA kernels behind the C ABI of
include/w4q.h); ``w4q`` is its thin Python binding.
"""
from . import w4q  # noqa: F401
from .w4q import (W4QError, device_error, kv8_append, kv8_attention, kv8_read,  # noqa: F401
                  kv8_workspace_bytes, moe_w4a16, moe_workspace_bytes, packed_bytes,
                  qk_norm_rope, split_choice,
                  w4_pack_weights, w4_unpack_weights, w4a8_gemm, w4a8_gemm_rowscale,
                  w4a8_group_dots, w4a8_group_dots_rowscale, w4a8_quantize_act,
                  w4a8_quantize_act_rowscale, w4a16_gemm, w8_gemv, workspace_bytes)
