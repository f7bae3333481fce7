"""gbattn: fused multi-head attention forward and backward for GB300 (sm_103a).

The computation lives in libgbattn.so (hand-written CUDA, C ABI in
include/gbattn.h, include/gbln.h and include/gbkv4.h); this package is its thin PyTorch binding.
"""

from .attention import (BlockMask, Fp8Operands, SeqLens, attn_bwd, attn_fwd, attn_fwd_fp8, get_status, make_params,
                        quantize_fp8)
from .kv4 import Kv4Cache, attn_fwd_kv4, kv4_read, kv4_write
from .layernorm import layernorm_residual

__all__ = ["attn_fwd", "attn_bwd", "BlockMask", "SeqLens", "get_status", "make_params", "layernorm_residual",
           "quantize_fp8", "attn_fwd_fp8", "Fp8Operands", "Kv4Cache", "kv4_write", "kv4_read", "attn_fwd_kv4"]
