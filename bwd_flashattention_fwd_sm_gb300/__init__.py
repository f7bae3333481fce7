"""gbattn: fused multi-head attention forward and backward for GB300 (sm_103a).

The computation lives in libgbattn.so (hand-written CUDA, C ABI in
include/gbattn.h, include/gbln.h, include/gbkv4.h and include/gbembed.h); this package is its thin PyTorch
binding.
"""

from .attention import (BlockMask, Fp8Operands, SeqLens, attn_bwd, attn_fwd, attn_fwd_fp8, get_status, make_params,
                        quantize_fp8)
from .drop import dropout
from .embed import embedding, embedding_bwd
from .kv4 import Kv4Cache, attn_fwd_kv4, kv4_read, kv4_write
from .layernorm import layernorm_residual, layernorm_residual_bwd

__all__ = ["attn_fwd", "attn_bwd", "BlockMask", "SeqLens", "get_status", "make_params", "layernorm_residual",
           "quantize_fp8", "attn_fwd_fp8", "Fp8Operands", "Kv4Cache", "kv4_write", "kv4_read", "attn_fwd_kv4",
           "layernorm_residual_bwd", "dropout", "embedding", "embedding_bwd"]
