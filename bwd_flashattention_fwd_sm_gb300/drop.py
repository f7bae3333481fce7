"""PyTorch-facing binding of ln_dropout (include/gbln.h): dropout whose mask is
computed from a seed, an offset and an element's place, and never stored.

Argument marshalling only; the computation runs in libgbattn.so.  There is no
CPU path: a tensor that is not on a CUDA device raises.
"""

from __future__ import annotations

import torch

from ._lib import LnDropoutC, LnParamsC, check
from .rows import DTYPES, as_rows, current_device, current_stream, elsewhere, library, like

_MOD = 1 << 64


def dropout_params(p, seed, offset, rng, device):
    """The C block of a dropout, or None where p is 0."""
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"dropout p={p}: must be between 0 and 1")
    if rng is not None and (rng.dtype not in (torch.int64, torch.uint64) or rng.numel() != 2
                            or rng.device != device or not rng.is_contiguous()):
        raise ValueError("rng must be a contiguous int64 tensor of 2 numbers, (seed, offset), on x's device")
    if p == 0.0:
        return None
    return LnDropoutC(p, int(seed) % _MOD, int(offset) % _MOD, None if rng is None else rng.data_ptr())


def dropout(x, p: float, *, seed: int = 0, offset: int = 0, rng=None, stream=None, out=None):
    """Dropout of x [..., cols], a bf16 or float32 CUDA tensor; of a gradient, its backward pass.

    An element is dropped (0) with the probability p, rounded to a multiple of 2^-16, else scaled by the
    inverse of the rate that stays.  Which ones follows from ``seed``, ``offset``, the row (leading axes taken
    together) and the column: the same numbers give the same mask, here and in layernorm_residual and its
    backward pass; each dropout of a step needs an offset of its own.  rng: an int64 CUDA
    tensor (seed, offset), added to the two (modulo 2^64) and read on the device when the kernel runs, so
    that a captured graph follows new values in it.  The sums decide: where a step's dropouts have the offsets
    0 .. n - 1, rng's offset has to grow by n at least from step to step, or masks come again.  out: a contiguous tensor like x, which may be x itself."""
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    dtype = DTYPES.get(x.dtype)
    if dtype is None:
        raise ValueError("x must be bfloat16 or float32")
    if x.dim() == 0:
        raise ValueError("x must have at least one axis")
    if out is not None and (out.shape != x.shape or out.dtype != x.dtype or out.device != x.device
                            or not out.is_contiguous()):
        raise ValueError("out must be contiguous and match x in shape, dtype and device")
    device = x.device
    if stream is not None or device.index != current_device():
        with elsewhere(device, stream, (x, rng, out)):
            return dropout(x, p, seed=seed, offset=offset, rng=rng, out=out)
    d = dropout_params(p, seed, offset, rng, device) or LnDropoutC()
    cols = x.shape[-1]
    src, stride = as_rows(x, cols)
    y = like(x) if out is None else out
    n = y.numel()
    if n:
        c = LnParamsC(n // cols, cols, stride, cols, cols, cols, 0.0, dtype)
        check(library().ln_dropout(c, d, src.data_ptr(), y.data_ptr(), current_stream(device.index)), "ln_dropout")
    return y
