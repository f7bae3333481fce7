"""What the bindings of the row operators share: a tensor [..., cols] as rows, and the
stream and device that a call runs on."""

from __future__ import annotations

import torch

from . import _lib
from ._lib import ATTN_BF16, ATTN_F32

current_device = torch.cuda.current_device
current_stream = torch._C._cuda_getCurrentRawStream  # of a device's index, as the handle that the library takes

DTYPES = {torch.bfloat16: ATTN_BF16, torch.float32: ATTN_F32}


def as_rows(t, cols: int):
    """t itself, or a contiguous copy where its rows of ``cols`` elements are not contiguous or not a fixed
    number of elements apart, and that number."""
    if t.is_contiguous():
        return t, cols
    shape, stride = t.shape, t.stride()
    if t.dim() > 1 and (stride[-1] == 1 or cols == 1):
        step = rows = None
        for n, s in zip(reversed(shape[:-1]), reversed(stride[:-1])):
            if n == 1:
                continue
            if step is None:
                step, rows = s, n
            elif s == step * rows:
                rows *= n
            else:
                step = -1
                break
        if step is None:
            return t, cols
        if step >= cols:
            return t, step
    return t.contiguous(), cols


class elsewhere:
    """With ``device`` current and, where ``stream`` is given, that stream: what is allocated for a call then belongs
    to the stream that it runs on, and what comes from another stream (``tensors``) is not given away before
    the call has run."""

    def __init__(self, device, stream, tensors):
        if stream is not None and stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        self._device, self._stream, self._tensors = torch.cuda.device(device), torch.cuda.stream(stream), ()
        if stream is not None:
            self._tensors = [t for t in tensors if t is not None]
            self._on = stream
            for t in self._tensors:
                if t.device != device:
                    raise ValueError(f"a tensor is on {t.device}, the others on {device}")

    def __enter__(self):
        for t in self._tensors:  # first: what raises here must leave device and stream as they were
            t.record_stream(self._on)
        self._device.__enter__()
        self._stream.__enter__()

    def __exit__(self, *error):
        self._stream.__exit__(*error)
        self._device.__exit__(*error)


def like(t):
    """A new contiguous tensor of t's shape and type (on the host a microsecond faster than torch.empty)."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def library():
    """The loaded library."""
    return _lib._lib or _lib.load()
