"""What the bindings of the row operators share: a tensor [..., cols] as rows, and the
stream and device that a call runs on."""

from __future__ import annotations

import torch

from . import _lib
from ._lib import ATTN_BF16, ATTN_F32

current_device = torch.cuda.current_device
current_stream = torch._C._cuda_getCurrentRawStream  # of a device's index, as the handle that the library takes

_get_stream = torch._C._cuda_getCurrentStream  # of a device's index: (stream_id, device_index, device_type)


def _make_current(stream_id, device_index, device_type):
    torch._C._cuda_setStream(stream_id=stream_id, device_index=device_index, device_type=device_type)


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
    the call has run.  (What torch.cuda.stream does, in 1 us instead of 7: calls with a stream wait for the host.)"""

    def __init__(self, device, stream, tensors):
        self._device, self._stream, self._tensors = device, stream, ()
        if stream is not None:
            if stream.device != device:
                raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
            self._tensors = [t for t in tensors if t is not None]
            for t in self._tensors:
                if t.device != device:
                    raise ValueError(f"a tensor is on {t.device}, the others on {device}")

    def __enter__(self):
        for t in self._tensors:  # first: what raises here must leave device and stream as they were
            t.record_stream(self._stream)
        self._guard = None
        if self._device.index != current_device():
            self._guard = torch.cuda.device(self._device)
            self._guard.__enter__()
        if self._stream is not None:
            self._before = _get_stream(self._device.index)
            _make_current(self._stream.stream_id, self._stream.device_index, self._stream.device_type)

    def __exit__(self, *error):
        if self._stream is not None:
            _make_current(*self._before)
        if self._guard is not None:
            self._guard.__exit__(*error)


def like(t):
    """A new contiguous tensor of t's shape and type (on the host a microsecond faster than torch.empty)."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def library():
    """The loaded library."""
    return _lib._lib or _lib.load()
