"""What the bindings of the row operators share: a tensor [..., cols] as rows, and the
stream and device that a call runs on."""

from __future__ import annotations

import torch

from ._lib import ATTN_BF16, ATTN_F32

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


def on_stream(device, stream, tensors, call):
    """call(handle) with ``device`` current and, where ``stream`` is given, that stream: what is allocated for
    the call then belongs to the stream that it runs on, and what comes from another stream (``tensors``) is not
    given away before the call has run."""
    index = device.index
    if stream is None and index == torch.cuda.current_device():
        return call(torch._C._cuda_getCurrentRawStream(index))
    with torch.cuda.device(device), torch.cuda.stream(stream):
        if stream is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
        return call(torch._C._cuda_getCurrentRawStream(index))
