"""PyTorch-facing binding of the 4-bit key/value cache (include/gbkv4.h): writing
keys and values into it, reading them back, and attention over it.

Argument marshalling only; the computation runs in libgbattn.so.  There is no
CPU path: a tensor that is not on a CUDA device raises.

A cache is a set of pages; which pages hold a sequence is the caller's, as an int32
``block_table`` [batch, max_pages], and so is how many positions it holds, as int32
``lens`` [batch] (the positions that a call deals with included).  Both are read on
the device when the kernels run, so a captured graph follows new values in them.
Every call deals with the newest tokens of each sequence:

  fixed length     k, v [B, Hkv, S, D], q, o [B, Hq, S, D]: S tokens of each
                   sequence, the positions lens - S .. lens - 1 (those below 0 are
                   padding); lse [B, Hq, S] float32
  variable length  k, v [T, Hkv, D], q, o [T, Hq, D] with ``seqlens`` (a SeqLens)
                   giving the packed rows' starts; lse [Hq, T] float32

Tensors may be views: any strides whose last one is 1 and whose others are whole
16-byte steps are used as they are; others are copied first.
"""

from __future__ import annotations

import math

import numpy as np
import torch

from . import _lib
from ._lib import ATTN_BF16, ATTN_F32, Kv4ParamsC, check
from .attention import SeqLens, _workspace

GROUP = 64  # values that share one (s, b) pair

_DTYPES = {torch.float32: ATTN_F32, torch.bfloat16: ATTN_BF16}


class Kv4Cache:
    """The arrays of a 4-bit cache, all contiguous on one device:

    k_codes, v_codes  uint8    [n_pages, heads_kv, page_size, head_dim / 2]
    k_scale, v_scale  bfloat16 [n_pages, heads_kv, page_size, head_dim / 64, 2]
    """

    def __init__(self, k_codes, v_codes, k_scale, v_scale):
        if k_codes.dim() != 4 or k_scale.dim() != 5:
            raise ValueError("codes are [n_pages, heads_kv, page_size, head_dim / 2] and scales "
                             "[n_pages, heads_kv, page_size, head_dim / 64, 2]")
        self.n_pages, self.heads_kv, self.page_size, half = k_codes.shape
        self.head_dim = 2 * half
        self.device = k_codes.device
        for name, t, shape, dtype in (
                ("k_codes", k_codes, tuple(k_codes.shape), torch.uint8),
                ("v_codes", v_codes, tuple(k_codes.shape), torch.uint8),
                ("k_scale", k_scale, (*k_codes.shape[:3], self.head_dim // GROUP, 2), torch.bfloat16),
                ("v_scale", v_scale, (*k_codes.shape[:3], self.head_dim // GROUP, 2), torch.bfloat16)):
            if not t.is_cuda or t.device != self.device:
                raise ValueError(f"{name}: gbattn runs on CUDA tensors of one device only")
            if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape}")
        self._arrays = (k_codes, k_scale, v_codes, v_scale)
        self._pointers = tuple(t.data_ptr() for t in self._arrays)

    k_codes = property(lambda self: self._arrays[0])
    k_scale = property(lambda self: self._arrays[1])
    v_codes = property(lambda self: self._arrays[2])
    v_scale = property(lambda self: self._arrays[3])

    @classmethod
    def empty(cls, n_pages, heads_kv, page_size, head_dim, device=None) -> "Kv4Cache":
        """A cache whose positions hold nothing yet (their memory is not initialised)."""
        if head_dim not in (64, 128, 256):
            raise ValueError(f"head_dim={head_dim}: only 64, 128 and 256 are implemented")
        dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        rows = (n_pages, heads_kv, page_size)
        codes = [torch.empty((*rows, head_dim // 2), dtype=torch.uint8, device=dev) for _ in "kv"]
        scales = [torch.empty((*rows, head_dim // GROUP, 2), dtype=torch.bfloat16, device=dev) for _ in "kv"]
        return cls(codes[0], codes[1], scales[0], scales[1])


def _usable(t):
    """t itself if the library can take its strides and address, else a copy."""
    step = 16 // t.element_size()
    strides = t.stride()
    if strides[-1] == 1 and t.data_ptr() % 16 == 0 and all(s % step == 0 for s in strides[:-1]):
        return t
    return t.clone(memory_format=torch.contiguous_format)


def _rows_overlap(shape, strides):
    """Whether two rows (the last axis, of stride 1) of such a tensor share an element."""
    axes = sorted((s, n) for s, n in zip(strides[:-1], shape[:-1]) if n > 1)
    span, apart = shape[-1], True  # each axis steps over all that the ones before it span: the usual layouts
    for s, n in axes:
        if s < shape[-1]:
            return True
        apart = apart and s >= span
        span += (n - 1) * s
    if apart:
        return False
    # all steps along the shorter axes: is there one along the longest that leads back?
    (far, most), *rest = sorted(axes, key=lambda a: -a[1])
    d = np.zeros(1, np.int64)
    for s, n in rest:
        d = (d[:, None] + np.arange(1 - n, n, dtype=np.int64) * s).ravel()
    for k in range(-1, 2):
        to = -(d // far) + k
        hit = (np.abs(d + to * far) < shape[-1]) & (np.abs(to) < most)
        hit[len(d) // 2] &= to[len(d) // 2] != 0  # a row and itself
        if hit.any():
            return True
    return False


def _share(a, b):
    """Whether two tensors of one shape have rows that share an element (unequal strides: whether they begin together)."""
    if a.numel() == 0 or a.data_ptr() == b.data_ptr():
        return a.numel() > 0
    apart = abs(a.data_ptr() - b.data_ptr()) // a.element_size()
    return a.stride() == b.stride() and _rows_overlap((2, *a.shape), (apart, *a.stride()))


def _fits(t):
    """Whether an output tensor can be written in place."""
    return t.data_ptr() % 16 == 0 and t.stride(-1) == 1 and all(
        s % (16 // t.element_size()) == 0 for s in t.stride()[:-1]) and not _rows_overlap(t.shape, t.stride())


def _params(x, y, cache, block_table, lens, seqlens, heads_q, heads_kv, scale=0.0, causal=True):
    """The C parameter block.  x and y have equal shapes and types (checked by the callers)."""
    dev = x.device
    if not x.is_cuda or dev != cache.device:
        raise ValueError("gbattn runs on CUDA tensors only, all of the cache's device")
    dtype = _DTYPES.get(x.dtype)
    if dtype is None:
        raise ValueError(f"unsupported dtype {x.dtype}: float32 or bfloat16")
    if x.shape[-1] != cache.head_dim:
        raise ValueError(f"head_dim {x.shape[-1]} does not match the cache's {cache.head_dim}")
    if heads_kv != cache.heads_kv:
        raise ValueError(f"{heads_kv} KV heads do not match the cache's {cache.heads_kv}")
    if block_table.dtype != torch.int32 or lens.dtype != torch.int32 or block_table.dim() != 2 or lens.dim() != 1:
        raise ValueError("block_table [batch, max_pages] and lens [batch] must be int32")
    if block_table.device != dev or lens.device != dev:
        raise ValueError("block_table and lens must be on the cache's device")
    batch, max_pages = block_table.shape
    if lens.shape[0] != batch:
        raise ValueError(f"lens has {lens.shape[0]} sequences, block_table {batch}")
    if (max_pages > 1 and block_table.stride(1) != 1) or (batch > 1 and lens.stride(0) != 1):
        raise ValueError("block_table's rows and lens must be contiguous")
    xs, ys = x.stride(), y.stride()
    if seqlens is not None:
        if x.dim() != 3:
            raise ValueError("variable length expects packed rows [T, heads, D]")
        if seqlens.n_seqs != batch or x.shape[0] != seqlens.total:
            raise ValueError(f"seqlens has {seqlens.n_seqs} sequences and {seqlens.total} rows, expected {batch} "
                             f"and {x.shape[0]}")
        if seqlens.device.device != dev:
            raise ValueError("seqlens must be on the cache's device")
        return Kv4ParamsC(batch, heads_q, heads_kv, cache.head_dim, cache.page_size, cache.n_pages, max_pages,
                          seqlens.max_len, block_table.data_ptr(), block_table.stride(0), lens.data_ptr(),
                          seqlens.device.data_ptr(), seqlens.host.ctypes.data, 0, xs[1], xs[0], 0, ys[1], ys[0],
                          scale, dtype, 1 if causal else 0)
    if x.dim() != 4:
        raise ValueError("fixed length expects [B, heads, S, D]")
    if x.shape[0] != batch:
        raise ValueError(f"{x.shape[0]} sequences, block_table has {batch}")
    return Kv4ParamsC(batch, heads_q, heads_kv, cache.head_dim, cache.page_size, cache.n_pages, max_pages,
                      x.shape[2], block_table.data_ptr(), block_table.stride(0), lens.data_ptr(), None, None,
                      xs[0], xs[1], xs[2], ys[0], ys[1], ys[2], scale, dtype, 1 if causal else 0)


def _on(cache, stream, call, *args):
    """call(cache, *args, handle) with the cache's device current and, where ``stream`` is given, that
    stream: what is allocated for the call then belongs to the stream that it runs on, and
    what comes from another stream is not given away before the call has run."""
    device = cache.device
    index = device.index
    if stream is None and index == torch.cuda.current_device():
        return call(cache, *args, torch._C._cuda_getCurrentRawStream(index))
    with torch.cuda.device(device), torch.cuda.stream(stream):
        if stream is not None:
            given = [*cache._arrays]
            for t in args:
                given += t if isinstance(t, (tuple, list)) else [t.device] if isinstance(t, SeqLens) else [t]
            for t in given:
                if isinstance(t, torch.Tensor) and t.is_cuda:
                    t.record_stream(stream)
        return call(cache, *args, torch._C._cuda_getCurrentRawStream(index))


def kv4_write(cache: Kv4Cache, k, v, block_table, lens, *, seqlens: SeqLens | None = None, stream=None) -> Kv4Cache:
    """Quantises the newest tokens' k and v to 4 bits and stores them.  Returns the cache.

    Pages that a sequence shares with another must not be written to."""
    if v.shape != k.shape or v.dtype != k.dtype or v.device != k.device:
        raise ValueError("v must match k in shape, dtype and device")
    return _on(cache, stream, _write, k, v, block_table, lens, seqlens)


def _write(cache, k, v, block_table, lens, seqlens, stream):
    k, v = _usable(k), _usable(v)
    heads = k.shape[1] if k.dim() > 1 else 0
    p = _params(k, v, cache, block_table, lens, seqlens, heads, heads)
    check(_lib.load().attn_kv4_write(p, k.data_ptr(), v.data_ptr(), *cache._pointers, stream), "attn_kv4_write")
    return cache


def kv4_read(cache: Kv4Cache, block_table, lens, seqlen: int | None = None, *, seqlens: SeqLens | None = None,
             dtype=torch.bfloat16, stream=None, out=None):
    """The newest tokens' keys and values, (k, v): ``seqlen`` of each sequence, or with
    ``seqlens`` a packed batch.  Rows of padding are 0.  out: a (k, v) pair to write to,
    two tensors apart."""
    if (seqlen is None) == (seqlens is None):
        raise ValueError("give either seqlen (a fixed number of tokens) or seqlens (a packed batch)")
    return _on(cache, stream, _read, block_table, lens, seqlen, seqlens, dtype, out)


def _read(cache, block_table, lens, seqlen, seqlens, dtype, out, stream):
    H, D = cache.heads_kv, cache.head_dim
    shape = (block_table.shape[0], H, int(seqlen), D) if seqlens is None else (seqlens.total, H, D)
    if out is None:
        k = torch.empty(shape, dtype=dtype, device=cache.device)
        v = torch.empty_like(k)
    else:
        k, v = out
        for t in out:
            if tuple(t.shape) != shape or t.dtype != k.dtype or t.device != cache.device or not _fits(t):
                raise ValueError(f"out must be two CUDA tensors of shape {shape} and one dtype, rows contiguous, "
                                 "16-byte aligned and apart")
        if _share(k, v):
            raise ValueError("out: k and v share memory")
    p = _params(k, v, cache, block_table, lens, seqlens, H, H)
    check(_lib.load().attn_kv4_read(p, *cache._pointers, k.data_ptr(), v.data_ptr(), stream), "attn_kv4_read")
    return k, v


def attn_fwd_kv4(q, cache: Kv4Cache, block_table, lens, *, causal=True, scale=None, seqlens: SeqLens | None = None,
                 stream=None, workspace=None, out=None):
    """O, LSE of the newest tokens' queries over all that the cache holds.  Returns (o, lse).

    causal: a token sees the positions up to its own; else all of its sequence's.  workspace: a tensor
    without gaps on the cache's device, taken if it is large enough.  out: O's tensor, which may be q itself."""
    return _on(cache, stream, _attend, q, block_table, lens, causal, scale, seqlens, workspace, out)


def _attend(cache, q, block_table, lens, causal, scale, seqlens, workspace, out, stream):
    lib = _lib.load()
    q = _usable(q)
    if out is None:
        o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    else:
        o = out
        if o.shape != q.shape or o.dtype != q.dtype or o.device != q.device or not _fits(o):
            raise ValueError("out must match q in shape, dtype and device, rows contiguous, 16-byte aligned and apart")
    heads = q.shape[1] if q.dim() > 1 else 0
    p = _params(q, o, cache, block_table, lens, seqlens, heads, cache.heads_kv,
                float(scale) if scale is not None else 1.0 / math.sqrt(cache.head_dim), causal)
    lse = torch.empty(q.shape[:3] if seqlens is None else (heads, q.shape[0]), dtype=torch.float32, device=q.device)
    need = lib.attn_kv4_workspace_size(p)
    ws = _workspace(need, q.device, workspace)
    check(lib.attn_fwd_kv4(p, q.data_ptr(), *cache._pointers, o.data_ptr(), lse.data_ptr(),
                           None if ws is None else ws.data_ptr(), need, stream), "attn_fwd_kv4")
    return o, lse
