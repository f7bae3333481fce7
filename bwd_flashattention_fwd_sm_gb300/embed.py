"""PyTorch-facing binding of the embedding table (include/gbembed.h): lookup with
scaling, and the table's gradient.

Argument marshalling only; the computation runs in libgbattn.so.  There is no
CPU path: a tensor that is not on a CUDA device raises.
"""

from __future__ import annotations

import torch

from ._lib import EmbeddingParamsC, check
from .attention import _workspace
from .rows import DTYPES, as_rows, current_device, current_stream, elsewhere, library


def _check_ids(ids, device):
    if ids.dtype not in (torch.int32, torch.int64) or ids.device != device:
        raise ValueError("ids must be an int32 or int64 tensor on the other arguments' device")


def embedding(weight, ids, *, scale: float = 1.0, stream=None):
    """y[..., :] = scale * weight[ids[...], :], in float32 and rounded once.

    weight: bf16 or float32 [vocab, dim]; ids: int32 or int64 of any shape.  An id outside the table gives a row
    of zeros and is recorded (get_status: ATTN_ERR_DEVICE_BOUNDS)."""
    if not weight.is_cuda:
        raise ValueError("weight must be a CUDA tensor")
    dtype = DTYPES.get(weight.dtype)
    if dtype is None or weight.dim() != 2:
        raise ValueError("weight must be bfloat16 or float32, [vocab, dim]")
    device = weight.device
    _check_ids(ids, device)
    if stream is not None or device.index != current_device():
        with elsewhere(device, stream, (weight, ids)):
            return embedding(weight, ids, scale=scale)
    vocab, dim = weight.shape
    weight, w_stride = as_rows(weight, dim)
    ids = ids.contiguous()
    y = torch.empty((*ids.shape, dim), dtype=weight.dtype, device=device)
    p = EmbeddingParamsC(ids.numel(), vocab, dim, dim, w_stride, scale, dtype, dtype, ids.dtype == torch.int64, 0, -1)
    check(library().attn_embedding_fwd(p, weight.data_ptr(), ids.data_ptr(), y.data_ptr(),
                                       current_stream(device.index)), "attn_embedding_fwd")
    return y


def embedding_bwd(dy, ids, num_embeddings: int, *, scale: float = 1.0, padding_id: int | None = None, dtype=None,
                  stream=None, workspace=None, out=None):
    """The gradient of embedding's table [num_embeddings, dim]: row v is scale times the sum of dy's rows whose id is v.

    dy: bf16 or float32 [..., dim], ids: as in the lookup, of dy's leading shape.  padding_id: a token that
    gives no gradient.  dtype: the gradient's type, dy's own by default.  out: a tensor [num_embeddings, dim]
    with contiguous rows, apart from dy and ids, to add the gradient to (tied weights, several steps in one gradient); rows
    that no token names are left as they are.  Sums are float32 in an order that ids, sizes and types decide: the same bits
    every time.  An id outside the table is recorded as in the lookup and gives nothing.  workspace: as for attn_bwd."""
    if not dy.is_cuda:
        raise ValueError("dy must be a CUDA tensor")
    device = dy.device
    if out is not None:
        if dtype is not None and dtype != out.dtype:
            raise ValueError("dtype is not out's")
        if out.dim() != 2 or out.shape[0] != num_embeddings or out.shape[1] != dy.shape[-1] or out.device != device:
            raise ValueError("out must be [num_embeddings, dim] on dy's device")
        if as_rows(out, out.shape[1])[0] is not out:
            raise ValueError("out's rows must be contiguous and apart")
    grad = dy.dtype if out is None and dtype is None else dtype if out is None else out.dtype
    if dy.dtype not in DTYPES or grad not in DTYPES:
        raise ValueError("dy and its gradient must be bfloat16 or float32")
    _check_ids(ids, device)
    if dy.shape[:-1] != ids.shape:
        raise ValueError(f"dy {tuple(dy.shape)} does not match ids {tuple(ids.shape)}")
    if padding_id is not None and padding_id < 0:
        raise ValueError(f"padding_id={padding_id}: must be a token (not counted from the table's end) or None")
    if stream is not None or device.index != current_device():
        with elsewhere(device, stream, (dy, ids, workspace, out)):
            return embedding_bwd(dy, ids, num_embeddings, scale=scale, padding_id=padding_id, dtype=grad,
                                 workspace=workspace, out=out)
    lib = library()
    dim = dy.shape[-1]
    dy, stride = as_rows(dy, dim)
    ids = ids.contiguous()
    dw, w_stride = out, dim
    if out is None:
        dw = torch.empty((num_embeddings, dim), dtype=grad, device=device)
    else:
        w_stride = as_rows(out, dim)[1]
    p = EmbeddingParamsC(ids.numel(), num_embeddings, dim, stride, w_stride, scale, DTYPES[dy.dtype], DTYPES[grad],
                         ids.dtype == torch.int64, out is not None, -1 if padding_id is None else padding_id)
    need = lib.attn_embedding_bwd_workspace_size(p)
    ws = _workspace(need, device, workspace)
    check(lib.attn_embedding_bwd(p, dy.data_ptr(), ids.data_ptr(), dw.data_ptr(), None if ws is None else ws.data_ptr(),
                                 need, current_stream(device.index)), "attn_embedding_bwd")
    return dw
