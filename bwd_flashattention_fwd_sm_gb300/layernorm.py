"""PyTorch-facing binding of include/gbln.h: fused dropout + residual add + LayerNorm
over the rows of a CUDA tensor, and its backward pass.

Argument marshalling only; the computation runs in libgbattn.so.  There is no
CPU path: a tensor that is not on a CUDA device raises.
"""

from __future__ import annotations

import torch

from . import _lib
from ._lib import LnBwdParamsC, LnParamsC, check
from .attention import _workspace
from .drop import dropout_params
from .rows import DTYPES, as_rows, on_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _cols(t):
    """The last axis' length."""
    if t.dim() == 0 or t.shape[-1] == 0:
        raise ValueError("a row needs at least one column")
    return t.shape[-1]


def _check_weight(name, t, cols):
    if t is not None and (t.dtype != torch.float32 or t.numel() != cols or not t.is_cuda):
        raise ValueError(f"{name} must be a float32 CUDA tensor of {cols} elements")


def layernorm_residual(x, residual=None, gamma=None, beta=None, *, eps: float = 1e-5, return_sum: bool = True,
                       return_stats: bool = False, dropout_p: float = 0.0, seed: int = 0, offset: int = 0, rng=None,
                       stream=None):
    """y = LayerNorm(D(x) + residual) * gamma + beta over the last dimension, D the dropout (see ``dropout`` for
    its arguments; none by default).

    x, residual: bf16 or float32 CUDA tensors of the same shape [..., cols];
    gamma, beta: float32 [cols] or None (1 and 0).
    Returns y, plus h = D(x) + residual if ``return_sum`` and (mean, rstd) per row
    (float32) if ``return_stats``.
    """
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    dtype = DTYPES.get(x.dtype)
    if dtype is None:
        raise ValueError("x must be bfloat16 or float32")
    cols = _cols(x)
    if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype
                                 or residual.device != x.device):
        raise ValueError("residual must match x in shape, dtype and device")
    _check_weight("gamma", gamma, cols)
    _check_weight("beta", beta, cols)
    d = dropout_params(dropout_p, seed, offset, rng, x.device)

    def call(handle):
        a, a_stride = as_rows(x, cols)
        r, r_stride = (None, cols) if residual is None else as_rows(residual, cols)
        g = None if gamma is None else gamma.contiguous()
        b = None if beta is None else beta.contiguous()
        rows = x.numel() // cols
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        h = torch.empty_like(y) if return_sum else None
        mean, rstd = (torch.empty((2, rows), dtype=torch.float32, device=x.device).unbind(0) if return_stats
                      else (None, None))
        p = LnParamsC(rows, cols, a_stride, r_stride, cols, cols, float(eps), dtype)
        check(_lib.load().ln_dropout_residual_fwd(p, d, a.data_ptr(), _ptr(r), _ptr(g), _ptr(b), y.data_ptr(),
                                                  _ptr(h), _ptr(mean), _ptr(rstd), handle), "ln_residual_fwd")
        out = [y]
        if return_sum:
            out.append(h)
        if return_stats:
            out += [mean, rstd]
        return out[0] if len(out) == 1 else tuple(out)

    return on_stream(x.device, stream, (x, residual, gamma, beta, rng), call)


def layernorm_residual_bwd(dy, h, mean, rstd, gamma=None, dh=None, *, dropout_p: float = 0.0, seed: int = 0,
                           offset: int = 0, rng=None, weight_grads: bool = True, stream=None, workspace=None):
    """The backward pass of layernorm_residual: (dx, dresidual, dgamma, dbeta).

    dy: the gradient at y; h, mean, rstd: the forward pass's (h is x itself where there was neither residual nor
    dropout); gamma: its gamma; dh: the gradient that arrives at h by another way (the residual stream going
    on), or None.  dropout_p, seed, offset, rng: the forward pass's, rng with the values it had then.
    dx and dresidual have dy's type; without dropout they are one tensor.  dgamma and dbeta are float32
    [cols], None where ``weight_grads`` is false; the same bits every time.  workspace: as for attn_bwd."""
    if not dy.is_cuda:
        raise ValueError("dy must be a CUDA tensor")
    dtype = DTYPES.get(dy.dtype)
    if dtype is None:
        raise ValueError("dy must be bfloat16 or float32")
    device = dy.device
    for name, t in (("h", h), ("dh", dh)):
        if t is not None and (t.shape != dy.shape or t.dtype != dy.dtype or t.device != device):
            raise ValueError(f"{name} must match dy in shape, dtype and device")
    cols = _cols(dy)
    rows = dy.numel() // cols
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t.dtype != torch.float32 or t.numel() != rows or t.device != device:
            raise ValueError(f"{name} must be a float32 CUDA tensor of {rows} elements")
    _check_weight("gamma", gamma, cols)
    d = dropout_params(dropout_p, seed, offset, rng, device)

    def call(handle):
        lib = _lib.load()
        a, a_stride = as_rows(dy, cols)
        b, b_stride = as_rows(h, cols)
        c, c_stride = (None, cols) if dh is None else as_rows(dh, cols)
        m, s = mean.contiguous(), rstd.contiguous()
        g = None if gamma is None else gamma.contiguous()
        dr = torch.empty(dy.shape, dtype=dy.dtype, device=device)
        dx = dr if d is None else torch.empty_like(dr)
        p = LnBwdParamsC(rows, cols, a_stride, c_stride, b_stride, cols, cols, dtype)
        dgamma = dbeta = ws = None
        need = 0
        if weight_grads:
            dgamma, dbeta = torch.empty((2, cols), dtype=torch.float32, device=device).unbind(0)
            need = lib.ln_residual_bwd_workspace_size(p)
            ws = _workspace(need, device, workspace)
        check(lib.ln_residual_bwd(p, d, a.data_ptr(), _ptr(c), b.data_ptr(), m.data_ptr(), s.data_ptr(), _ptr(g),
                                  None if d is None else dx.data_ptr(), dr.data_ptr(), _ptr(dgamma), _ptr(dbeta),
                                  _ptr(ws), need, handle), "ln_residual_bwd")
        return dx, dr, dgamma, dbeta

    return on_stream(device, stream, (dy, h, mean, rstd, gamma, dh, rng, workspace), call)
