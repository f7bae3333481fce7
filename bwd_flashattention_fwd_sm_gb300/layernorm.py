"""PyTorch-facing binding of include/gbln.h: fused dropout + residual add + LayerNorm
over the rows of a CUDA tensor, and its backward pass.

Argument marshalling only; the computation runs in libgbattn.so.  There is no
CPU path: a tensor that is not on a CUDA device raises.
"""

from __future__ import annotations

import torch

from ._lib import SIZE_MAX, LnBwdParamsC, LnParamsC, check
from .attention import _workspace
from .drop import dropout_params
from .rows import DTYPES, as_rows, current_device, current_stream, elsewhere, library, like


def _ptr(t):
    return None if t is None else t.data_ptr()


def _cols(t):
    """The last axis' length."""
    if t.dim() == 0 or t.shape[-1] == 0:
        raise ValueError("a row needs at least one column")
    return t.shape[-1]


def _check_weight(name, t, cols, device):
    if t is not None and (t.dtype != torch.float32 or t.numel() != cols or t.device != device):
        raise ValueError(f"{name} must be a float32 CUDA tensor of {cols} elements on the other arguments' device")


def _at_vectors(x, x_stride, residual, r_stride, cols):
    """x and residual for the forward pass without dropout: views that put rows of whole 16-byte vectors at other
    places, copied where that pays.  The kernel takes the copies as vectors, the views by single elements.

    Rows that are multiples of 256 vectors, and those of more than 512, are summed in another order as
    vectors: always, so that a view gives the bits of its copy ([16384, 4096] bf16: 233 us with one copy, 369 with two, by
    elements 388 and 390; [64, 4096] some 15 and 10).  Others where one large bf16 tensor is to be copied ([16384, 1024]: 109
    us against 134, [1024, 1024] 17 both, [64, 1024] 14 against 9); two copies take longer there than the elements do
    (148 against 134), and so does one of float32 ([16384, 1028] 130 against 124)."""
    size = x.element_size()
    vectors, rest = divmod(cols * size, 16)
    if rest:
        return x, x_stride, residual, r_stride
    moved = [t is not None and step != cols and (t.data_ptr() | step * size) % 16 != 0
             for t, step in ((x, x_stride), (residual, r_stride))]
    if vectors % 256 == 0 or vectors > 512 or (sum(moved) == 1 and size == 2 and x.numel() >= 1 << 20):
        if moved[0]:
            x, x_stride = x.contiguous(), cols
        if moved[1]:
            residual, r_stride = residual.contiguous(), cols
    return x, x_stride, residual, r_stride


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
    device = x.device
    if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype or residual.device != device):
        raise ValueError("residual must match x in shape, dtype and device")
    _check_weight("gamma", gamma, cols, device)
    _check_weight("beta", beta, cols, device)
    if stream is not None or device.index != current_device():
        with elsewhere(device, stream, (x, residual, gamma, beta, rng)):
            return layernorm_residual(x, residual, gamma, beta, eps=eps, return_sum=return_sum,
                                      return_stats=return_stats, dropout_p=dropout_p, seed=seed, offset=offset, rng=rng)
    d = dropout_params(dropout_p, seed, offset, rng, device)
    y = like(x)
    x, x_stride = as_rows(x, cols)
    r_stride = cols
    if residual is not None:
        residual, r_stride = as_rows(residual, cols)
    if (x_stride != cols or r_stride != cols) and dropout_p < 2.0 ** -17:  # less than half a step of the rate
        x, x_stride, residual, r_stride = _at_vectors(x, x_stride, residual, r_stride, cols)
    gamma = None if gamma is None else gamma.contiguous()
    beta = None if beta is None else beta.contiguous()
    rows = x.numel() // cols
    h = mean = rstd = None
    if return_sum:
        h = torch.empty_like(y)
    if return_stats:
        mean = torch.empty(rows, dtype=torch.float32, device=device)
        rstd = torch.empty_like(mean)
    p = LnParamsC(rows, cols, x_stride, r_stride, cols, cols, float(eps), dtype)
    check(library().ln_dropout_residual_fwd(p, d, x.data_ptr(), _ptr(residual), _ptr(gamma), _ptr(beta), y.data_ptr(),
                                            _ptr(h), _ptr(mean), _ptr(rstd), current_stream(device.index)),
          "ln_residual_fwd")
    if return_sum:
        return (y, h, mean, rstd) if return_stats else (y, h)
    return (y, mean, rstd) if return_stats else y


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
    device, shape = dy.device, dy.shape
    cols = _cols(dy)
    rows = dy.numel() // cols
    if h.shape != shape or h.dtype != dy.dtype or h.device != device:
        raise ValueError("h must match dy in shape, dtype and device")
    if dh is not None and (dh.shape != shape or dh.dtype != dy.dtype or dh.device != device):
        raise ValueError("dh must match dy in shape, dtype and device")
    for t in (mean, rstd):
        if t.dtype != torch.float32 or t.numel() != rows or t.device != device:
            raise ValueError(f"mean and rstd must be float32 CUDA tensors of {rows} elements")
    _check_weight("gamma", gamma, cols, device)
    if stream is not None or device.index != current_device():
        with elsewhere(device, stream, (dy, h, mean, rstd, gamma, dh, rng, workspace)):
            return layernorm_residual_bwd(dy, h, mean, rstd, gamma, dh, dropout_p=dropout_p, seed=seed, offset=offset,
                                          rng=rng, weight_grads=weight_grads, workspace=workspace)
    d = dropout_params(dropout_p, seed, offset, rng, device)
    lib = library()
    dr = like(dy)
    dy, dy_stride = as_rows(dy, cols)
    h, h_stride = as_rows(h, cols)
    dh_stride = cols
    if dh is not None:
        dh, dh_stride = as_rows(dh, cols)
    mean, rstd = mean.contiguous(), rstd.contiguous()
    gamma = None if gamma is None else gamma.contiguous()
    dx = dr if d is None else torch.empty_like(dr)
    p = LnBwdParamsC(rows, cols, dy_stride, dh_stride, h_stride, cols, cols, dtype)
    dgamma = dbeta = ws = None
    need = 0
    if weight_grads:
        dgamma = torch.empty(cols, dtype=torch.float32, device=device)
        dbeta = torch.empty_like(dgamma)
        need = lib.ln_residual_bwd_workspace_size(p)
        if workspace is None and 0 < need < SIZE_MAX:
            ws = torch.empty(need, dtype=torch.uint8, device=device)
        else:
            ws = _workspace(need, device, workspace)
    check(lib.ln_residual_bwd(p, d, dy.data_ptr(), _ptr(dh), h.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                              _ptr(gamma), None if d is None else dx.data_ptr(), dr.data_ptr(), _ptr(dgamma),
                              _ptr(dbeta), _ptr(ws), need, current_stream(device.index)), "ln_residual_bwd")
    return dx, dr, dgamma, dbeta
