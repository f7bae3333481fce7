"""The C entries of dropout, LayerNorm's backward pass and the embedding table without a
GPU: refusals before any device work, and workspace sizes."""

import ctypes

import pytest
import torch

import bwd_flashattention_fwd_sm_gb300 as G
from bwd_flashattention_fwd_sm_gb300 import _lib
from bwd_flashattention_fwd_sm_gb300._lib import EmbeddingParamsC, LnBwdParamsC, LnDropoutC, LnParamsC
from bwd_flashattention_fwd_sm_gb300.rows import as_rows

FAKE = 1 << 20  # an aligned non-NULL address; never dereferenced by host validation
INVALID, UNSUPPORTED, NO_GPU = _lib.ATTN_ERR_INVALID_ARG, _lib.ATTN_ERR_UNSUPPORTED, _lib.ATTN_ERR_CUDA


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def ln_params(**kw):
    p = LnParamsC(8, 64, 64, 64, 64, 64, 1e-5, _lib.ATTN_BF16)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def drop(**kw):
    d = LnDropoutC(0.1, 1, 2, FAKE)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def dropout(lib, p, d, x=FAKE, y=FAKE):
    return lib.ln_dropout(p, d, x, y, None)


def ln_fwd(lib, p, d):
    return lib.ln_dropout_residual_fwd(p, d, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None)


def bwd_params(**kw):
    p = LnBwdParamsC(8000, 64, 64, 64, 64, 64, 64, _lib.ATTN_BF16)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


NAMES = ("dy", "dh", "h", "mean", "rstd", "gamma", "dx", "dr", "dgamma", "dbeta")


def bwd(lib, p, d=None, ws=FAKE, ws_bytes=1 << 40, **ptr):
    return lib.ln_residual_bwd(p, d, *[ptr.get(n, FAKE) for n in NAMES], ws, ws_bytes, None)


def embed_params(**kw):
    p = EmbeddingParamsC(800, 100, 64, 64, 64, 1.0, _lib.ATTN_BF16, _lib.ATTN_BF16, 1, 0, -1)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def embed(lib, p, weight=FAKE, ids=FAKE, y=FAKE):
    return lib.attn_embedding_fwd(p, weight, ids, y, None)


def embed_bwd(lib, p, dy=FAKE, ids=FAKE, dw=FAKE, ws=FAKE, ws_bytes=1 << 60):
    return lib.attn_embedding_bwd(p, dy, ids, dw, ws, ws_bytes, None)


def test_valid_calls_fail_only_for_want_of_a_gpu(lib):
    for dtype in (_lib.ATTN_BF16, _lib.ATTN_F32):
        assert dropout(lib, ln_params(dtype=dtype), drop()) == NO_GPU
        assert ln_fwd(lib, ln_params(dtype=dtype), drop()) == NO_GPU
        assert ln_fwd(lib, ln_params(dtype=dtype), None) == NO_GPU
        assert bwd(lib, bwd_params(dtype=dtype), drop()) == NO_GPU
        assert bwd(lib, bwd_params(dtype=dtype), None, dh=None, gamma=None, dx=None, dgamma=None) == NO_GPU
        assert embed(lib, embed_params(dtype=dtype)) == NO_GPU
        assert embed_bwd(lib, embed_params(dtype=dtype)) == NO_GPU


@pytest.mark.parametrize("change, code", [
    ({"dtype": 5}, INVALID), ({"rows": -1}, INVALID), ({"cols": -1}, INVALID), ({"x_stride": 63}, INVALID),
    ({"y_stride": 63}, INVALID), ({"rows": 1 << 32}, UNSUPPORTED),
    ({"cols": 1 << 32, "x_stride": 1 << 32, "y_stride": 1 << 32}, UNSUPPORTED),
])
def test_dropout_refusals(lib, change, code):
    assert dropout(lib, ln_params(**change), drop()) == code
    assert lib.attn_last_error() != b""


@pytest.mark.parametrize("change", [{"p": -0.1}, {"p": 1.1}, {"p": float("nan")}, {"rng": FAKE + 4}])
def test_dropout_arguments_refused_everywhere(lib, change):
    assert dropout(lib, ln_params(), drop(**change)) == INVALID
    assert ln_fwd(lib, ln_params(), drop(**change)) == INVALID
    assert bwd(lib, bwd_params(), drop(**change)) == INVALID


def test_dropout_pointers(lib):
    assert lib.ln_dropout(None, drop(), FAKE, FAKE, None) == INVALID
    assert dropout(lib, ln_params(), None) == INVALID
    assert dropout(lib, ln_params(), drop(), x=None) == INVALID
    assert dropout(lib, ln_params(), drop(), y=FAKE + 1) == INVALID
    assert dropout(lib, ln_params(dtype=_lib.ATTN_F32), drop(), y=FAKE + 2) == INVALID
    # 8 rows of 64 bf16, 64 or 128 elements apart: y on x's elements, beside them, between them, x itself
    wide = dict(x_stride=128, y_stride=128)
    for change, y, code in (({}, FAKE + 128, INVALID), ({}, FAKE + 1024, NO_GPU), ({}, FAKE, NO_GPU),
                            (wide, FAKE + 128, NO_GPU), (wide, FAKE - 128, NO_GPU), (wide, FAKE + 126, INVALID),
                            (wide, FAKE + 130, INVALID), (wide, FAKE + 256, INVALID), (wide, FAKE, NO_GPU),
                            ({"x_stride": 128}, FAKE, INVALID), ({"x_stride": 128}, FAKE + 2048, NO_GPU),
                            ({"rows": 1, "x_stride": 128}, FAKE, NO_GPU), ({"rows": 1}, FAKE + 126, INVALID)):
        assert dropout(lib, ln_params(**change), drop(), y=y) == code, (change, y - FAKE)
    for empty in ({"rows": 0}, {"cols": 0, "x_stride": 0, "y_stride": 0}):
        assert dropout(lib, ln_params(**empty), drop(), x=None, y=None) == _lib.ATTN_OK


def test_forward_refusals(lib):
    assert ln_fwd(lib, ln_params(cols=16385, x_stride=1 << 15, r_stride=1 << 15, y_stride=1 << 15, h_stride=1 << 15),
                  drop()) == UNSUPPORTED
    assert ln_fwd(lib, ln_params(rows=1 << 32), drop()) == UNSUPPORTED
    assert ln_fwd(lib, ln_params(rows=1 << 32), drop(p=0.0)) == NO_GPU  # nothing is dropped
    assert ln_fwd(lib, ln_params(rows=0), drop()) == _lib.ATTN_OK


@pytest.mark.parametrize("change, code", [
    ({"dtype": 5}, INVALID), ({"rows": -1}, INVALID), ({"cols": 0}, INVALID), ({"cols": 16385}, UNSUPPORTED),
])
def test_bwd_refusals(lib, change, code):
    p = bwd_params(**change)
    assert bwd(lib, p) == code
    assert lib.ln_residual_bwd_workspace_size(p) == _lib.SIZE_MAX


def test_bwd_strides_pointers_and_workspace(lib):
    for s in ("dy_stride", "dh_stride", "h_stride", "dx_stride", "dr_stride"):
        assert bwd(lib, bwd_params(**{s: 63})) == INVALID
    for n in NAMES:
        assert bwd(lib, bwd_params(), drop(), **{n: FAKE + 1}) == INVALID
    for n in ("dy", "h", "mean", "rstd"):
        assert bwd(lib, bwd_params(), **{n: None}) == INVALID
    assert bwd(lib, bwd_params(dh_stride=0), dh=None) == NO_GPU
    assert bwd(lib, bwd_params(rows=1 << 32), drop()) == UNSUPPORTED
    need = lib.ln_residual_bwd_workspace_size(bwd_params())
    assert 0 < need < 1 << 20
    assert bwd(lib, bwd_params(), ws=None) == _lib.ATTN_ERR_WORKSPACE
    assert bwd(lib, bwd_params(), ws=FAKE + 16) == _lib.ATTN_ERR_WORKSPACE
    assert bwd(lib, bwd_params(), ws_bytes=need - 1) == _lib.ATTN_ERR_WORKSPACE
    assert bwd(lib, bwd_params(), ws=None, ws_bytes=0, dgamma=None, dbeta=None) == NO_GPU
    few = bwd_params(rows=100)
    assert lib.ln_residual_bwd_workspace_size(few) == 0 and bwd(lib, few, ws=None, ws_bytes=0) == NO_GPU
    none = dict.fromkeys(NAMES)
    assert bwd(lib, bwd_params(rows=0), ws=None, ws_bytes=0, **none) == _lib.ATTN_OK
    # the columns' partial sums: never more than the largest grid's
    for rows in (200000, 1 << 40):
        for cols in (1, 64, 1000, 16384):
            p = bwd_params(rows=rows, cols=cols)
            assert 8 * cols <= lib.ln_residual_bwd_workspace_size(p) < 5000 * cols


@pytest.mark.parametrize("change, code", [
    ({"dtype": 5}, INVALID), ({"tokens": -1}, INVALID), ({"vocab": -1}, INVALID), ({"dim": -1}, INVALID),
    ({"x_stride": 63}, INVALID), ({"w_stride": 63}, INVALID), ({"scale": float("inf")}, INVALID),
    ({"scale": float("nan")}, INVALID), ({"tokens": 2 ** 31 - 1}, UNSUPPORTED), ({"vocab": 2 ** 31 - 1}, UNSUPPORTED),
    ({"dim": 2 ** 20 + 1, "x_stride": 1 << 21, "w_stride": 1 << 21}, UNSUPPORTED),
])
def test_embedding_refusals(lib, change, code):
    p = embed_params(**change)
    assert embed(lib, p) == code
    assert embed_bwd(lib, p) == code
    assert lib.attn_embedding_bwd_workspace_size(p) == _lib.SIZE_MAX


def test_embedding_pointers_and_workspace(lib):
    assert embed_bwd(lib, embed_params(w_dtype=5)) == INVALID
    for bad in ({"weight": None}, {"ids": None}, {"y": None}, {"ids": FAKE + 4}, {"y": FAKE + 1}):
        assert embed(lib, embed_params(), **bad) == INVALID
    for bad in ({"dy": None}, {"ids": None}, {"dw": None}, {"ids": FAKE + 4}, {"dw": FAKE + 1}):
        assert embed_bwd(lib, embed_params(), **bad) == INVALID
    assert embed(lib, embed_params(ids_64=0), ids=FAKE + 4) == NO_GPU
    need = lib.attn_embedding_bwd_workspace_size(embed_params())
    assert embed_bwd(lib, embed_params(), ws=None) == _lib.ATTN_ERR_WORKSPACE
    assert embed_bwd(lib, embed_params(), ws=FAKE + 16) == _lib.ATTN_ERR_WORKSPACE
    assert embed_bwd(lib, embed_params(), ws_bytes=need - 1) == _lib.ATTN_ERR_WORKSPACE
    few = embed_params(tokens=8)
    assert lib.attn_embedding_bwd_workspace_size(few) == 0 and embed_bwd(lib, few, ws=None, ws_bytes=0) == NO_GPU
    assert embed(lib, embed_params(tokens=0), None, None, None) == _lib.ATTN_OK
    assert embed(lib, embed_params(dim=0), None, None, None) == _lib.ATTN_OK
    assert embed_bwd(lib, embed_params(vocab=0), None, None, None, None, 0) == _lib.ATTN_OK
    assert embed_bwd(lib, embed_params(tokens=0, accumulate=1), None, None, None, None, 0) == _lib.ATTN_OK
    assert embed_bwd(lib, embed_params(tokens=0), None, None, FAKE, None, 0) == NO_GPU  # writes zeros
    assert embed(lib, embed_params(vocab=0), weight=None) == NO_GPU  # writes zeros, records the ids


def test_bindings_refuse_host_tensors_and_bad_arguments():
    x = torch.zeros(4, 8)
    i = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: G.dropout(x, 0.1), lambda: G.layernorm_residual(x), lambda: G.embedding(x, i),
                 lambda: G.layernorm_residual_bwd(x, x, x[:, 0], x[:, 0]), lambda: G.embedding_bwd(x, i, 4)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="between 0 and 1"):
        G.drop.dropout_params(1.5, 0, 0, None, x.device)
    for rng in (torch.zeros(2), torch.zeros(3, dtype=torch.int64), torch.zeros(4, dtype=torch.int64)[::2]):
        with pytest.raises(ValueError, match="rng"):
            G.drop.dropout_params(0.5, 0, 0, rng, x.device)
    assert G.drop.dropout_params(0.0, 0, 0, None, x.device) is None
    d = G.drop.dropout_params(0.5, -1, 1 << 65, None, x.device)
    assert (d.seed, d.offset) == (2 ** 64 - 1, 0)


def test_rows_of_a_view():
    """A tensor whose rows are a fixed number of elements apart is used as it is, another copied."""
    base = torch.arange(2 * 3 * 4 * 10.0).reshape(2, 3, 4, 10)
    for view, step in ((base, 10), (base[..., :7], 10), (base[:, :, 1], 40), (base[:, 1, 2], 120),
                       (base[0, 0, 0], 10), (base[:1, :1, :1, :5], 5), (base[..., :1], 10)):
        rows, stride = as_rows(view, view.shape[-1])
        flat = view.reshape(-1, view.shape[-1])
        got = rows.as_strided(flat.shape, (stride, 1)) if flat.shape[0] > 1 else rows.reshape(flat.shape)
        assert torch.equal(got, flat)
        if rows is view:
            assert stride == step or flat.shape[0] == 1
    for view in (base.transpose(2, 3), base[..., ::2], base[:, :2], base[:, 1:2], base[:1].expand(3, 3, 4, 10), base.flip(2)):
        rows, stride = as_rows(view, view.shape[-1])
        assert torch.equal(rows.as_strided((view.numel() // view.shape[-1], view.shape[-1]), (stride, 1)),
                           view.reshape(-1, view.shape[-1]))
    one = torch.zeros(5, 1)[:, :1].expand(5, 1)
    assert as_rows(one, 1)[1] == 1
