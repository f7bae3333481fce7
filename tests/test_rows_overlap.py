"""Outputs of the row operators over their inputs are refused."""

import os
import subprocess

import pytest
import torch

from bwd_flashattention_fwd_sm_gb300 import _lib, build, embedding_bwd
from bwd_flashattention_fwd_sm_gb300._lib import EmbeddingParamsC, LnBwdParamsC, LnDropoutC

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, WORKSPACE = _lib.ATTN_ERR_INVALID_ARG, _lib.ATTN_ERR_WORKSPACE


def test_which_rows_share_memory(tmp_path):
    """The function that the entries call, against a count of every byte."""
    exe = str(tmp_path / "overlap")
    r = subprocess.run([build.nvcc(), "-std=c++17", "-I", build.CSRC, os.path.join(ROOT, "tests", "overlap_host.cu"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [40, 700])  # without and with a sort
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_gradient_over_its_own_inputs(tokens, dtype):
    dim = 16
    ids = torch.randint(0, tokens, (tokens,), device="cuda")
    both = torch.randn(3 * tokens, dim, device="cuda").to(dtype)
    keep = both.clone()
    dy = both[tokens:2 * tokens]
    for first in (1, tokens, 2 * tokens - 1):
        with pytest.raises(_lib.AttnError, match="overlaps dy"):
            embedding_bwd(dy, ids, tokens, out=both[first:first + tokens])
    with pytest.raises(_lib.AttnError, match="overlaps dy"):
        embedding_bwd(dy, ids, tokens, out=dy)
    assert torch.equal(both, keep)
    for first in (0, 2 * tokens):  # beside it
        out = both[first:first + tokens]
        ref = embedding_bwd(dy, ids, tokens, out=out.clone())
        assert embedding_bwd(dy, ids, tokens, out=out) is out and torch.equal(out, ref)
    assert torch.equal(dy, keep[tokens:2 * tokens])
    # columns beside each other in the same rows
    wide = torch.randn(tokens, 2 * dim, device="cuda").to(dtype)
    ref = embedding_bwd(wide[:, :dim], ids, tokens, out=wide[:, dim:].clone())
    assert torch.equal(embedding_bwd(wide[:, :dim], ids, tokens, out=wide[:, dim:]), ref)
    with pytest.raises(_lib.AttnError, match="overlaps dy"):
        embedding_bwd(wide[:, :dim], ids, tokens, out=wide[:, dim - 1:2 * dim - 1])


@pytest.mark.gpu
def test_c_entries_refuse_ids_and_workspace_too():
    lib, t, v, d = _lib.load(), 800, 100, 64
    p = EmbeddingParamsC(t, v, d, d, d, 1.0, _lib.ATTN_F32, _lib.ATTN_F32, 1, 0, -1)
    need = lib.attn_embedding_bwd_workspace_size(p)
    buf = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    a = buf.data_ptr()
    x, w, ids, ws = a, a + 4 * t * d, a + 4 * (t + v) * d, a + (1 << 20)  # apart
    assert 4 * (t + v) * d + 8 * t <= 1 << 20 and need <= 1 << 20

    def fwd(weight=w, ids=ids, y=x):
        return lib.attn_embedding_fwd(p, weight, ids, y, None)

    def bwd(dy=x, ids=ids, dw=w, ws=ws):
        return lib.attn_embedding_bwd(p, dy, ids, dw, ws, need, None)

    assert fwd() == 0 and bwd() == 0
    assert fwd(y=w) == INVALID and fwd(y=w + 4 * (v * d - 1)) == INVALID and fwd(weight=x + 16) == INVALID
    assert fwd(ids=x + 8) == INVALID and fwd(ids=x + 4 * t * d - 8) == INVALID
    assert bwd(dw=x) == INVALID and bwd(dw=ids) == INVALID and bwd(ids=w + 8) == INVALID
    for at in (a, a + 4 * t * d - 256, a + (1 << 18) - (1 << 16)):
        assert bwd(ws=at) == WORKSPACE
    assert bwd(ws=ids // 256 * 256) == WORKSPACE and bwd(dw=ws + need - 4) == WORKSPACE
    torch.cuda.synchronize()
    assert _lib.load().attn_get_status(None) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("drops", [False, True])
@pytest.mark.parametrize("cols", [64, 4096])  # with and without a join of the blocks' sums over a workspace
def test_layernorm_backward_over_its_own_inputs(cols, drops):
    lib, rows, step = _lib.load(), 200, 2 * cols
    p = LnBwdParamsC(rows, cols, step, step, step, step, step, _lib.ATTN_F32)
    d = LnDropoutC(0.3, 1, 2, None) if drops else None
    need = lib.ln_residual_bwd_workspace_size(p)
    assert (need > 0) == (cols == 4096)
    g = torch.Generator(device="cuda").manual_seed(1)
    new = lambda *shape: torch.randn(*shape, generator=g, device="cuda")
    t = {n: new(rows + 2, step) for n in ("dy", "dh", "h", "dx", "dr")}
    t.update({n: new(rows).abs() for n in ("mean", "rstd")}, **{n: new(2 * cols) for n in ("gamma", "dgamma", "dbeta")})
    t["ws"] = torch.zeros(need + 4 * rows * step, dtype=torch.uint8, device="cuda")
    at = {n: v.data_ptr() for n, v in t.items()}
    order = ("dy", "dh", "h", "mean", "rstd", "gamma", "dx", "dr", "dgamma", "dbeta", "ws")

    def call(**ptr):
        return lib.ln_residual_bwd(p, d, *[ptr.get(n, at[n]) for n in order], need, None)

    def results(**views):
        torch.cuda.synchronize()
        return [views.get(n, t[n])[:rows, :cols].clone() for n in ("dx", "dr")] + [t[n][:cols].clone()
                                                                               for n in ("dgamma", "dbeta")]

    assert call() == 0
    ref = results()
    one_row, one = 4 * step, 4
    for out in ("dx", "dr"):
        for other in ("dy", "dh", "h", "dr" if out == "dx" else "dx"):
            for off in (one, one_row, -one_row, one_row - 4 * (cols - 1)):
                assert call(**{out: at[other] + off}) == INVALID, (out, other, off)
        for small in ("mean", "rstd", "gamma"):
            assert call(**{small: at[out] + one_row}) == INVALID
        assert call(**{out: at["h"]}) == INVALID
    for out in ("dgamma", "dbeta"):
        for other in ("dy", "dx", "mean", "gamma", "dbeta" if out == "dgamma" else "dgamma"):
            assert call(**{out: at[other]}) == INVALID, (out, other)
    assert call(dr=at["dx"]) == (INVALID if drops else 0)
    if need:
        for other in ("dy", "dr", "gamma"):
            assert call(**{other: at["ws"]}) == INVALID
        assert call(dbeta=at["ws"] + need - one) == INVALID
    # what is allowed: in the gaps between the other's rows, and in place
    for views in ({"dx": t["dy"][:, cols:]}, {"dr": t["h"][:, cols:], "dx": t["dh"][:, cols:]}):
        assert call(**{n: v.data_ptr() for n, v in views.items()}) == 0
        assert all(torch.equal(a, b) for a, b in zip(results(**views), ref))
    kept = {n: t[n].clone() for n in ("dy", "dh")}
    for places in ({"dx": "dy"}, {"dr": "dy"}, {"dx": "dh"}, {"dr": "dh"}, {"dx": "dy", "dr": "dh"}, {"dx": "dh", "dr": "dy"}):
        for n, v in kept.items():
            t[n].copy_(v)
        torch.cuda.synchronize()
        assert call(**{n: at[v] for n, v in places.items()}) == 0
        assert all(torch.equal(a, b) for a, b in zip(results(**{n: t[v] for n, v in places.items()}), ref))
    assert lib.attn_get_status(None) == 0
