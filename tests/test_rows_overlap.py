"""Outputs of the row operators over their inputs are refused."""

import os
import subprocess

import pytest
import torch

from bwd_flashattention_fwd_sm_gb300 import _lib, build, embedding_bwd
from bwd_flashattention_fwd_sm_gb300._lib import EmbeddingParamsC

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
