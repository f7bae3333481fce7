"""The row operators under the checked library (GBATTN_CHECKED=1), with valid inputs: every computed place
of the embedding's sort and sums lies inside its array, and the results are those of the plain library."""

import os
import subprocess
import sys

import pytest
import torch

from bwd_flashattention_fwd_sm_gb300 import dropout, embedding, embedding_bwd, layernorm_residual, layernorm_residual_bwd

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def results():
    g = torch.Generator().manual_seed(1)
    out = []
    for tokens, vocab, dim in ((7, 3, 8), (3000, 50, 130), (20000, 70000, 16)):
        dy = torch.randn(tokens, dim, generator=g).cuda()
        ids = torch.randint(0, vocab, (tokens,), generator=g).cuda()
        out += [embedding(dy[:vocab], ids % min(vocab, tokens)), embedding_bwd(dy, ids, vocab, padding_id=1)]
    for rows, cols in ((40, 100), (50, 1003), (30, 4096)):
        x = torch.randn(rows, cols, generator=g).to(torch.bfloat16).cuda()
        y, h, mean, rstd = layernorm_residual(x, x, return_stats=True, dropout_p=0.2, seed=1)
        out += [dropout(x, 0.3), y, *layernorm_residual_bwd(y, h, mean, rstd, dropout_p=0.2, seed=1)]
    torch.cuda.synchronize()
    return [t.cpu() for t in out]


def test_checked_library_gives_the_same(tmp_path):
    path = str(tmp_path / "checked.pt")
    script = (f"import sys; sys.path[:0] = [{ROOT!r}, {os.path.join(ROOT, 'tests')!r}]\n"
              "import torch\nimport test_gpu_rows_checked as T\n"
              "from bwd_flashattention_fwd_sm_gb300 import _lib, get_status\n"
              "assert _lib.load().attn_version().endswith(b' checked')\n"
              f"torch.save(T.results(), {path!r})\nassert get_status() == 0\n")
    r = subprocess.run([sys.executable, "-c", script], env=dict(os.environ, GBATTN_CHECKED="1"), capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-2000:])
    for a, b in zip(results(), torch.load(path)):
        assert torch.equal(a, b)
