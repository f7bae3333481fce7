"""LayerNorm's backward pass where dy, h, mean or rstd of a row is not finite: it reaches that row of dr and
the columns' sums that it belongs to, and nothing else, in every form of the kernel.  The forward pass with dropout likewise."""

import numpy as np
import pytest
import torch

from bwd_flashattention_fwd_sm_gb300 import layernorm_residual, layernorm_residual_bwd
from oracle import rows as R

from test_gpu_ln_bwd import DTYPES, make

pytestmark = pytest.mark.gpu

# up to 32 vectors, one block a row, two blocks a row, each as whole vectors and not; more rows than blocks take at once
WIDTHS = {"bf16": [64, 101, 256, 403, 2048, 2049, 16384, 16370], "f32": [64, 101, 256, 251, 2048, 2049, 6313, 16384, 16377]}


def run(t, off=0, **kw):
    """off: every tensor this many elements off a 16-byte place, h one more (the form that moves single elements)."""
    d = {n: None if v is None else v.cuda() for n, v in t.items()}
    if off:
        for n, o in (("dy", off), ("h", off + 1), ("dh", off)):
            flat = torch.zeros(d[n].numel() + 8, dtype=d[n].dtype, device="cuda")
            flat[o:o + d[n].numel()] = d[n].view(-1)
            d[n] = flat[o:o + d[n].numel()].view(d[n].shape)
    return [v.cpu() for v in layernorm_residual_bwd(d["dy"], d["h"], d["mean"], d["rstd"], d["gamma"], d["dh"], **kw)]


@pytest.mark.parametrize("dtype, cols, off", [(d, c, 0) for d in WIDTHS for c in WIDTHS[d]]
                         + [(d, c, 1) for d in WIDTHS for c in (100, 4096, 16384)])
def test_what_is_not_finite_stays_in_its_row_and_columns(dtype, cols, off):
    rows = 20000 if cols <= 256 else 1000
    at = 7 if cols < 1000 else rows - 300
    inp = make(rows, cols, dtype, seed=cols)
    kw = dict(dropout_p=0.5, seed=4)
    clean = run(inp, off, **kw)
    assert all(torch.isfinite(t).all() for t in clean)
    keep = torch.from_numpy(R.dropout_bits(np.array([at]), cols, 4, 0)[0] >= 32768)
    others = torch.arange(rows) != at
    for bad in (float("nan"), float("inf"), -float("inf")):
        for name in ("dy", "h", "mean", "rstd"):
            where = {0, cols // 3, cols - 1} if name in ("dy", "h") else {None}
            for c in where:
                broken = {n: None if t is None else t.clone() for n, t in inp.items()}
                if c is None:
                    broken[name][at] = bad
                else:
                    broken[name][at, c] = bad
                dx, dr, dgamma, dbeta = run(broken, off, **kw)
                what = f"{name} {bad} at {c}"
                for got, ref in ((dx, clean[0]), (dr, clean[1])):
                    assert torch.equal(got[others], ref[others]), what
                assert not torch.isfinite(dr[at]).any(), what
                assert not torch.isfinite(dx[at][keep]).any() and not dx[at][~keep].any(), what
                hit = torch.ones(cols, dtype=torch.bool) if c is None else torch.arange(cols) == c
                assert not torch.isfinite(dgamma[hit]).any() and torch.equal(dgamma[~hit], clean[2][~hit]), what
                if name == "dy":
                    assert not torch.isfinite(dbeta[hit]).any() and torch.equal(dbeta[~hit], clean[3][~hit]), what
                else:
                    assert torch.equal(dbeta, clean[3]), what


@pytest.mark.parametrize("dtype, cols, off", [(d, c, 0) for d in WIDTHS for c in WIDTHS[d]]
                         + [(d, c, 1) for d in WIDTHS for c in (100, 4096, 16384)])
def test_forward_with_dropout(dtype, cols, off):
    """What is dropped leaves no trace, whatever it was; what is kept reaches its element of h and its row of y."""
    rows, at = (20000, 7) if cols <= 256 else (1000, 700)
    g = torch.Generator().manual_seed(cols)
    x = torch.randn(rows, cols, generator=g).to(DTYPES[dtype])
    r = torch.randn(rows, cols, generator=g).to(DTYPES[dtype])
    gamma, beta = torch.randn(cols, generator=g) + 2, torch.randn(cols, generator=g)
    keep = torch.from_numpy(R.dropout_bits(np.array([at]), cols, 4, 0)[0] >= 32768)
    others = torch.arange(rows) != at

    def fwd(x, r):
        flat = torch.zeros(x.numel() + 8, dtype=x.dtype, device="cuda")
        flat[off:off + x.numel()] = x.cuda().view(-1)
        return [t.cpu() for t in layernorm_residual(flat[off:off + x.numel()].view(x.shape), r.cuda(), gamma.cuda(),
                                                    beta.cuda(), return_stats=True, dropout_p=0.5, seed=4)]

    clean = fwd(x, r)
    for bad in (float("nan"), float("inf"), -float("inf")):
        broken = x.clone()
        broken[at][~keep] = bad
        assert all(torch.equal(a, b) for a, b in zip(fwd(broken, r), clean))
        for name in ("x", "r"):
            xr = {"x": x.clone(), "r": r.clone()}
            c = int(keep.nonzero()[-1])
            xr[name][at, c] = bad
            got = fwd(xr["x"], xr["r"])
            for a, b in zip(got, clean):
                assert torch.equal(a[others], b[others])
            y, h, mean, rstd = (t[at] for t in got)
            assert not torch.isfinite(y).any() and not torch.isfinite(h[c]) and not torch.isfinite(mean)
            rest = torch.arange(cols) != c
            assert torch.equal(h[rest], clean[1][at][rest])
