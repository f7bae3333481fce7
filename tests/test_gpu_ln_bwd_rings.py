"""LayerNorm's backward pass where every block takes many rows that are no whole vectors: the elements at
a row's ends come into a stage of the ring through one thread and are read by another, while the stage is used again
and again.  Against the float64 oracle; tolerances as in test_gpu_ln_bwd.py."""

import numpy as np
import pytest
import torch

from bwd_flashattention_fwd_sm_gb300 import layernorm_residual
from oracle import rows as R

from parity_util import compare
from test_gpu_ln_bwd import DTYPES, U, check, f64, make, run

pytestmark = pytest.mark.gpu


# float32 with dh: so long that two stages are all there is, one block a row and two
@pytest.mark.parametrize("shape", [(400, 8187), (305, 6309), (1000, 7001), (200, 16379), (700, 12621)],
                         ids=lambda s: f"{s[0]}x{s[1]}")
def test_rings_of_two_stages(shape):
    rows, cols = shape
    inp = make(rows, cols, "f32", seed=cols)
    plain, dropping = run(inp), run(inp, dropout_p=0.3, seed=rows, offset=cols)
    check(plain, inp)
    check(dropping, inp, 0.3, rows, cols)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(plain, run(inp)))
        assert all(torch.equal(a, b) for a, b in zip(dropping, run(inp, dropout_p=0.3, seed=rows, offset=cols)))


# 33 to 64 vectors: a warp a row
@pytest.mark.parametrize("dtype, cols", [("bf16", 261), ("bf16", 403), ("bf16", 503), ("f32", 131), ("f32", 202), ("f32", 251)])
def test_rings_of_one_warp(dtype, cols):
    rows = 30011
    inp = make(rows, cols, dtype, seed=cols)
    got = run(inp, dropout_p=0.3, seed=rows, offset=cols)
    check(got, inp, 0.3, rows, cols)
    assert all(torch.equal(a, b) for a, b in zip(got, run(inp, dropout_p=0.3, seed=rows, offset=cols)))
    # the forward pass of the same rows
    x, r = inp["dy"], inp["dh"]
    y, h, mean, rstd = layernorm_residual(x.cuda(), r.cuda(), inp["gamma"].cuda(), return_stats=True, dropout_p=0.3,
                                          seed=rows, offset=cols)
    ref = R.ln_dropout_residual(f64(x), f64(r), f64(inp["gamma"]), None, 1e-5, 0.3, rows, cols)
    compare("y", f64(y), ref[0], dtype)
    half = torch.finfo(x.dtype).eps / 2
    assert np.all(np.abs(f64(h) - ref[1]) <= half * np.abs(ref[1]) + 4 * U * (np.abs(f64(x)) / 0.7 + np.abs(ref[1])))
