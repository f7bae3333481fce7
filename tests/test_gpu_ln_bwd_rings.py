"""LayerNorm's backward pass where every block takes many rows that are no whole vectors: the elements at
a row's ends come into a stage of the ring through one thread and are read by another, while the stage is used again
and again.  Against the float64 oracle; tolerances as in test_gpu_ln_bwd.py."""

import pytest
import torch

from test_gpu_ln_bwd import check, make, run

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
