"""Which views LayerNorm without dropout copies before its kernel runs (on the CPU: the rule alone)."""

import pytest
import torch

from bwd_flashattention_fwd_sm_gb300.layernorm import _at_vectors
from bwd_flashattention_fwd_sm_gb300.rows import as_rows

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("rows, cols, step, first, dtype, one, two", [
    (8, 4096, 4100, 0, BF16, True, True), (8, 4096, 4104, 1, BF16, True, True), (8, 4096, 4104, 8, BF16, False, False),
    (8, 1024, 1028, 0, BF16, False, False), (1024, 1024, 1028, 0, BF16, True, False), (1023, 1024, 1028, 0, BF16, False, False),
    (1024, 1024, 1025, 0, F32, True, True), (2048, 1028, 1029, 0, F32, False, False), (8, 2052, 2053, 0, F32, True, True),
    (2048, 1028, 1032, 2, F32, False, False), (8, 4097, 4100, 0, BF16, False, False), (2048, 1022, 1024, 0, BF16, False, False),
])
def test_which_views_are_copied(rows, cols, step, first, dtype, one, two):
    base = torch.arange(rows * step + 16).to(dtype)
    assert base.data_ptr() % 16 == 0
    view = base[first:first + rows * step].view(rows, step)[:, :cols]
    whole = view.contiguous()
    for x, r, copied in ((view, None, one), (view, whole, one), (whole, view, one), (view, view, two)):
        x1, xs = as_rows(x, cols)
        r1, rs = (None, cols) if r is None else as_rows(r, cols)
        x2, xs2, r2, rs2 = _at_vectors(x1, xs, r1, rs, cols)
        for t, t2, s2 in ((x, x2, xs2), (r, r2, rs2)):
            if t is None:
                assert t2 is None
            elif t is view and copied:
                assert t2.is_contiguous() and s2 == cols and torch.equal(t2, view)
            else:
                assert t2 is t and s2 == (step if t is view else cols)
