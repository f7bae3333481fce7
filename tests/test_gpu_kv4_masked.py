"""GPU tests of a cache with a key or value that is not finite, at a position that only the last tokens of a
call see: it reaches the rows that see it, and no other.  Oracle and tolerances as in test_gpu_kv4.py."""

import numpy as np
import pytest
import torch

from bwd_flashattention_fwd_sm_gb300 import attn_fwd_kv4, get_status

from test_gpu_kv4 import DEV, DT, Paged, check_attend

pytestmark = pytest.mark.gpu

CASES = [  # D, Hq, Hkv, t, dtype: up to 24 rows on a KV head, float32, then more
    (64, 4, 2, 5, "bf16"), (128, 8, 2, 5, "bf16"), (256, 4, 2, 7, "bf16"), (64, 4, 4, 9, "f32"), (128, 4, 2, 5, "f32"),
    (64, 8, 2, 40, "bf16"), (128, 8, 2, 40, "bf16"),
]


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")], ids=str)
@pytest.mark.parametrize("what", [0, 1], ids=["step", "offset"])
@pytest.mark.parametrize("which", [0, 1], ids=["key", "value"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_what_is_not_finite_stays_with_the_rows_that_see_it(case, which, what, value):
    D, Hq, Hkv, t, dtype = case
    if what == 0 and value < 0:
        pytest.skip("a step is not negative")
    lens, back, group = [150, 64, 385], 3, D // 64 - 1  # seen by the last three tokens; the last group of the row
    c = Paged(lens, Hkv, D, 16, seed=D + t)
    q = torch.randn(3, Hq, t, D, generator=torch.Generator().manual_seed(t)).to(DT[dtype])
    call = lambda: attn_fwd_kv4(q.to(DEV), c.cache, c.table_dev, c.lens_dev)  # noqa: E731
    clean = [x.double().cpu().numpy() for x in call()]
    for n, length in enumerate(lens):
        at = length - back
        (c.cache.k_scale, c.cache.v_scale)[which][int(c.table[n, at // 16]), :, at % 16, group, what] = value
    o, lse = (x.double().cpu().numpy() for x in call())
    assert get_status() == 0
    # the rows that see it, and where it is a value only its group of them
    hit_o, hit_l = np.zeros(o.shape, bool), np.zeros(lse.shape, bool)
    if which == 0:
        hit_o[:, :, -back:], hit_l[:, :, -back:] = True, True
    else:
        hit_o[:, :, -back:, group * 64 :] = True
        assert not np.isfinite(o[hit_o]).any()
    assert np.isfinite(o[~hit_o]).all() and np.isfinite(lse[~hit_l]).all()
    check_attend(c, q.double().numpy(), np.where(hit_o, clean[0], o), np.where(hit_l, clean[1], lse), D ** -0.5, True,
                 dtype, f"masked {case} {which} {what} {value}")
