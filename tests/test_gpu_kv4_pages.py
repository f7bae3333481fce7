"""GPU tests of page lists that name no page: whatever the number, it is recorded and left out."""

import pytest
import torch

from bwd_flashattention_fwd_sm_gb300 import _lib, attn_fwd_kv4, get_status

from test_gpu_kv4 import DEV, Paged, check_attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("entry", [-1, -2, -3, -(1 << 31), 1 << 20, (1 << 31) - 1])
@pytest.mark.parametrize("t", [1, 40], ids=["few", "many"])  # the two kernels
def test_an_entry_that_is_no_page_is_recorded(t, entry):
    c = Paged([200, 200], 2, 128, 16, seed=5)
    q = torch.randn(2, 8, t, 128, generator=torch.Generator().manual_seed(t)).to(torch.bfloat16).to(DEV)
    good = attn_fwd_kv4(q, c.cache, c.table_dev, c.lens_dev)
    assert get_status() == 0
    bad = c.table_dev.clone()
    bad[0, 3] = entry
    o, lse = attn_fwd_kv4(q, c.cache, bad, c.lens_dev)
    assert get_status() == _lib.ATTN_ERR_DEVICE_BOUNDS and get_status() == 0
    assert torch.isfinite(o.float()).all() and not torch.equal(o[0], good[0][0])
    assert torch.equal(o[1], good[0][1]) and torch.equal(lse[1], good[1][1])  # the other sequence is as it was
    # behind a sequence's end the list is not read
    beyond = torch.full((2, 20), entry, dtype=torch.int32, device=DEV)
    beyond[:, :13] = c.table_dev
    o, lse = attn_fwd_kv4(q, c.cache, beyond, c.lens_dev)
    assert get_status() == 0
    check_attend(c, q.double().cpu().numpy(), o.double().cpu().numpy(), lse.double().cpu().numpy(), 128 ** -0.5, True,
                 "bf16", f"beyond {t} {entry}")
