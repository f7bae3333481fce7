"""GPU tests of the many-row form of the attention over the 4-bit cache (csrc/kv4_tc.cu): blocks
that deal with several pieces of work one after the other.  Oracle and tolerances as in
test_gpu_kv4.py."""

import numpy as np
import pytest
import torch

from bwd_flashattention_fwd_sm_gb300 import attn_fwd_kv4, get_status

from test_gpu_kv4 import DEV, Paged, check_attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_several_pieces_a_block(D, causal):
    """480 row tiles, more than three a block, of one to three tiles of keys; every fifth sequence is empty, and
    its pieces have no key at all.  What a piece leaves for its rows' other warps (sums of the weights, sums of Q) has
    to last until they have read it: the same bits each time, and the oracle's values."""
    r = np.random.default_rng(D)
    lens = [0 if n % 5 == 2 else int(r.integers(1, 300)) for n in range(60)]
    c = Paged(lens, 8, D, 16, seed=D + 7)
    q = torch.randn(60, 32, 8, D, generator=torch.Generator().manual_seed(D)).to(torch.bfloat16)
    qd = q.to(DEV)
    o, lse = attn_fwd_kv4(qd, c.cache, c.table_dev, c.lens_dev, causal=causal, scale=0.2)
    for _ in range(20):
        o2, lse2 = attn_fwd_kv4(qd, c.cache, c.table_dev, c.lens_dev, causal=causal, scale=0.2)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert get_status() == 0
    check_attend(c, q.double().numpy(), o.double().cpu().numpy(), lse.double().cpu().numpy(), 0.2, causal, "bf16",
                 f"pieces {D} {causal}")
