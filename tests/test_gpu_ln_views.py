"""LayerNorm without dropout over views: the bits of the same call over contiguous copies."""

import pytest
import torch

from bwd_flashattention_fwd_sm_gb300 import layernorm_residual

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("cols", [64, 1000, 2048, 4096, 8192, 16384, 4095, 9])
def test_a_view_gives_the_bits_of_its_copy(cols, dtype):
    """Rows at 16-byte places and at others, of whole vectors and not; p = 2^-18 drops nothing and is the same call."""
    dt = getattr(torch, dtype)
    g = torch.Generator(device="cuda").manual_seed(cols)
    gamma = torch.randn(cols, generator=g, device="cuda")
    for before, behind in ((1, 0), (0, 4), (2, 2), (8, 8), (0, 24)):
        wide = torch.randn(2, 3, 20, before + cols + behind, generator=g, device="cuda").to(dt)[..., before:before + cols]
        x, r = wide
        for residual in (None, r, r.contiguous()):
            for p in (0.0, 2.0 ** -18):
                got = layernorm_residual(x, residual, gamma, return_stats=True, dropout_p=p)
                ref = layernorm_residual(x.contiguous(), None if residual is None else residual.contiguous(), gamma,
                                         return_stats=True)
                assert all(torch.equal(a, b) for a, b in zip(got, ref))
