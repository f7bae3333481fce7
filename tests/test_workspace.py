"""What the bindings take as a caller's workspace: its address goes to the kernels, so it has to
be memory of the call's device, and all of its bytes the caller's."""

import pytest
import torch

from bwd_flashattention_fwd_sm_gb300 import Kv4Cache, attn_bwd, attn_fwd, attn_fwd_kv4
from bwd_flashattention_fwd_sm_gb300.attention import _workspace

CPU = torch.device("cpu")


def test_of_the_device_and_large_enough_is_taken():
    ws = torch.empty(64, dtype=torch.float32)
    assert _workspace(256, CPU, ws) is ws
    assert _workspace(0, CPU, ws) is None
    more = _workspace(257, CPU, ws)  # too small: a new one
    assert more is not ws and more.numel() * more.element_size() >= 257
    assert _workspace(16, CPU).device == CPU
    for t in (torch.empty(64, 64).t(), torch.empty(4, 1, 8, 16).permute(2, 0, 3, 1), torch.empty(2, 64, 64)[1]):
        assert _workspace(4 * t.numel(), CPU, t) is t  # any order of the axes


@pytest.mark.parametrize("ws, device", [
    (torch.empty(1 << 12, dtype=torch.uint8), torch.device("cuda", 0)),  # host memory
    (torch.empty(1, dtype=torch.uint8).expand(1 << 12), CPU),           # one byte that counts as many
    (torch.empty(1 << 13, dtype=torch.uint8)[::2], CPU),                # with bytes of others between
    (torch.empty(64, 64)[:, :63], CPU),
    (torch.empty(64, 64).as_strided((32, 64), (32, 1)), CPU),           # rows that overlap
])
def test_refused(ws, device):
    with pytest.raises(ValueError, match="workspace"):
        _workspace(1 << 10, device, ws)


@pytest.mark.gpu
@pytest.mark.parametrize("wrong", [lambda: torch.empty(1 << 24, dtype=torch.uint8),
                                   lambda: torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 24)])
def test_refused_by_the_calls(wrong):
    dev = torch.device("cuda", 0)
    q = torch.randn(1, 2, 128, 64, device=dev).to(torch.bfloat16)
    o, lse = attn_fwd(q, q, q)
    cache = Kv4Cache.empty(8, 2, 16, 64, device=dev)
    table = torch.zeros(1, 8, dtype=torch.int32, device=dev)
    lens = torch.zeros(1, dtype=torch.int32, device=dev)
    for call in (lambda ws: attn_fwd(q, q, q, workspace=ws), lambda ws: attn_bwd(q, q, q, o, q, lse, workspace=ws),
                 lambda ws: attn_fwd_kv4(q, cache, table, lens, workspace=ws),
                 lambda ws: attn_fwd_kv4(q[:, :, :1], cache, table, lens, workspace=ws)):
        with pytest.raises(ValueError, match="workspace"):
            call(wrong())
        call(torch.empty(1 << 24, dtype=torch.uint8, device=dev))
    torch.cuda.synchronize()
