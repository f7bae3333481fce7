"""Guard regions around what the attention over the 4-bit cache writes: O, LSE and the workspace, which has
exactly the size that the library asks for.  And O written over the queries."""

import numpy as np
import pytest
import torch

from bwd_flashattention_fwd_sm_gb300 import Kv4Cache, SeqLens, _lib, attn_fwd_kv4, get_status, kv4_read, kv4_write
from bwd_flashattention_fwd_sm_gb300.kv4 import _params

from test_gpu_guards import Guarded
from test_gpu_kv4 import DEV, DT, Paged

pytestmark = pytest.mark.gpu

CASES = {  # D, Hq, Hkv, dtype, lens, rows: of each sequence, or one count for all
    "one_token_split": (128, 8, 2, "bf16", [9000, 17], 1),
    "one_tile": (128, 4, 1, "bf16", [60, 3], 1),
    "a_few": (64, 10, 2, "bf16", [700, 333], 3),
    "d256": (256, 4, 2, "bf16", [1500, 900], 7),
    "f32": (64, 4, 4, "f32", [2100, 40], 2),
    "f32_d256": (256, 2, 1, "f32", [700, 40], 5),
    "many": (128, 8, 2, "bf16", [4000, 130], 33),
    "many_d64": (64, 8, 1, "bf16", [900, 129, 5], 40),
    "packed": (128, 8, 2, "bf16", [900, 0, 333, 5], [1, 2, 3, 1]),
    "packed_many": (64, 8, 2, "bf16", [900, 0, 333, 5], [70, 2, 1, 9]),
}


def inputs(kind):
    D, Hq, Hkv, dtype, lens, rows = CASES[kind]
    c = Paged(lens, Hkv, D, 16, seed=len(kind))
    g = torch.Generator().manual_seed(D)
    if isinstance(rows, int):
        return c, torch.randn(len(lens), Hq, rows, D, generator=g).to(DT[dtype]).to(DEV), None
    sl = SeqLens(np.concatenate([[0], np.cumsum(rows)]), device=DEV)
    return c, torch.randn(sl.total, Hq, D, generator=g).to(DT[dtype]).to(DEV), sl


@pytest.mark.parametrize("kind", CASES)
def test_outputs_and_workspace_guards_intact(kind):
    c, q, sl = inputs(kind)
    Hq = q.shape[1]
    o = Guarded(q.shape, q.dtype)
    lse = Guarded(q.shape[:3] if sl is None else (Hq, q.shape[0]), torch.float32)
    p = _params(q, o.t, c.cache, c.table_dev, c.lens_dev, sl, Hq, c.Hkv, 0.1, True)
    lib = _lib.load()
    ws = Guarded((0,), torch.uint8, nbytes=lib.attn_kv4_workspace_size(p))
    stream = torch.cuda.current_stream().cuda_stream
    for _ in range(2):  # the second call finds the first one's leavings in the workspace
        rc = lib.attn_fwd_kv4(p, q.data_ptr(), *c.cache._pointers, o.t.data_ptr(), lse.t.data_ptr(), ws.raw.data_ptr(),
                              ws.nbytes, stream)
        assert rc == _lib.ATTN_OK, lib.attn_last_error()
    want = attn_fwd_kv4(q, c.cache, c.table_dev, c.lens_dev, scale=0.1, seqlens=sl)
    torch.cuda.synchronize()
    assert get_status() == 0
    for name, guarded in (("o", o), ("lse", lse), ("workspace", ws)):
        assert guarded.intact(), f"{name}[{kind}]: bytes outside it were written"
    assert torch.equal(o.t, want[0]) and torch.equal(lse.t, want[1])


@pytest.mark.parametrize("kind", CASES)
def test_o_over_the_queries(kind):
    c, q, sl = inputs(kind)
    want = attn_fwd_kv4(q, c.cache, c.table_dev, c.lens_dev, seqlens=sl)
    got = attn_fwd_kv4(q, c.cache, c.table_dev, c.lens_dev, seqlens=sl, out=q)
    torch.cuda.synchronize()
    assert get_status() == 0 and got[0] is q
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("t", [1, 40])
def test_a_cache_without_a_page(t):
    """Sequences that say they hold something: recorded, O 0 and LSE minus infinity; empty ones are no error."""
    cache = Kv4Cache.empty(0, 2, 16, 128, device=DEV)
    q, k = torch.randn(2, 8, t, 128, device=DEV).to(torch.bfloat16), torch.ones(2, 2, t, 128, device=DEV)
    table = torch.zeros(2, 4, dtype=torch.int32, device=DEV)
    for lens, status in ((torch.zeros(2, dtype=torch.int32, device=DEV), 0),
                         (torch.full((2,), 50, dtype=torch.int32, device=DEV), _lib.ATTN_ERR_DEVICE_BOUNDS)):
        o, lse = attn_fwd_kv4(q, cache, table, lens)
        assert get_status() == status
        assert torch.all(o == 0) and torch.all(torch.isneginf(lse))
        kv4_write(cache, k, k, table, lens)
        assert get_status() == status
        for x in kv4_read(cache, table, lens, t):
            assert torch.all(x == 0)
        assert get_status() == status
