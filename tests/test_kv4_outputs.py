"""Outputs of the 4-bit cache's calls whose rows overlap, so that two rows would be written to one
place: refused by the binding, and by the C entries where one stride shows it.  Inputs may overlap."""

import itertools

import numpy as np
import pytest
import torch

from bwd_flashattention_fwd_sm_gb300 import Kv4Cache, _lib, attn_fwd_kv4, get_status, kv4_read
from bwd_flashattention_fwd_sm_gb300.kv4 import _fits, _rows_overlap, _share

from test_kv4_abi import FAKE, params

CUDA, INVALID = _lib.ATTN_ERR_CUDA, _lib.ATTN_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def both(lib, p):
    """The read, whose outputs are x and y; the attention, whose output is y."""
    return (lib.attn_kv4_read(p, FAKE, FAKE, FAKE, FAKE, FAKE, 2 * FAKE, None),
            lib.attn_fwd_kv4(p, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 40, None))


def layout(which, b, h, s, **kw):
    return params(**{f"{which}_stride_b": b, f"{which}_stride_h": h, f"{which}_stride_s": s, **kw})


@pytest.mark.parametrize("step", [0, 64])
@pytest.mark.parametrize("axis", [0, 1, 2])
def test_an_expanded_output_is_refused(lib, axis, step):
    st = [8 * 3 * 128, 3 * 128, 128]
    st[axis] = step
    assert both(lib, layout("y", *st)) == (INVALID, INVALID)
    assert b"overlap" in lib.attn_last_error()
    assert both(lib, layout("x", *st)) == (INVALID, CUDA)
    assert lib.attn_kv4_write(layout("y", *st), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None) == CUDA
    assert lib.attn_kv4_write(layout("x", *st), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None) == CUDA


def test_an_axis_of_one_entry_may_have_any_stride(lib):
    assert both(lib, layout("y", 0, 3 * 128, 128, batch=1)) == (CUDA, CUDA)
    assert both(lib, layout("y", 8 * 128, 128, 0, seqlen=1)) == (CUDA, CUDA)
    assert both(lib, layout("y", 3 * 128, 0, 128, heads_q=1, heads_kv=1)) == (CUDA, CUDA)


def test_packed_rows(lib):
    cu = np.asarray([0, 3, 5], np.int32)
    for s, h, code in ((8 * 128, 128, CUDA), (0, 128, INVALID), (8 * 128, 0, INVALID), (128, 5 * 128, CUDA)):
        p = layout("y", 0, h, s, cu_seqlens=FAKE, cu_seqlens_host=cu.ctypes.data)
        assert lib.attn_fwd_kv4(p, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 40, None) == code, (s, h)


def test_any_layout_against_an_enumeration():
    """Strides from half a row on, in all orders, up to four axes: found exactly where two rows share an element."""
    r = np.random.default_rng(1)
    for _ in range(3000):
        n = [int(x) for x in r.choice([1, 2, 3, 5], r.integers(2, 4))]
        st = [int(x) for x in r.choice([0, 64, 128, 192, 256, 320, 384, 512, 640, 768, 1000, 1536, 2560], len(n))]
        at = np.sort(np.array(list(itertools.product(*map(range, n)))) @ np.array(st))
        assert _rows_overlap((*n, 128), (*st, 1)) == bool(np.any(np.diff(at) < 128)), (n, st)
    # rows between one another's, which no order of the axes tells apart
    assert not _rows_overlap((2, 2, 1, 128), (384, 256, 640, 1))


def test_usual_views_fit():
    flat = torch.zeros(2 * 4 * 6 * 64)
    whole = flat.view(2, 4, 6, 64)
    for t in (whole, whole.transpose(1, 2), whole[:, :, 1:4], whole[:, ::2], flat.view(8, 6, 64), whole[:0]):
        assert _fits(t)
    assert not _fits(whole[:1].expand(2, 4, 6, 64))
    assert not _fits(whole[:, :, :1].expand(2, 4, 6, 64))
    assert not _fits(flat.as_strided((2, 4, 6, 64), (4 * 64, 64, 64, 1)))


def test_two_outputs_that_share_memory():
    both = torch.zeros(2, 5, 2, 3, 64)  # [batch, tokens, keys or values, heads, head_dim]
    k, v = both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2)
    assert not _share(k, v) and not _share(v, k) and not _share(k[:0], k[:0])
    assert _share(k, k) and _share(k[:, :, :4], k[:, :, 1:]) and _share(k[:, :, 1:], k[:, :, :4])
    assert not _share(k[:, :2], v[:, :2]) and not _share(torch.zeros(2, 64), torch.zeros(2, 64))
    rows = torch.zeros(8, 64)
    assert _share(rows[:4], rows[3:7]) and not _share(rows[:4], rows[4:]) and not _share(rows[::2], rows[1::2])


@pytest.mark.gpu
def test_refused_by_the_calls():
    dev = torch.device("cuda", 0)
    cache = Kv4Cache.empty(8, 2, 16, 64, device=dev)
    table = torch.zeros(2, 2, dtype=torch.int32, device=dev)
    lens = torch.zeros(2, dtype=torch.int32, device=dev)
    q = torch.zeros(2, 4, 3, 64, dtype=torch.bfloat16, device=dev)
    k = torch.zeros(2, 2, 3, 64, dtype=torch.bfloat16, device=dev)
    for wrong in (q[:1].expand(2, 4, 3, 64), q[:, :1].expand(2, 4, 3, 64), q[:, :, :1].expand(2, 4, 3, 64)):
        with pytest.raises(ValueError, match="apart"):
            attn_fwd_kv4(q, cache, table, lens, out=wrong)
    long = torch.zeros(2, 2, 7, 64, dtype=torch.bfloat16, device=dev)
    for wrong in ((k, k), (long[:, :, :3], long[:, :, 2:5]), (k, k[:1].expand(2, 2, 3, 64)), (k[:, :1].expand(2, 2, 3, 64), k)):
        with pytest.raises(ValueError):
            kv4_read(cache, table, lens, 3, out=wrong)
    attn_fwd_kv4(q[:1].expand(2, 4, 3, 64), cache, table, lens, out=torch.empty_like(q))  # an input may
    kv4_read(cache, table, lens, 3, out=(k, torch.empty_like(k)))
    kv4_read(cache, table, lens, 3, out=(long[:, :, :3], long[:, :, 3:6]))
    torch.cuda.synchronize()
    assert get_status() == 0
