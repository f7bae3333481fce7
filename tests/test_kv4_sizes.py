"""How many rows a call of the 4-bit cache takes: packed ones are counted as they are, not as if every
sequence were the longest; counts whose product passes 64 bits are refused."""

import numpy as np
import pytest
import torch

from bwd_flashattention_fwd_sm_gb300 import SeqLens, _lib, attn_fwd_kv4, get_status, kv4_read, kv4_write

from test_kv4_abi import FAKE, calls, params

CUDA, UNSUPPORTED = _lib.ATTN_ERR_CUDA, _lib.ATTN_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def packed(counts, **kw):
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    kw = {"seqlen": max(counts), "heads_q": 8, "heads_kv": 8, "x_stride_h": 128, "x_stride_s": 1024, "y_stride_h": 128,
          "y_stride_s": 1024, **kw}
    return params(cu_seqlens=FAKE, cu_seqlens_host=cu.ctypes.data, batch=len(counts), **kw), cu


def test_a_long_sequence_beside_many_short_ones(lib):
    p, cu = packed([1 << 20] + [1] * 299)  # 300 * 2^20 * 8 > 2^31
    assert calls(lib, p) == (CUDA,) * 3 and lib.attn_kv4_workspace_size(p) not in (0, _lib.SIZE_MAX)
    p, cu = packed([3, 1, 1], seqlen=(1 << 31) - 1)  # "at least the most of any"
    assert calls(lib, p) == (CUDA,) * 3
    need = lib.attn_kv4_workspace_size(p)
    assert 0 < need < 1 << 30
    p, cu = packed([3] + [1] * 4999, seqlen=(1 << 31) - 1, heads_q=1 << 10, heads_kv=1 << 10, y_stride_s=1 << 17)
    assert calls(lib, p)[2] == CUDA and lib.attn_kv4_workspace_size(p) < 1 << 30


def test_limits(lib):
    wide = {"y_stride_s": 1 << 37, "x_stride_s": 1 << 37}
    p, cu = packed([1 << 20], heads_q=1 << 10, heads_kv=1 << 10, **wide)  # 2^30 rows: the attention's most
    assert calls(lib, p) == (CUDA,) * 3
    p, cu = packed([(1 << 20) + 1], heads_q=1 << 10, heads_kv=1 << 10, **wide)
    assert calls(lib, p) == (CUDA, CUDA, UNSUPPORTED)
    p, cu = packed([1 << 20, 1 << 20], heads_q=1 << 10, heads_kv=1 << 10, **wide)
    assert calls(lib, p) == (UNSUPPORTED,) * 3
    # more blocks of 16 rows than a launch has: 2^16 sequences, each as long as the longest
    p, cu = packed([1 << 20] + [1] * ((1 << 16) - 1))
    assert calls(lib, p) == (UNSUPPORTED, UNSUPPORTED, CUDA)


def test_products_beyond_64_bits(lib):
    for b, s, h in ((1 << 20, 1 << 22, 1 << 22), (1 << 30, 1 << 30, 1 << 4), ((1 << 31) - 1,) * 3):
        p = params(batch=b, seqlen=s, heads_q=h, heads_kv=h, y_stride_h=1 << 20, y_stride_b=1 << 40)
        assert calls(lib, p) == (UNSUPPORTED,) * 3, (b, s, h)
        assert lib.attn_kv4_workspace_size(p) == _lib.SIZE_MAX


@pytest.mark.gpu
def test_a_long_sequence_beside_many_short_ones_on_the_device():
    """More than 2^31 rows if every sequence were the longest.  All but the last 400 rows of the long one are padding."""
    from test_gpu_kv4 import DEV, Paged, check_attend

    H, D, long = 8, 64, 1 << 20
    r = np.random.default_rng(0)
    lens = [400] + r.integers(1, 60, 299).tolist()
    c = Paged(lens, H, D, 16, seed=1)
    sl = SeqLens(np.concatenate([[0], long + np.arange(300)]), device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    k, v, q = (torch.randn(sl.total, H, D, generator=g, device=DEV).to(torch.bfloat16) for _ in "kvq")
    o, lse = attn_fwd_kv4(q, c.cache, c.table_dev, c.lens_dev, seqlens=sl)
    torch.cuda.synchronize()
    assert get_status() == 0
    pad = long - 400
    assert torch.all(o[:pad] == 0) and torch.all(torch.isneginf(lse[:, :pad]))
    starts = [pad, *range(long, long + 300)]
    cut = lambda x: [x[a:b].transpose(0, 1).double().cpu().numpy() for a, b in zip(starts, starts[1:])]  # noqa: E731
    check_attend(c, cut(q), cut(o), [lse[:, a:b].double().cpu().numpy() for a, b in zip(starts, starts[1:])], D ** -0.5,
                 True, "bf16", "long and short")
    # written and read back: as in a call of the rows that are positions alone
    kv4_write(c.cache, k, v, c.table_dev, c.lens_dev, seqlens=sl)
    got = kv4_read(c.cache, c.table_dev, c.lens_dev, seqlens=sl)
    short = SeqLens(np.concatenate([[0], 400 + np.arange(300)]), device=DEV)
    other = Paged(lens, H, D, 16, seed=1)
    kv4_write(other.cache, k[pad:].contiguous(), v[pad:].contiguous(), other.table_dev, other.lens_dev, seqlens=short)
    want = kv4_read(other.cache, other.table_dev, other.lens_dev, seqlens=short)
    torch.cuda.synchronize()
    assert get_status() == 0
    for a, b in zip(got, want):
        assert torch.all(a[:pad] == 0) and torch.equal(a[pad:], b)
    for name in ("k_codes", "v_codes"):
        assert torch.equal(getattr(c.cache, name), getattr(other.cache, name))
