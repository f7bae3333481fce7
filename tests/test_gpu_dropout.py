"""Dropout on the GPU: the mask has to be the oracle's, element by element, and what stays
is one product.

Tolerance.  The factor is rounded to float32 (2^-24) and so is the product (2^-24); the
result is rounded to the tensor's type (finfo.eps / 2): eps / 2 + 2^-22 relative
covers them and their products.
"""

import numpy as np
import pytest
import torch

from bwd_flashattention_fwd_sm_gb300 import dropout, get_status, layernorm_residual, layernorm_residual_bwd
from bwd_flashattention_fwd_sm_gb300._lib import AttnError
from oracle import rows as R

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    return (x + torch.sign(x)).to(DTYPES[dtype])  # no zeros: a zero in the result was dropped


def check(got, x, p, seed, offset, rows=None):
    cols = x.shape[-1]
    got = got.double().cpu().numpy().reshape(-1, cols)
    ref = R.dropout(x.double().cpu().numpy().reshape(-1, cols), p, seed, offset, rows)
    assert np.array_equal(got == 0, ref == 0)
    tol = torch.finfo(x.dtype).eps / 2 + 2.0 ** -22
    assert np.all(np.abs(got - ref) <= tol * np.abs(ref))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (1, 8), (5, 9), (257, 64), (1000, 1), (33, 1003), (2, 3, 40),
                                   (70000,), (4, 16384), (611, 2050)], ids=str)
def test_mask_and_values(shape, dtype):
    x = make(shape, dtype, 5)
    for p, seed, offset in ((0.1, 1, 2), (0.5, -3, 2 ** 63 + 5), (0.99, 2 ** 40, 0)):
        got = dropout(x.cuda(), p, seed=seed, offset=offset)
        assert got.shape == x.shape and got.dtype == x.dtype
        check(got, x, p, seed, offset)


def test_ends_of_the_range():
    x = make((37, 100), "bf16", 1).cuda()
    assert torch.equal(dropout(x, 0.0), x)
    assert torch.equal(dropout(x, 2.0 ** -18), x)  # below half a step of the rate
    assert not dropout(x, 1.0).any()
    check(dropout(x, 1 - 2.0 ** -16, seed=3), x, 1 - 2.0 ** -16, 3, 0)
    for shape in ((0, 8), (8, 0), (0,)):
        e = torch.empty(shape, device="cuda")
        assert dropout(e, 0.5).shape == e.shape


def test_what_is_dropped_is_zero_whatever_it_held():
    for bad in (float("nan"), float("inf"), torch.finfo(torch.float32).min):
        x = torch.full((64, 128), bad, device="cuda")
        got = dropout(x, 0.5, seed=9)
        keep = torch.from_numpy(R.dropout_bits(64, 128, 9, 0) >= 32768)
        assert not got.cpu()[~keep].any()
        assert torch.equal(got.cpu()[keep], (x.cpu() * 2)[keep]) or (torch.isnan(got.cpu()[keep]).all() and bad != bad)


def test_pair_on_the_device_is_added_and_read_when_the_kernel_runs():
    x = make((40, 96), "f32", 2).cuda()
    rng = torch.tensor([2 ** 62, -7], device="cuda")
    check(dropout(x, 0.3, seed=2 ** 63 + 11, offset=5, rng=rng), x, 0.3, 2 ** 62 + 2 ** 63 + 11, -2)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        dropout(x, 0.3, rng=rng)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        y = dropout(x, 0.3, rng=rng)
    for seed, offset in ((1, 1), (1, 2), (-5, 2 ** 40)):
        rng.copy_(torch.tensor([seed, offset]))
        graph.replay()
        check(y, x, 0.3, seed, offset)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_views_and_in_place(dtype):
    base = make((20, 3, 80), dtype, 4).cuda()
    for view in (base[:, 1], base[..., 8:72], base[..., 1:70], base.transpose(0, 1), base[::2], base[..., ::2]):
        check(dropout(view, 0.2, seed=8, offset=1), view.contiguous(), 0.2, 8, 1)
    x = base.clone()
    out = dropout(x, 0.2, seed=8, offset=1, out=x)
    assert out.data_ptr() == x.data_ptr()
    check(out, base, 0.2, 8, 1)
    whole = base.clone().view(-1)
    with pytest.raises(AttnError, match="overlap"):
        dropout(whole[:-8], 0.2, out=whole[8:])
    with pytest.raises(ValueError, match="out"):
        dropout(base, 0.2, out=torch.empty(20, 3, 160, device="cuda", dtype=base.dtype)[..., ::2])


def test_gradient_is_the_same_dropout():
    """dropout is linear in x: <dy, D(x)> = <D(dy), x>, and the masks agree bit for bit."""
    x, dy = make((64, 200), "f32", 1).cuda(), make((64, 200), "f32", 2).cuda()
    y, dx = dropout(x, 0.4, seed=3, offset=4), dropout(dy, 0.4, seed=3, offset=4)
    assert torch.equal(y == 0, dx == 0)
    a, b = (dy.double() * y.double()).sum(), (dx.double() * x.double()).sum()
    assert abs(a - b) <= 2.0 ** -22 * (dy.double() * y.double()).abs().sum()


def test_same_mask_in_front_of_the_norm_and_in_its_backward_pass():
    x = make((50, 328), "bf16", 6).cuda()
    kw = dict(seed=5, offset=6)
    y = dropout(x, 0.25, **kw)
    _, h, mean, rstd = layernorm_residual(x, return_stats=True, dropout_p=0.25, **kw)
    assert torch.equal(h, y)
    dh = make((50, 328), "bf16", 7).cuda()
    dx, dr, _, _ = layernorm_residual_bwd(torch.zeros_like(dh), h, mean, rstd, dh=dh, dropout_p=0.25, **kw)
    assert torch.equal(dr, dh)
    assert torch.equal(dx, dropout(dh, 0.25, **kw))


def test_far_rows_and_a_long_row():
    """Sampled rows of a tensor with more elements than 31 bits count, and the end of one row as long."""
    n = (1 << 31) + 24
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y = dropout(x, 0.5, seed=1, offset=2, out=x)
    cols = (n + 7) // 8 * 8
    words = R.philox4x32([np.arange(cols // 8 - 8, cols // 8), np.zeros(8), np.full(8, 2), np.zeros(8)], (1, 0), 7)
    bits = np.stack([(words[e // 2] >> np.uint64(16 * (e % 2))) & np.uint64(0xFFFF) for e in range(8)], 1).ravel()
    assert np.array_equal(y[-64:].float().cpu().numpy() != 0, bits >= 32768)
    assert abs(float((y[::4097] == 0).float().mean()) - 0.5) < 5 * 0.5 / np.sqrt(n / 4097)
    x.fill_(1)
    y = dropout(x.view(-1, 8), 0.5, seed=1, offset=2)
    for row in (0, 12345678, n // 8 - 1):
        check(y[row:row + 1], torch.ones(1, 8, dtype=torch.bfloat16), 0.5, 1, 2, rows=[row])
    assert get_status() == 0


def test_on_another_stream():
    x = make((2048, 1024), "bf16", 3).cuda()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = dropout(x, 0.1, seed=1, stream=s)
    s.synchronize()
    check(y, x, 0.1, 1, 0)
