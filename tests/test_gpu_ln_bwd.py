"""LayerNorm's backward pass and the forward pass with dropout on the GPU, against the
float64 oracle.

Tolerances, with u = 2^-24 (float32's half step), n columns, R rows, per element:
  dr    xh has two roundings (2u).  A row's sums run over at most 32 terms in a thread, 5
        exchanges and 16 warps, so each term passes at most 56 additions; with its products and the
        division by n a sum is off by at most 60u sum|terms| / n.  The rest is six operations on
        the terms.  Together: u rstd (8 |g| + 64 mean|g| + |xh| (70 mean|g xh| + 8 |mean(g xh)|)) + 4u
        (|dr| + |dh|), and half a step of the type (finfo.eps / 2) of dr.
  dx    the same, times the factor, and three more roundings (3u |dx|).
  dgamma, dbeta
        a column's term passes at most R / 152 + 1 additions in a thread (R / 256 and more rows at once where one
        cluster does it all and R is above 256), 64 in a block, 304 / 16 + 16 or 8 in the join, and has at most
        4 roundings of its own: (R / 152 + 108) u sum|terms|.
  forward with dropout: as tests/test_gpu_ln.py, h in addition off by the factor's and the product's
        rounding: (eps / 2) |h| + 4u (|D(x)| + |h|).
"""

import ctypes
import threading

import numpy as np
import pytest
import torch

from bwd_flashattention_fwd_sm_gb300 import _lib, attn_bwd, attn_fwd, dropout, embedding, embedding_bwd
from bwd_flashattention_fwd_sm_gb300 import get_status, layernorm_residual, layernorm_residual_bwd
from bwd_flashattention_fwd_sm_gb300._lib import LnBwdParamsC, LnDropoutC
from oracle import rows as R

from parity_util import compare

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def make(rows, cols, dtype, seed, dh=True, gamma=True):
    g = torch.Generator().manual_seed(seed)
    dt = DTYPES[dtype]
    h = (torch.randn(rows, cols, generator=g) * 2 + 0.5).to(dt)
    dy = torch.randn(rows, cols, generator=g).to(dt)
    mean = h.double().mean(1)
    rstd = 1 / torch.sqrt((h.double() - mean[:, None]).square().mean(1) + 1e-5)
    return dict(dy=dy, h=h, mean=mean.float(), rstd=rstd.float(),
                gamma=torch.randn(cols, generator=g) * 0.5 + 1 if gamma else None,
                dh=torch.randn(rows, cols, generator=g).to(dt) if dh else None)


def check(got, inp, p=0.0, seed=0, offset=0, rows=None):
    """rows: the row numbers, where inp and the first two of got hold some rows of a larger tensor (the other two
    are not looked at then)."""
    dy, h, mean, rstd, gamma, dh = (f64(inp[n]) for n in ("dy", "h", "mean", "rstd", "gamma", "dh"))
    dx, dr, dgamma, dbeta = (f64(t) for t in got)
    half = torch.finfo(inp["dy"].dtype).eps / 2
    ref, rgamma, rbeta = R.ln_bwd(dy, h, mean, rstd, gamma, dh)
    g = dy if gamma is None else dy * gamma
    xh = (h - mean[:, None]) * rstd[:, None]
    av = lambda t: t.mean(1, keepdims=True)
    wide = U * rstd[:, None] * (8 * np.abs(g) + 64 * av(np.abs(g))
                                + np.abs(xh) * (70 * av(np.abs(g * xh)) + 8 * np.abs(av(g * xh))))
    wide = wide + 4 * U * (np.abs(ref) + (0 if dh is None else np.abs(dh)))
    assert np.all(np.abs(dr - ref) <= wide + half * np.abs(ref)), "dr"
    if p > 0:
        t = np.floor(65536 * p + 0.5)
        refx = R.dropout(ref, p, seed, offset, rows)
        keep = R.dropout_bits(ref.shape[0] if rows is None else rows, ref.shape[1], seed, offset) >= t
        assert not dx[~keep].any(), "dropped"
        assert np.all(np.abs(dx - refx) <= wide * (65536 / (65536 - t)) + (half + 3 * U) * np.abs(refx)), "dx"
    else:
        assert np.array_equal(dx, dr)
    if rows is None and dgamma is not None:
        n = (dy.shape[0] / 152 + 108) * U
        assert np.all(np.abs(dgamma - rgamma) <= n * np.abs(dy * xh).sum(0)), "dgamma"
        assert np.all(np.abs(dbeta - rbeta) <= n * np.abs(dy).sum(0)), "dbeta"


def run(inp, **kw):
    d = {n: None if t is None else t.cuda() for n, t in inp.items()}
    return layernorm_residual_bwd(d["dy"], d["h"], d["mean"], d["rstd"], d["gamma"], d["dh"], **kw)


SHAPES = [(130000, 1), (64, 2048), (65, 2048), (128, 1024), (131, 1001), (8, 16380), (16, 4097), (1, 1), (2, 3), (3, 7),
          (1, 16), (300, 64), (9, 100), (33, 256), (7, 257), (64, 1000), (17, 1024), (5, 1030), (40, 2048), (23, 2049), (128, 4096), (33, 4104), (19, 5000), (12, 8192), (6, 8200), (4, 12289), (8, 16384),
          (5, 16383), (3000, 48), (700, 520)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_against_the_formula(shape, dtype):
    rows, cols = shape
    inp = make(rows, cols, dtype, seed=rows + cols)
    check(run(inp), inp)
    check(run(inp, dropout_p=0.3, seed=rows, offset=cols), inp, 0.3, rows, cols)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [72, 2056])
def test_without_what_is_optional(cols, dtype):
    inp = make(50, cols, dtype, seed=1, dh=False, gamma=False)
    check(run(inp), inp)
    check(run(inp, dropout_p=0.5, seed=1), inp, 0.5, 1, 0)
    dx, dr, dgamma, dbeta = run(inp, weight_grads=False)
    assert dgamma is None and dbeta is None
    check((dx, dr, None, None), inp)
    dx, dr, dgamma, dbeta = layernorm_residual_bwd(*(inp[n][:0].cuda() for n in ("dy", "h", "mean", "rstd")))
    assert dx.shape == (0, cols) and not dgamma.any() and not dbeta.any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_everything_is_dropped(dtype):
    inp = make(9, 200, dtype, seed=2)
    dx, dr, _, _ = run(inp, dropout_p=1.0)
    assert not dx.any()
    check((dr, dr, None, None), inp)


def test_nan_and_infinity_stay_in_their_row():
    """A row of NaN reaches its own dr and the columns' sums, and no other row; what is dropped of it is 0."""
    inp = make(20, 300, "f32", seed=3)
    clean = run(inp, dropout_p=0.5, seed=4)
    for bad in (float("nan"), float("inf")):
        broken = {n: None if t is None else t.clone() for n, t in inp.items()}
        broken["dh"][7] = bad
        dx, dr, dgamma, dbeta = run(broken, dropout_p=0.5, seed=4)
        keep = torch.from_numpy(R.dropout_bits(20, 300, 4, 0) >= 32768)[7]
        others = torch.arange(20) != 7
        assert torch.equal(dx.cpu()[others], clean[0].cpu()[others])
        assert torch.equal(dr.cpu()[others], clean[1].cpu()[others])
        assert not dx.cpu()[7][~keep].any() and not torch.isfinite(dx.cpu()[7][keep]).any()
        assert torch.equal(dgamma, clean[2]) and torch.equal(dbeta, clean[3])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows_sampled(dtype):
    """More rows than blocks many times over; dgamma and dbeta in full."""
    for rows, cols in ((100003, 32), (16384, 1024), (5000, 4096)):
        inp = make(rows, cols, dtype, seed=rows)
        got = run(inp, dropout_p=0.1, seed=5, offset=6)
        check(got, inp, 0.1, 5, 6)


def test_same_bits_every_time_and_on_any_workspace():
    inp = make(3001, 1500, "bf16", seed=8)
    a = run(inp, dropout_p=0.1, seed=1)
    ws = torch.full((1 << 24,), 0xFF, dtype=torch.uint8, device="cuda")
    for kw in ({}, {"workspace": ws}):
        b = run(inp, dropout_p=0.1, seed=1, **kw)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_views():
    """Rows a fixed number of elements apart are used as they are; other views are copied."""
    inp = make(24, 208, "bf16", seed=9)
    ref = run(inp, dropout_p=0.2, seed=3)
    wide = {n: torch.full((24, 240), float("nan"), dtype=torch.bfloat16).cuda() for n in ("dy", "h", "dh")}
    for off in (0, 8, 5):
        d = {n: None if t is None else t.cuda() for n, t in inp.items()}
        for n in wide:
            wide[n].fill_(float("nan"))
            wide[n][:, off:off + 208] = d[n]
            d[n] = wide[n][:, off:off + 208]
        got = layernorm_residual_bwd(d["dy"], d["h"], d["mean"], d["rstd"], d["gamma"], d["dh"], dropout_p=0.2, seed=3)
        check(got, inp, 0.2, 3, 0)
        if off != 5:
            assert all(torch.equal(x, y) for x, y in zip(ref, got))
    t = {n: inp[n].cuda() for n in ("dy", "h", "dh")}
    d = {n: v.t().contiguous().t() for n, v in t.items()}
    got = layernorm_residual_bwd(d["dy"], d["h"], inp["mean"].cuda(), inp["rstd"].cuda(), inp["gamma"].cuda(), d["dh"],
                                 dropout_p=0.2, seed=3)
    assert all(torch.equal(x, y) for x, y in zip(ref, got))
    shaped = layernorm_residual_bwd(t["dy"].view(4, 6, 208), t["h"].view(4, 6, 208), inp["mean"].cuda().view(4, 6),
                                    inp["rstd"].cuda().view(4, 6), inp["gamma"].cuda(), t["dh"].view(4, 6, 208),
                                    dropout_p=0.2, seed=3)
    assert shaped[0].shape == (4, 6, 208) and torch.equal(shaped[0].view(24, 208), ref[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [5, 130, 1000, 2049, 4096, 7001, 12288, 16384])
def test_tensors_that_begin_at_different_places(cols, dtype):
    """h one element off 16 bytes, dh with wider rows, dy and the outputs in place: no form that moves whole rows."""
    inp = make(70, cols, dtype, seed=cols)
    d = {n: None if t is None else t.cuda() for n, t in inp.items()}
    off = torch.full((70 * cols + 1,), float("nan"), dtype=DTYPES[dtype], device="cuda")
    off[1:] = d["h"].view(-1)
    wide = torch.full((70, cols + 24), float("nan"), dtype=DTYPES[dtype], device="cuda")
    wide[:, :cols] = d["dh"]
    got = layernorm_residual_bwd(d["dy"], off[1:].view(70, cols), d["mean"], d["rstd"], d["gamma"], wide[:, :cols],
                                 dropout_p=0.2, seed=3)
    check(got, inp, 0.2, 3, 0)
    # the same in the forward pass
    x, r = inp["dy"], inp["dh"]
    off[1:] = x.cuda().view(-1)
    y, h, mean, rstd = layernorm_residual(off[1:].view(70, cols), wide[:, :cols], d["gamma"], return_stats=True,
                                          dropout_p=0.2, seed=3)
    ref = R.ln_dropout_residual(f64(x), f64(r), f64(inp["gamma"]), None, 1e-5, 0.2, 3, 0)
    if cols > 5:  # five columns may be nearly alike, and y then as far off as 1 / std says
        compare("y", f64(y), ref[0], dtype)
    half = torch.finfo(x.dtype).eps / 2
    assert np.all(np.abs(f64(h) - ref[1]) <= half * np.abs(ref[1]) + 4 * U * (np.abs(f64(x)) / 0.8 + np.abs(ref[1])))


@pytest.mark.parametrize("cols, step", [(100, 104), (100, 101), (1024, 1032), (2048, 2056), (4096, 4100), (9000, 9008)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_c_entry_writes_nothing_between_rows_or_behind(cols, step, dtype):
    """Outputs with gaps between their rows, in buffers with a pattern around them and a workspace of exactly the size
    asked for; dx and dr in place of dy and dh."""
    lib, rows, dt = _lib.load(), 37, DTYPES[dtype]
    inp = make(rows, cols, dtype, seed=cols)
    ref = run(inp, dropout_p=0.2, seed=3, offset=1)

    def strided(src=None):
        buf = torch.full((rows * step + 64,), 7.0, dtype=dt, device="cuda")
        view = buf[32:32 + rows * step].view(rows, step)
        if src is not None:
            view[:, :cols] = src.cuda()
        return buf, view

    def intact(buf, view):
        return bool((buf[:32] == 7).all()) and bool((buf[32 + rows * step:] == 7).all()) and bool(
            (view[:, cols:] == 7).all())

    p = LnBwdParamsC(rows, cols, step, step, step, step, step, inp_dtype(dt))
    d = LnDropoutC(0.2, 3, 1, None)
    need = lib.ln_residual_bwd_workspace_size(p)
    mean, rstd, gamma = (inp[n].cuda() for n in ("mean", "rstd", "gamma"))
    for in_place in (False, True):
        dy, h, dh = strided(inp["dy"]), strided(inp["h"]), strided(inp["dh"])
        dx, dr = (dy, dh) if in_place else (strided(), strided())
        ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
        sums = torch.full((2 * cols + 64,), 7.0, device="cuda")
        code = lib.ln_residual_bwd(p, d, dy[1].data_ptr(), dh[1].data_ptr(), h[1].data_ptr(), mean.data_ptr(),
                                   rstd.data_ptr(), gamma.data_ptr(), dx[1].data_ptr(), dr[1].data_ptr(),
                                   sums[16:].data_ptr(), sums[32 + cols:].data_ptr(), ws.data_ptr(), need,
                                   ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert code == 0
        torch.cuda.synchronize()
        assert bool((ws[need:] == 0x5A).all())
        assert intact(*dx) and intact(*dr) and intact(*h)
        assert bool((sums[:16] == 7).all()) and bool((sums[16 + cols:32 + cols] == 7).all())
        assert bool((sums[32 + 2 * cols:] == 7).all())
        got = (dx[1][:, :cols], dr[1][:, :cols], sums[16:16 + cols], sums[32 + cols:32 + 2 * cols])
        check(got, inp, 0.2, 3, 1)
        if (step * dt.itemsize) % 16 == 0 and (cols * dt.itemsize) % 16 == 0:  # else the order of the sums differs
            assert all(torch.equal(x, y) for x, y in zip(ref, got))


def inp_dtype(dt):
    return _lib.ATTN_BF16 if dt == torch.bfloat16 else _lib.ATTN_F32


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(3, 7), (64, 1000), (128, 4096), (33, 4104), (8, 16384), (5, 2049), (11, 8192),
                                   (2000, 64), (1001, 101), (700, 128), (5000, 250), (40, 30), (3, 16), (9, 300),
                                   (50, 520), (400, 16384), (301, 16370), (90, 12290), (3, 9000)],
                         ids=lambda s: f"{s[0]}x{s[1]}")
def test_forward_with_dropout(shape, dtype):
    rows, cols = shape
    g = torch.Generator().manual_seed(rows)
    x = (torch.randn(rows, cols, generator=g) * 2 + 0.5).to(DTYPES[dtype])
    r = torch.randn(rows, cols, generator=g).to(DTYPES[dtype])
    gamma, beta = torch.randn(cols, generator=g) * 0.5 + 1, torch.randn(cols, generator=g) * 0.1
    for res in (r, None):
        y, h, mean, rstd = (f64(t) for t in layernorm_residual(
            x.cuda(), None if res is None else res.cuda(), gamma.cuda(), beta.cuda(), return_stats=True,
            dropout_p=0.3, seed=rows, offset=cols))
        dropped = R.dropout(f64(x), 0.3, rows, cols)
        ry, rh, rmean, rrstd = R.ln_dropout_residual(f64(x), f64(res), f64(gamma), f64(beta), 1e-5, 0.3, rows, cols)
        compare("y", y, ry, dtype)
        half = torch.finfo(x.dtype).eps / 2
        assert np.all(np.abs(h - rh) <= half * np.abs(rh) + 4 * U * (np.abs(dropped) + np.abs(rh)))
        scale = np.abs(rmean) + 1.0 / rrstd
        assert np.all(np.abs(mean - rmean) <= 1e-5 * scale) and np.all(np.abs(rstd - rrstd) <= 1e-5 * rrstd)


def test_forward_without_dropout_keeps_its_bits():
    """p = 0, or below half a step of the rate, is the call without dropout."""
    x = torch.randn(100, 1000, device="cuda").to(torch.bfloat16)
    a = layernorm_residual(x, x, return_stats=True)
    for p in (0.0, 2.0 ** -18):
        assert all(torch.equal(s, t) for s, t in zip(a, layernorm_residual(x, x, return_stats=True, dropout_p=p, seed=3)))


def test_two_streams_and_two_graphs():
    """Two problems queued on two streams at once, then as two captured graphs replayed together: each call has its
    own workspace, so the results are those of one after the other."""
    problems = [{n: None if t is None else t.cuda() for n, t in make(r, c, "bf16", seed=r).items()}
                for r, c in ((4096, 1024), (3000, 4096))]
    args = [[d[n] for n in ("dy", "h", "mean", "rstd", "gamma", "dh")] for d in problems]
    ref = [layernorm_residual_bwd(*a, dropout_p=0.1, seed=1) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    for _ in range(3):
        got = [layernorm_residual_bwd(*a, dropout_p=0.1, seed=1, stream=s) for a, s in zip(args, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for g, r in zip(got, ref) for x, y in zip(g, r))
    graphs, outs = [], []
    for a in args:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(layernorm_residual_bwd(*a, dropout_p=0.1, seed=1))
        graphs.append(graph)
    for out in outs:
        for t in out:
            t.zero_()
    torch.cuda.synchronize()
    for g, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for g, r in zip(outs, ref) for x, y in zip(g, r))


def test_a_captured_layer_follows_the_pair_on_the_device():
    """Forward and backward pass captured once; each replay drops by the pair's values of its time."""
    x = torch.randn(40, 520, device="cuda").to(torch.bfloat16)
    dy, rng = torch.randn_like(x), torch.zeros(2, dtype=torch.int64, device="cuda")

    def layer(**kw):
        y, h, mean, rstd = layernorm_residual(x, None, return_stats=True, dropout_p=0.3, **kw)
        return (y, h, *layernorm_residual_bwd(dy, h, mean, rstd, dropout_p=0.3, **kw))

    layer(rng=rng, offset=5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(rng=rng, offset=5)
    for seed, offset in ((3, 4), (-9, 2 ** 40)):
        rng.copy_(torch.tensor([seed, offset]))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, layer(seed=seed, offset=offset + 5)))


def test_two_threads():
    """Calls of different sizes from two host threads at once: each launch finds its kernel's limits set for it."""
    args, kw = [], dict(dropout_p=0.1, seed=1)
    for rows, cols in ((300, 4096), (200, 2000), (300, 2056), (160, 8192), (700, 70), (20, 16384)):
        d = {n: None if t is None else t.cuda() for n, t in make(rows, cols, "bf16", seed=rows).items()}
        args.append([d[n] for n in ("dy", "h", "mean", "rstd", "gamma", "dh")])

    def both(a):
        return (*layernorm_residual_bwd(*a, **kw), *layernorm_residual(a[0], a[1], a[4], **kw))

    ref = [both(a) for a in args]
    torch.cuda.synchronize()
    wrong, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]

    def work(which):
        try:
            with torch.cuda.stream(streams[which]):
                for i in range(60):
                    k = (i * (which + 1) + which) % len(args)
                    if not all(torch.equal(x, y) for x, y in zip(both(args[k]), ref[k])):
                        wrong.append(k)
        except Exception as e:  # what a thread raises would be lost
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(w,)) for w in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("cols", [4096, 4099, 40])
def test_offsets_beyond_31_bits(cols):
    """Tensors of more elements than 31 bits count; sampled rows, the last among them, and the sums' magnitude."""
    rows = ((1 << 31) + (1 << 20)) // cols
    dy = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    dy.normal_()
    h = torch.empty_like(dy).normal_(0.5, 2.0)
    mean, rstd = torch.full((rows,), 0.5, device="cuda"), torch.full((rows,), 0.5, device="cuda")
    dx, dr, dgamma, dbeta = layernorm_residual_bwd(dy, h, mean, rstd, dropout_p=0.1, seed=1, offset=2)
    at = torch.tensor([0, 1, 7, 8, rows // 2, rows - 9, rows - 1])
    inp = dict(dy=dy[at], h=h[at], mean=mean[at], rstd=rstd[at], gamma=None, dh=None)
    check((dx[at], dr[at], None, None), {n: None if t is None else t.cpu() for n, t in inp.items()}, 0.1, 1, 2,
          rows=at.numpy())
    # sums of about 2^31 / cols terms: against the same in 64 bits, by pieces
    ref, size = torch.zeros(cols, dtype=torch.float64, device="cuda"), torch.zeros(cols, dtype=torch.float64, device="cuda")
    for i in range(0, rows, rows // 64 + 1):
        part = dy[i:i + rows // 64 + 1].double()
        ref += part.sum(0)
        size += part.abs().sum(0)
    assert bool(((dbeta.double() - ref).abs() <= (rows / 152 + 108) * U * size).all())
    del dx, dr
    x, out = dy, layernorm_residual(dy, h, dropout_p=0.1, seed=1, offset=2)
    y, hh = out
    ref = R.dropout(f64(x[at]), 0.1, 1, 2, at.numpy()) + f64(h[at])
    assert np.all(np.abs(f64(hh[at]) - ref) <= 2.0 ** -8 * np.abs(ref) + 8 * U * (np.abs(f64(x[at])) + np.abs(ref)))
    assert bool(torch.isfinite(y[-1].float()).all()) and get_status() == 0


def test_a_small_model_forward_and_backward():
    """The operators as a model uses them: a table's rows, dropout + add + norm, attention on the normed rows, dropout +
    add + norm again, and all of it backwards; the gradients against float64 autograd of the same masks.

    Everything is float32, so each operator is off by some tens of u of its terms' magnitudes and
    the whole by that times the chain's length and condition; 1e-4 of a gradient's largest element leaves
    a factor of several tens and would show a wrong factor, mask, row or missing term at once."""
    B, S, H, D, V, p, seed = 2, 40, 2, 64, 50, 0.2, 11
    C = H * D
    g = torch.Generator().manual_seed(1)
    table, place = torch.randn(V, C, generator=g), torch.randn(S, C, generator=g)
    ids = torch.randint(0, V, (B, S), generator=g)
    ga, ba, gb, bb = (torch.randn(C, generator=g) * 0.3 + k for k in (1, 0, 1, 0))
    dy = torch.randn(B, S, C, generator=g)
    masks = [torch.from_numpy(R.dropout(np.ones((B * S, C)), p, seed, k)).view(B, S, C).cuda() for k in range(3)]

    # float64, from the definitions
    leaves = [t.double().cuda().requires_grad_() for t in (table, place, ga, ba, gb, bb)]
    T, P, GA, BA, GB, BB = leaves

    def norm(h, w, b):
        m = h.mean(-1, keepdim=True)
        return (h - m) / torch.sqrt((h - m).square().mean(-1, keepdim=True) + 1e-5) * w + b

    def heads(t):
        return t.view(B, S, H, D).transpose(1, 2)

    h1 = masks[0] * (T[ids.cuda()] * 4.0) + P
    n1 = norm(h1, GA, BA)
    s = heads(n1) @ heads(n1).transpose(-1, -2) / D ** 0.5
    s = s.masked_fill(torch.ones(S, S, device="cuda").triu(1).bool(), -torch.inf)
    att = (torch.softmax(s, -1) @ heads(n1)).transpose(1, 2).reshape(B, S, C)
    h2 = masks[1] * att + h1
    y = masks[2] * norm(h2, GB, BB)
    ref = torch.autograd.grad(y, leaves, dy.double().cuda())

    # the operators
    cu = [t.cuda() for t in (table, place, ga, ba, gb, bb, dy)]
    T, P, GA, BA, GB, BB, dY = cu
    rng = torch.tensor([seed, 0], device="cuda")
    drop = lambda k: dict(dropout_p=p, offset=k, rng=rng)
    emb = embedding(T, ids.cuda(), scale=4.0)
    n1, h1, m1, r1 = layernorm_residual(emb, P.expand(B, S, C), GA, BA, return_stats=True, **drop(0))
    q = heads(n1).contiguous()
    o, lse = attn_fwd(q, q, q, causal=True)
    att = o.transpose(1, 2).reshape(B, S, C)
    n2, h2, m2, r2 = layernorm_residual(att, h1, GB, BB, return_stats=True, **drop(1))
    out = dropout(n2, p, offset=2, rng=rng)
    assert float((out.double() - y.detach()).abs().max()) <= 1e-4 * float(y.detach().abs().max())

    dn2 = dropout(dY, p, offset=2, rng=rng)
    datt, dh1, dgb, dbb = layernorm_residual_bwd(dn2, h2, m2, r2, GB, **drop(1))
    dq, dk, dv = attn_bwd(q, q, q, o, heads(datt).contiguous(), lse, causal=True)
    dn1 = (dq + dk + dv).transpose(1, 2).reshape(B, S, C)
    demb, dres, dga, dba = layernorm_residual_bwd(dn1, h1, m1, r1, GA, dh1, **drop(0))
    dtable = embedding_bwd(demb, ids.cuda(), V, scale=4.0)
    for name, a, b in zip(("table", "place", "gamma1", "beta1", "gamma2", "beta2"),
                          (dtable, dres.sum(0), dga, dba, dgb, dbb), ref):
        assert float((a.double() - b).abs().max()) <= 1e-4 * float(b.abs().max()), name
    assert get_status() == 0
