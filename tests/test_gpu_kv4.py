"""GPU tests of the 4-bit key/value cache against its oracle (oracle/kv4.py, float64).

kv4_write, kv4_read: bit-identical to the oracle (each code is decided in float32 on
both sides; a value read back is s (u - 8) + b, exact but for one float32 rounding,
then one to the output's type); every byte that no row names stays as it was.

attn_fwd_kv4, element by element.  eps = 2^-24 is half a float32 step at 1.  A score
is a float32 sum of D / 64 group sums of 64 products plus offsets: off by at most
(D + 16) eps W with W = scale sum |q| (16 s + |b|); exp2's approximation adds 2^-21
and sums over n positions n eps.  So each p is off by d = (D + 16) eps W + n eps +
2^-21 of itself, O by at most 2 d A (numerator and sum) with A = sum p (|s (u - 8)| +
|b|), LSE by d + 4 eps |LSE|.  The weights p s are float16 in units of 2^e / 2^7, 2^(e - 1)
<= the largest step s of the head: off by 2^-11 of themselves (float32: two parts, 2^-23),
and below float16's normal range by half its least step, 2^-25 units <= 2^-31 of the
largest s.  With |u - 8| <= 8 and sum p >= 1 in the units that the maximum sets: 2^-11
R (2^-23 R), R = sum p |s (u - 8)|, and n 2^-28 max s.  With more than 24 bfloat16 query
rows on a KV head (head dim 64 or 128) the rounded weights are p alone, in units in which 1
is 2^7, and offsets are multiplied by them too: p' = p (1 + e), |e| <= 2^-11, or off by
2^-25 = 2^-32 of 1 below the normal range, so that sum p' (s (u - 8) + b) is off by 2^-11 A
and n 2^-32 (8 max s + max |b|); s (u - 8) itself is float16 in units in which the largest s
is at least 2^11, off by 2^-36 of that (n 2^-28 max s has room for both).  O is rounded
once: 2^-8 |O| for bfloat16, eps |O| for float32.
"""

import numpy as np
import pytest
import torch

from bwd_flashattention_fwd_sm_gb300 import (Kv4Cache, SeqLens, _lib, attn_fwd, attn_fwd_kv4, get_status, kv4_read,
                                             kv4_write)
from oracle import kv4

from parity_util import _log_margin

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
EPS = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


class Paged:
    """A cache with random rows in it (quantised by the oracle), pages in random order;
    what no sequence holds is NaN scales and random codes."""

    def __init__(self, lens, Hkv, D, page, seed, spare=2):
        r = np.random.default_rng(seed)
        self.lens, self.page, self.D, self.Hkv = list(lens), page, D, Hkv
        per = [-(-n // page) for n in lens]
        self.n_pages, width = sum(per) + spare, max(per + [1])
        order = r.permutation(self.n_pages)
        self.table = np.zeros((len(lens), width), np.int32)
        self.codes = [r.integers(0, 256, (self.n_pages, Hkv, page, D // 2), dtype=np.uint8) for _ in "kv"]
        self.scale = [np.full((self.n_pages, Hkv, page, D // 64, 2), np.nan, np.float32) for _ in "kv"]
        at = 0
        for n, (length, count) in enumerate(zip(lens, per)):
            ids = order[at : at + count]
            at += count
            self.table[n, :count] = ids
            for c, s in zip(self.codes, self.scale):
                x = r.normal(size=(Hkv, length, D)).astype(np.float32) * r.choice([0.3, 1, 2], (Hkv, length, 1)) + 0.2
                u, st, b = kv4.quantise(x)
                for j in range(length):
                    c[ids[j // page], :, j % page] = kv4.pack(u[:, j])
                    s[ids[j // page], :, j % page, :, 0], s[ids[j // page], :, j % page, :, 1] = st[:, j], b[:, j]
        gpu = [torch.from_numpy(c).to(DEV) for c in self.codes]
        gpus = [torch.from_numpy(s).to(DEV).to(torch.bfloat16) for s in self.scale]
        self.cache = Kv4Cache(gpu[0], gpu[1], gpus[0], gpus[1])
        self.table_dev = torch.from_numpy(self.table).to(DEV)
        self.lens_dev = torch.tensor(self.lens, dtype=torch.int32, device=DEV)

    def rows(self, n, which):
        return kv4.rows(self.codes[which], self.scale[which], self.table[n], self.page, self.lens[n])


def check_attend(c, q, o, lse, scale, causal, dtype, name):
    """q, o [n][Hq, t, D] and lse [n][Hq, t] as lists over the sequences."""
    worst = [0.0, 0.0]
    for n in range(len(c.lens)):
        t = q[n].shape[1]
        if c.lens[n] == 0:
            ku = np.zeros((c.Hkv, 0, c.D), np.uint8), np.zeros((c.Hkv, 0, c.D // 64)), np.zeros((c.Hkv, 0, c.D // 64))
            vu = ku
        else:
            ku, vu = c.rows(n, 0), c.rows(n, 1)
        ro, rl, A, R, W = kv4.attend(q[n], kv4.parts(*ku), kv4.parts(*vu), ku[1], scale, causal)
        d = (c.D + 16) * EPS * W + c.lens[n] * EPS + 2.0 ** -21
        go, gl = o[n].astype(np.float64), lse[n].astype(np.float64)
        assert np.array_equal(np.isneginf(gl), np.isneginf(rl)), name
        empty = np.isneginf(rl)
        assert np.all(go[empty] == 0)
        tol = 2 * d[..., None] * A
        many = dtype == "bf16" and c.D <= 128 and max(x.shape[1] for x in q) * (q[n].shape[0] // c.Hkv) > 24
        tol += 2.0 ** -11 * (A if many else R) + 2.0 ** -8 * np.abs(ro) * (1 + 2.0 ** -8) if dtype == "bf16" else 2 * EPS * (R + np.abs(ro))
        if c.lens[n]:
            tol += c.lens[n] * 2.0 ** -28 * np.repeat(vu[1].max((1, 2)), go.shape[0] // c.Hkv)[:, None, None]
            if many:
                tol += c.lens[n] * 2.0 ** -32 * np.repeat(np.abs(vu[2]).max((1, 2)), go.shape[0] // c.Hkv)[:, None, None]
        err = np.abs(go - ro)
        lerr = np.abs(np.where(empty, 0, gl) - np.where(empty, 0, rl))[~empty]
        ltol = (d + 4 * EPS * np.abs(np.where(empty, 0, rl)))[~empty]
        ok = err <= tol + 1e-30
        assert np.all(ok), f"{name}: sequence {n}: max err/tol {np.max(err / (tol + 1e-30)):.3f}"
        assert np.all(lerr <= ltol), f"{name}: sequence {n}: LSE {np.max(lerr / ltol):.3f}"
        if err.size and not np.all(empty):
            worst = [max(worst[0], float(np.max(err / (tol + 1e-30)))), max(worst[1], float(np.max(lerr / ltol)))]
    _log_margin(f"o[{name}]", dtype, 0.0, 0.0, worst[0], 0)
    _log_margin(f"lse[{name}]", dtype, 0.0, 0.0, worst[1], 0)


def attend_fixed(c, Hq, t, dtype, seed, scale, causal=True, **kw):
    q = torch.randn(len(c.lens), Hq, t, c.D, generator=torch.Generator().manual_seed(seed)).to(DT[dtype])
    o, lse = attn_fwd_kv4(q.to(DEV), c.cache, c.table_dev, c.lens_dev, causal=causal, scale=scale, **kw)
    torch.cuda.synchronize()
    assert get_status() == 0
    return q.double().numpy(), o.double().cpu().numpy(), lse.double().cpu().numpy()


# ---------------------------------------------------------------- write and read


def new_rows(counts, Hkv, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return [tuple((torch.randn(Hkv, t, D, generator=g) * 2 + 0.3).to(DT[dtype]) for _ in "kv") for t in counts]


def expected_write(c, news):
    codes, scale = [x.copy() for x in c.codes], [x.copy() for x in c.scale]
    for n, kv in enumerate(news):
        t = kv[0].shape[1]
        for x, cc, ss in zip(kv, codes, scale):
            u, s, b = kv4.quantise(x.float().numpy())
            for i in range(t):
                pos = c.lens[n] - t + i
                if pos >= 0:
                    p, j = c.table[n, pos // c.page], pos % c.page
                    cc[p, :, j] = kv4.pack(u[:, i])
                    ss[p, :, j, :, 0], ss[p, :, j, :, 1] = s[:, i], b[:, i]
    return codes, scale


def same_cache(c, codes, scale):
    for got, want in zip((c.cache.k_codes, c.cache.v_codes), codes):
        assert np.array_equal(got.cpu().numpy(), want)
    for got, want in zip((c.cache.k_scale, c.cache.v_scale), scale):
        assert np.array_equal(got.float().cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D, Hkv, page, lens, t", [
    (128, 2, 16, [1, 16, 17, 300], 1),
    (64, 3, 48, [100, 5, 0, 48], 7),       # padding in two sequences, one of them empty
    (256, 1, 16, [33], 33),
    (128, 8, 64, [130, 257], 129),
])
def test_write_fixed_is_bit_exact_and_touches_nothing_else(D, Hkv, page, lens, t, dtype):
    c = Paged(lens, Hkv, D, page, seed=D + t)
    news = new_rows([t] * len(lens), Hkv, D, dtype, seed=t)
    k, v = (torch.stack([x[i] for x in news]).to(DEV) for i in (0, 1))
    assert kv4_write(c.cache, k, v, c.table_dev, c.lens_dev) is c.cache
    torch.cuda.synchronize()
    assert get_status() == 0
    same_cache(c, *expected_write(c, news))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_write_and_read_packed(D, dtype):
    lens, counts, Hkv, page = [40, 3, 64, 7, 129], [40, 1, 0, 9, 100], 3, 32  # the fourth has more rows than positions
    c = Paged(lens, Hkv, D, page, seed=D)
    news = new_rows(counts, Hkv, D, dtype, seed=D + 1)
    k, v = (torch.cat([x[i].transpose(0, 1) for x in news]).to(DEV) for i in (0, 1))
    sl = SeqLens(np.concatenate([[0], np.cumsum(counts)]), device=DEV)
    kv4_write(c.cache, k, v, c.table_dev, c.lens_dev, seqlens=sl)
    rk, rv = kv4_read(c.cache, c.table_dev, c.lens_dev, seqlens=sl, dtype=DT[dtype])
    torch.cuda.synchronize()
    assert get_status() == 0
    codes, scale = expected_write(c, news)
    same_cache(c, codes, scale)
    for which, got in enumerate((rk, rv)):
        got = got.cpu()
        for n, t in enumerate(counts):
            rows = got[sl.host[n] : sl.host[n + 1]].transpose(0, 1)
            u, s, b = kv4.quantise(news[n][which].float().numpy())
            want = torch.from_numpy(sum(kv4.parts(u, s, b))).float().to(DT[dtype])
            want[:, : max(0, t - lens[n])] = 0
            assert torch.equal(rows, want), (n, which)


def test_write_equal_values_zeros_and_large_ones():
    c = Paged([6], 1, 64, 16, seed=5)
    x = torch.zeros(1, 1, 6, 64)
    x[0, 0, 1] = -3.5
    x[0, 0, 2] = torch.linspace(-1e30, 1e30, 64)
    x[0, 0, 3] = torch.linspace(0, 1e-37, 64)
    x[0, 0, 4] = torch.linspace(100, 100.5, 64)
    x[0, 0, 5, 0] = 1e-3
    for dtype in ("f32", "bf16"):
        k = x.to(DT[dtype])
        kv4_write(c.cache, k.to(DEV), (-k).to(DEV), c.table_dev, c.lens_dev)
        torch.cuda.synchronize()
        same_cache(c, *expected_write(c, [(k[0], -k[0])]))


def test_read_fixed_into_given_tensors_leaves_their_surroundings():
    c = Paged([70, 20, 0], 2, 128, 16, seed=8)
    S = 33
    buf = torch.full((3, 2, S + 2, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    k, v = buf[:, :, 1:-1], buf.clone()[:, :, 1:-1]
    got = kv4_read(c.cache, c.table_dev, c.lens_dev, S, out=(k, v))
    assert got[0] is k and got[1] is v
    torch.cuda.synchronize()
    assert torch.all(buf[:, :, 0] == 7) and torch.all(buf[:, :, -1] == 7)
    for n, length in enumerate(c.lens):
        have = min(S, length)
        assert torch.all(k[n, :, : S - have] == 0) and torch.all(v[n, :, : S - have] == 0)
        if have:
            for which, out in enumerate((k, v)):
                want = torch.from_numpy(sum(kv4.parts(*c.rows(n, which)))).float().to(torch.bfloat16)[:, -have:]
                assert torch.equal(out[n, :, S - have :].cpu(), want)


# ---------------------------------------------------------------- attention

ATTEND = [
    # D, Hq, Hkv, page, lens, t, causal
    (128, 8, 2, 16, [1], 1, True),
    (128, 8, 2, 16, [0, 1, 15, 16, 17, 31, 33, 128, 129, 1000], 1, True),
    (128, 32, 8, 64, [777, 64, 65], 1, True),
    (64, 16, 16, 32, [500, 3], 1, True),
    (256, 4, 2, 48, [100, 47, 48, 49, 400], 1, True),
    (128, 14, 2, 16, [300, 20], 1, True),          # seven query heads on one
    (128, 16, 1, 256, [700], 1, True),
    (64, 40, 1, 16, [90, 200], 1, False),          # forty
    (128, 8, 2, 16, [40, 3, 0, 260], 5, True),     # padding in two sequences
    (128, 4, 4, 16, [40, 3, 0, 260], 5, False),
    (64, 8, 2, 64, [150, 33], 33, True),
    (256, 8, 4, 16, [75, 20], 19, True),
    (128, 4, 1, 16, [333], 100, True),             # 400 rows on one head
    (128, 2, 1, 128, [2000], 1, True),
    (128, 32, 1, 16, [1, 0, 127, 128, 129, 260], 1, True),   # 32 rows, key tiles of 128
    (64, 24, 1, 48, [130, 700], 3, False),
    (128, 20, 1, 16, [333, 64], 1, True),                    # 20 rows
    (128, 8, 2, 16, [300, 4, 0, 513], 70, True),             # row tiles of 128, padding
    (64, 4, 4, 16, [600], 600, True),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "x".join(map(str, c)).replace(" ", ""))
def test_attend_fixed(case, dtype):
    D, Hq, Hkv, page, lens, t, causal = case
    c = Paged(lens, Hkv, D, page, seed=Hq + t)
    scale = 1.0 / np.sqrt(D)
    q, o, lse = attend_fixed(c, Hq, t, dtype, seed=t + D, scale=scale, causal=causal)
    check_attend(c, q, o, lse, scale, causal, dtype, f"{case}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D, Hq, Hkv, causal", [(128, 8, 2, True), (64, 4, 4, False), (256, 6, 2, True)])
def test_attend_packed(D, Hq, Hkv, causal, dtype):
    lens, counts = [40, 3, 64, 7, 129, 300, 0], [40, 1, 0, 9, 70, 1, 2]
    c = Paged(lens, Hkv, D, 16, seed=D + 3)
    sl = SeqLens(np.concatenate([[0], np.cumsum(counts)]), device=DEV)
    q = torch.randn(sl.total, Hq, D, generator=torch.Generator().manual_seed(D)).to(DT[dtype])
    o, lse = attn_fwd_kv4(q.to(DEV), c.cache, c.table_dev, c.lens_dev, causal=causal, seqlens=sl)
    torch.cuda.synchronize()
    assert get_status() == 0 and lse.shape == (Hq, sl.total)
    cut = lambda x: [x[a:b].transpose(0, 1).double().cpu().numpy() for a, b in zip(sl.host, sl.host[1:])]  # noqa: E731
    check_attend(c, cut(q), cut(o), [lse[:, a:b].double().cpu().numpy() for a, b in zip(sl.host, sl.host[1:])],
                 1.0 / np.sqrt(D), causal, dtype, f"packed {D} {Hq} {Hkv}")


@pytest.mark.parametrize("scale, spread", [(3.0, 1.0), (-0.2, 1.0), (0.0, 1.0), (0.1, 1e-20), (0.1, 1e18)])
def test_attend_extreme_scores(scale, spread):
    """Scores in the hundreds, of the other sign, all equal; queries far from 1."""
    c = Paged([200, 37], 2, 128, 16, seed=17)
    q = (torch.randn(2, 8, 1, 128, generator=torch.Generator().manual_seed(2)) * spread).to(torch.bfloat16)
    o, lse = attn_fwd_kv4(q.to(DEV), c.cache, c.table_dev, c.lens_dev, scale=scale / spread)
    torch.cuda.synchronize()
    check_attend(c, q.double().numpy(), o.double().cpu().numpy(), lse.double().cpu().numpy(), scale / spread, True,
                 "bf16", f"scale {scale} {spread}")


def test_attend_values_of_very_different_size():
    """A first position that takes nearly all the weight and holds tiny values, as a sink does."""
    c = Paged([3000], 1, 128, 16, seed=23)
    first = c.table[0, 0]
    c.scale[1][first, :, 0] *= 2.0 ** -20
    q = torch.randn(1, 4, 1, 128, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    u, s, b = kv4.quantise((q[0, 0, 0].float().numpy() * 3)[None])  # a key along the first query
    c.codes[0][first, :, 0] = kv4.pack(u)
    c.scale[0][first, :, 0, :, 0], c.scale[0][first, :, 0, :, 1] = s, b
    for t, x in ((c.cache.k_codes, c.codes[0]), (c.cache.k_scale, c.scale[0]), (c.cache.v_scale, c.scale[1])):
        t.copy_(torch.from_numpy(x).to(DEV).to(t.dtype))
    for scale in (1 / np.sqrt(128), 0.03):
        o, lse = attn_fwd_kv4(q.to(DEV), c.cache, c.table_dev, c.lens_dev, scale=scale)
        check_attend(c, q.double().numpy(), o.double().cpu().numpy(), lse.double().cpu().numpy(), scale, True, "bf16",
                     "sink")


@pytest.mark.parametrize("D, t, length", [(128, 1, 20000), (64, 4, 9000), (256, 1, 5000), (128, 9, 9000), (64, 7, 5001)])
def test_attend_long(D, t, length):
    """A key axis long enough to be split over many blocks; the same bits each time."""
    c = Paged([length, 1], 1, D, 64, seed=length)
    q, o, lse = attend_fixed(c, 4, t, "bf16", seed=1, scale=0.1)
    q, o2, lse2 = attend_fixed(c, 4, t, "bf16", seed=1, scale=0.1)
    assert np.array_equal(o, o2) and np.array_equal(lse, lse2)
    check_attend(c, q, o, lse, 0.1, True, "bf16", f"long {D} {length}")


def test_attend_many_sequences():
    """More sequences than a block has threads, most of them empty."""
    r = np.random.default_rng(6)
    lens = np.where(r.random(700) < 0.7, 0, r.integers(1, 40, 700)).tolist()
    c = Paged(lens, 1, 64, 16, seed=4)
    q, o, lse = attend_fixed(c, 2, 1, "bf16", seed=4, scale=0.125)
    check_attend(c, q, o, lse, 0.125, True, "bf16", "many")


def test_strided_views_and_unaligned_tensors():
    """q, k and v as slices of one projection's output, and tensors that start off a 16-byte boundary."""
    B, S, Hq, Hkv, D = 2, 3, 4, 2, 128
    c = Paged([50, 21], Hkv, D, 16, seed=9)
    qkv = torch.randn(B, S, (Hq + 2 * Hkv) * D, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    views = [x.unflatten(2, (-1, D)).transpose(1, 2) for x in qkv.to(DEV).split([Hq * D, Hkv * D, Hkv * D], 2)]
    kv4_write(c.cache, views[1], views[2], c.table_dev, c.lens_dev)
    host = [x.unflatten(2, (-1, D)).transpose(1, 2) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], 2)]
    c.codes, c.scale = expected_write(c, [(host[1][n], host[2][n]) for n in range(B)])
    same_cache(c, c.codes, c.scale)
    o, lse = attn_fwd_kv4(views[0], c.cache, c.table_dev, c.lens_dev)
    o_out = torch.empty(B, S, Hq, D, dtype=torch.bfloat16, device=DEV).transpose(1, 2)
    o2, _ = attn_fwd_kv4(views[0], c.cache, c.table_dev, c.lens_dev, out=o_out)
    flat = torch.zeros(views[0].numel() + 1, dtype=torch.bfloat16, device=DEV)[1:]
    off = flat.view(B, Hq, S, D).copy_(views[0])
    assert off.data_ptr() % 16
    o3, _ = attn_fwd_kv4(off, c.cache, c.table_dev, c.lens_dev)
    wide = torch.zeros(2, 9, dtype=torch.int32, device=DEV)
    wide[:, : c.table.shape[1]] = c.table_dev
    o4, _ = attn_fwd_kv4(views[0], c.cache, wide[:, : c.table.shape[1]], c.lens_dev)
    torch.cuda.synchronize()
    assert o2 is o_out and torch.equal(o, o2) and torch.equal(o, o3) and torch.equal(o, o4)
    check_attend(c, host[0].double().numpy(), o.double().cpu().numpy(), lse.double().cpu().numpy(), D ** -0.5, True,
                 "bf16", "views")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scale, spread", [(3.0, 1.0), (-0.2, 1.0), (0.0, 1.0), (0.1, 1e-20), (0.1, 1e18)])
def test_many_rows_extreme_scores(scale, spread, D):
    """The same with more than 24 rows on a KV head, padding among them."""
    c = Paged([200, 17], 2, D, 16, seed=18)
    q = (torch.randn(2, 8, 20, D, generator=torch.Generator().manual_seed(2)) * spread).to(torch.bfloat16)
    o, lse = attn_fwd_kv4(q.to(DEV), c.cache, c.table_dev, c.lens_dev, scale=scale / spread)
    torch.cuda.synchronize()
    check_attend(c, q.double().numpy(), o.double().cpu().numpy(), lse.double().cpu().numpy(), scale / spread, True,
                 "bf16", f"rows scale {scale} {spread}")


def test_many_rows_long_split_and_bit_identical():
    c = Paged([20000, 130], 1, 128, 64, seed=19)
    q, o, lse = attend_fixed(c, 8, 5, "bf16", seed=1, scale=0.1)
    q, o2, lse2 = attend_fixed(c, 8, 5, "bf16", seed=1, scale=0.1)
    assert np.array_equal(o, o2) and np.array_equal(lse, lse2)
    check_attend(c, q, o, lse, 0.1, True, "bf16", "rows long")


def test_many_rows_broken_queries_and_pages():
    """Infinities and NaN stay in their rows; a page that is none is left out and recorded."""
    c = Paged([150, 70], 2, 128, 16, seed=62)
    q = torch.randn(2, 8, 40, 128, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(DEV)
    o, lse = attn_fwd_kv4(q, c.cache, c.table_dev, c.lens_dev)
    broken = q.clone()
    broken[0, 1, 3, 5], broken[1, 6, 39, 0] = float("nan"), float("inf")
    o2, lse2 = attn_fwd_kv4(broken, c.cache, c.table_dev, c.lens_dev)
    hit = torch.zeros(2, 8, 40, dtype=torch.bool, device=DEV)
    hit[0, 1, 3] = hit[1, 6, 39] = True
    assert torch.equal(o[~hit], o2[~hit]) and torch.equal(lse[~hit], lse2[~hit])
    assert not torch.isfinite(o2[0, 1, 3]).any()
    bad = c.table_dev.clone()
    bad[0, 1], bad[1] = c.n_pages, -1
    o, lse = attn_fwd_kv4(q, c.cache, bad, c.lens_dev, causal=False)
    assert get_status() == _lib.ATTN_ERR_DEVICE_BOUNDS and get_status() == 0
    assert torch.all(o[1] == 0) and torch.all(torch.isneginf(lse[1]))
    keep = Paged([134, 0], 2, 128, 16, seed=62)  # the first sequence without its second page
    for which in range(2):
        for dst, src in ((keep.codes, c.codes), (keep.scale, c.scale)):
            for i, j in enumerate(j for j in range(10) if j != 1):
                dst[which][keep.table[0, i]] = src[which][c.table[0, j]]
    check_attend(keep, q.double().cpu().numpy(), o.double().cpu().numpy(), lse.double().cpu().numpy(), 128 ** -0.5,
                 False, "bf16", "rows bad pages")


# ---------------------------------------------------------------- as they are used


def test_prompt_then_tokens_then_resume():
    """A prompt through attn_fwd and kv4_write, some decoding steps, then the whole cache
    read back into attn_fwd: its last row is the last step's answer."""
    B, Hq, Hkv, D, page, prompt, steps = 2, 8, 2, 128, 16, 45, 4
    g = torch.Generator(device=DEV).manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    cache = Kv4Cache.empty(12, Hkv, page, D, device=DEV)
    table = torch.tensor([[7, 2, 9, 11], [0, 5, 3, 8]], dtype=torch.int32, device=DEV)
    lens = torch.full((B,), prompt, dtype=torch.int32, device=DEV)
    q, k, v = rand(B, Hq, prompt, D), rand(B, Hkv, prompt, D), rand(B, Hkv, prompt, D)
    kr, vr = k, v
    kv4_write(cache, k, v, table, lens)
    # over the prompt alone the cache's attention is the full one on the values read back
    kq, vq = kv4_read(cache, table, lens, prompt)
    o, lse = attn_fwd_kv4(q, cache, table, lens)
    o_ref, lse_ref = attn_fwd(q, kq, vq, causal=True)
    # both round P to bf16 (2^-8) and O (2^-8); keys and values read back are rounded to bf16 (2^-8)
    A = attn_fwd(q, kq, vq.abs(), causal=True)[0].float()
    assert torch.all((o.float() - o_ref.float()).abs() <= 2.0 ** -8 * (4 * A + o_ref.float().abs() * 2) + 0.1 * A)
    for _ in range(steps):
        lens += 1
        q, k, v = rand(B, Hq, 1, D), rand(B, Hkv, 1, D), rand(B, Hkv, 1, D)
        kr, vr = torch.cat([kr, k], 2), torch.cat([vr, v], 2)
        kv4_write(cache, k, v, table, lens)
        o, lse = attn_fwd_kv4(q, cache, table, lens)
    kq, vq = kv4_read(cache, table, lens, prompt + steps, dtype=torch.float32)
    kf, vf = (x.repeat_interleave(Hq // Hkv, 1).double() for x in (kq, vq))
    s = (q.double() @ kf.transpose(2, 3)) / D ** 0.5
    ref = torch.softmax(s, -1) @ vf
    A = torch.softmax(s, -1) @ vf.abs()
    torch.cuda.synchronize()
    assert get_status() == 0
    assert torch.all((o.double() - ref).abs() <= 2.0 ** -8 * (2.2 * A + ref.abs()) + 1e-5 * A)
    assert torch.all((lse.double() - torch.logsumexp(s, -1)).abs() < 1e-4)
    # what was written is what went in, to half a step of each group and b's rounding
    for x, y in ((kr, kq), (vr, vq)):
        grp = x.float().unflatten(-1, (-1, 64))
        step = (grp.amax(-1, True) - grp.amin(-1, True)) / 15
        bound = 0.5 * step * (1 + 2.0 ** -6) + 2.0 ** -8 * grp.abs().amax(-1, True) + 8 * 2.0 ** -8 * step
        assert torch.all((grp - y.unflatten(-1, (-1, 64))).abs() <= bound)


def test_captured_step_follows_new_lengths_and_pages():
    """A decoding step captured once; replayed with other lengths, page lists and inputs
    written into the same tensors.  A second graph of another shape shares nothing."""
    Hq, Hkv, D, page = 8, 2, 128, 16
    c = Paged([111, 47], Hkv, D, page, seed=31, spare=20)  # the next page begins at the second step
    q = torch.zeros(2, Hq, 1, D, dtype=torch.bfloat16, device=DEV)
    k, v = (torch.zeros(2, Hkv, 1, D, dtype=torch.bfloat16, device=DEV) for _ in "kv")
    q2 = torch.zeros(2, Hq, 3, D, dtype=torch.bfloat16, device=DEV)
    table = torch.zeros(2, 64, dtype=torch.int32, device=DEV)
    table[:, : c.table.shape[1]] = c.table_dev
    free = sorted(set(range(c.n_pages)) - set(c.table[0, :7]) - set(c.table[1, :3]))

    def step():
        kv4_write(c.cache, k, v, table, c.lens_dev)
        return attn_fwd_kv4(q, c.cache, table, c.lens_dev)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
        attn_fwd_kv4(q2, c.cache, table, c.lens_dev)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        out = step()
    with torch.cuda.graph(g2):
        out2 = attn_fwd_kv4(q2, c.cache, table, c.lens_dev)
    gen = torch.Generator(device=DEV).manual_seed(1)
    for rep in range(3):
        for t in (q, k, v, q2):
            t.copy_(torch.randn(t.shape, generator=gen, device=DEV))
        if rep:
            c.lens_dev += 1
            need = -(-c.lens_dev.cpu() // page)
            for n in range(2):
                have = 7 if n == 0 else 3
                for i in range(have, int(need[n])):
                    if table[n, i] == 0:
                        table[n, i] = free.pop()
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        got, got2 = [x.clone() for x in out], [x.clone() for x in out2]
        want = step()
        want2 = attn_fwd_kv4(q2, c.cache, table, c.lens_dev)
        for a, b in zip([*got, *got2], [*want, *want2]):
            assert torch.equal(a, b), rep
    torch.cuda.synchronize()
    assert get_status() == 0


def test_two_streams_at_once():
    a = Paged([5000, 300], 2, 128, 64, seed=41)
    b = Paged([900, 2500, 7], 2, 64, 16, seed=42)
    qa = torch.randn(2, 8, 1, 128, device=DEV).to(torch.bfloat16)
    qb = torch.randn(3, 4, 2, 64, device=DEV)
    runs = [(qa, a), (qb, b)]
    want = [attn_fwd_kv4(q, c.cache, c.table_dev, c.lens_dev) for q, c in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [attn_fwd_kv4(q, c.cache, c.table_dev, c.lens_dev, stream=s) for (q, c), s in zip(runs, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_many_rows_captured_and_on_two_streams():
    """Prompt chunks: a captured call follows new lengths, two graphs and two streams share nothing."""
    a, b = Paged([700, 90], 2, 128, 64, seed=43), Paged([260, 1000, 7], 1, 64, 16, seed=44)
    qa = torch.randn(2, 8, 30, 128, device=DEV).to(torch.bfloat16)
    qb = torch.randn(3, 4, 40, 64, device=DEV).to(torch.bfloat16)
    runs = [(qa, a), (qb, b)]
    call = lambda q, c, **kw: attn_fwd_kv4(q, c.cache, c.table_dev, c.lens_dev, **kw)  # noqa: E731
    want = [call(q, c) for q, c in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [call(q, c, stream=s) for (q, c), s in zip(runs, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    graphs, outs = [], []
    for q, c in runs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(call(q, c))
    for less in (0, 3):
        for _, c in runs:
            c.lens_dev -= less
        for g, s in zip(graphs, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (q, c), g in zip(runs, outs):
            w = call(q, c)
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    torch.cuda.synchronize()
    assert get_status() == 0


# ---------------------------------------------------------------- large caches, refusals


def test_offsets_beyond_32_bits():
    """Pages behind the first 8 GiB of a cache."""
    Hkv, D, page, n_pages = 8, 128, 256, 70000  # codes: 9.2 GB each for keys and values
    cache = Kv4Cache.empty(n_pages, Hkv, page, D, device=DEV)
    table = torch.tensor([[n_pages - 1, 3, n_pages - 2]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([600], dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(2)
    k, v = (torch.randn(1, Hkv, 600, D, generator=g, device=DEV) for _ in "kv")
    kv4_write(cache, k, v, table, lens)
    small = Kv4Cache.empty(3, Hkv, page, D, device=DEV)
    table3 = torch.tensor([[0, 1, 2]], dtype=torch.int32, device=DEV)
    kv4_write(small, k, v, table3, lens)
    q = torch.randn(1, 16, 1, D, generator=g, device=DEV).to(torch.bfloat16)
    for x, y in zip((*kv4_read(cache, table, lens, 600), *attn_fwd_kv4(q, cache, table, lens)),
                    (*kv4_read(small, table3, lens, 600), *attn_fwd_kv4(q, small, table3, lens))):
        assert torch.equal(x, y)
    torch.cuda.synchronize()
    assert get_status() == 0


def test_bad_pages_and_lengths_are_recorded_and_left_out():
    """A page list that names no page: a write skips it, a read gives zeros, the attention
    leaves its positions out; a length the list cannot hold is cut.  The status says so."""
    c = Paged([64, 40], 2, 128, 16, seed=51)
    before = [t.clone() for t in (c.cache.k_codes, c.cache.v_codes)]
    bad = c.table_dev.clone()
    bad[0, 1] = c.n_pages
    bad[0, 3] = -5
    q = torch.randn(2, 4, 1, 128, device=DEV).to(torch.bfloat16)
    o, lse = attn_fwd_kv4(q, c.cache, bad, c.lens_dev, causal=False)
    assert get_status() == _lib.ATTN_ERR_DEVICE_BOUNDS and get_status() == 0
    keep = Paged([32, 40], 2, 128, 16, seed=51)
    for n in range(2):
        for which in range(2):
            for dst, src in ((keep.codes, c.codes), (keep.scale, c.scale)):
                pages = [0, 2] if n == 0 else [0, 1, 2]
                for i, j in enumerate(pages):
                    dst[which][keep.table[n, i]] = src[which][c.table[n, j]]
    check_attend(keep, q.double().cpu().numpy(), o.double().cpu().numpy(), lse.double().cpu().numpy(), 128 ** -0.5,
                 False, "bf16", "bad pages")
    k, v = kv4_read(c.cache, bad, c.lens_dev, 64)
    assert get_status() == _lib.ATTN_ERR_DEVICE_BOUNDS
    assert torch.all(k[0, :, 16:32] == 0) and torch.all(v[0, :, 48:] == 0) and torch.any(k[0, :, 32:48] != 0)
    rows = torch.randn(2, 2, 16, 128, device=DEV)
    bad[1] = -1
    kv4_write(c.cache, rows, rows, bad, c.lens_dev)
    assert get_status() == _lib.ATTN_ERR_DEVICE_BOUNDS
    for a, b in zip(before, (c.cache.k_codes, c.cache.v_codes)):
        assert torch.equal(a, b)
    long = torch.tensor([c.table.shape[1] * 16 + 1, -3], dtype=torch.int32, device=DEV)
    o, lse = attn_fwd_kv4(q, c.cache, c.table_dev, long, causal=False)
    full = torch.tensor([c.table.shape[1] * 16, 0], dtype=torch.int32, device=DEV)
    assert get_status() == _lib.ATTN_ERR_DEVICE_BOUNDS
    o2, lse2 = attn_fwd_kv4(q, c.cache, c.table_dev, full, causal=False)
    assert get_status() == 0
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.all(o[1] == 0) and torch.all(torch.isneginf(lse[1]))


def test_infinite_and_nan_queries_stay_in_their_rows():
    c = Paged([50, 50], 2, 128, 16, seed=61)
    q = torch.randn(2, 8, 2, 128, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(DEV)
    o, lse = attn_fwd_kv4(q, c.cache, c.table_dev, c.lens_dev)
    broken = q.clone()
    broken[0, 1, 0, 5], broken[1, 6, 1, 0] = float("nan"), float("inf")
    o2, lse2 = attn_fwd_kv4(broken, c.cache, c.table_dev, c.lens_dev)
    hit = torch.zeros(2, 8, 2, dtype=torch.bool, device=DEV)
    hit[0, 1, 0] = hit[1, 6, 1] = True
    assert torch.equal(o[~hit], o2[~hit]) and torch.equal(lse[~hit], lse2[~hit])
    assert not torch.isfinite(o2[0, 1, 0]).any()


def test_refusals_of_the_binding():
    c = Paged([20, 30], 2, 128, 16, seed=71)
    q = torch.zeros(2, 8, 1, 128, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(2, 2, 1, 128, dtype=torch.bfloat16, device=DEV)
    call = lambda q=q, table=c.table_dev, lens=c.lens_dev, **kw: attn_fwd_kv4(q, c.cache, table, lens, **kw)  # noqa: E731
    for wrong in (lambda: call(q=q.half()), lambda: call(q=q.cpu()), lambda: call(q=q[..., :64]), lambda: call(q=q[:1]),
                  lambda: call(q=q[0]), lambda: call(table=c.table_dev.long()), lambda: call(lens=c.lens_dev.long()),
                  lambda: call(lens=c.lens_dev[:1]), lambda: call(table=c.table_dev.cpu()),
                  lambda: call(table=c.table_dev.t().contiguous().t()), lambda: call(out=q[:1]),
                  lambda: call(seqlens=SeqLens([0, 1, 2], device=DEV)),
                  lambda: kv4_write(c.cache, k, k.float(), c.table_dev, c.lens_dev),
                  lambda: kv4_write(c.cache, k[:, :1], k[:, :1], c.table_dev, c.lens_dev),
                  lambda: kv4_read(c.cache, c.table_dev, c.lens_dev),
                  lambda: kv4_read(c.cache, c.table_dev, c.lens_dev, 2, dtype=torch.float16),
                  lambda: kv4_read(c.cache, c.table_dev, c.lens_dev, 2, out=(k, k)),
                  lambda: Kv4Cache(c.cache.k_codes, c.cache.v_codes[:1], c.cache.k_scale, c.cache.v_scale),
                  lambda: Kv4Cache.empty(2, 2, 16, 96, device=DEV)):
        with pytest.raises((ValueError, _lib.AttnError)):
            wrong()
    for wrong in (lambda: call(q=torch.zeros(2, 7, 1, 128, dtype=torch.bfloat16, device=DEV)),
                  lambda: call(scale=float("inf")),
                  lambda: kv4_read(Kv4Cache.empty(2, 2, 24, 128, device=DEV), c.table_dev, c.lens_dev, 1)):
        with pytest.raises(_lib.AttnError):
            wrong()
    torch.cuda.synchronize()
    assert get_status() == 0
