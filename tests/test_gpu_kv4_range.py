"""GPU tests of the attention over the 4-bit cache where positions' values differ in size by many
powers of two, and of float32 rows over long contexts, against the oracle.

Up to 24 bfloat16 query rows on a KV head, or float32 (csrc/kv4_attn.cu): the weights w = p s of a row and group are
float16 (float32: float16 parts) in units in which W, the largest of them, is 2^4 at least.  bfloat16:
off by 2^-11 w, below float16's normal range by half its least step, 2^-25 units <= 2^-29 W; times |u - 8| <= 8
over n positions 2^-11 R + n 2^-26 W.  float32: off by 2^-24 w (the product's rounding), and by 2^-37
units <= 2^-41 W: n 2^-38 W.  All of it is relative to the row's own weights, whatever
the largest step of the head is.  Scores, exp2, sums and O's rounding as in test_gpu_kv4.py.

For float32 rows those bounds add up worst cases and lie far above the errors, so their errors are
held to float32 arithmetic's as well: the root mean square over a head's O (its LSE) is at most four times what
the same formulas in float32 (products and sums of torch on the same device, exp) give, plus one rounding of the
largest: exp2's approximation is off by four half steps where exp is off by one.  An LSE is one number, whose
roundings may cancel in one form and add up in the other: it is (m + log2 l) ln 2 in float32, where the largest score
m in units of ln 2 is a rounded product, and the sum, ln 2 and the product are rounded: 4 half steps.
"""

import numpy as np
import pytest
import torch

from bwd_flashattention_fwd_sm_gb300 import attn_fwd_kv4, get_status
from oracle import kv4

from test_gpu_kv4 import DEV, DT, EPS, Paged

pytestmark = pytest.mark.gpu


def upload(c):
    for t, x in ((c.cache.k_codes, c.codes[0]), (c.cache.v_codes, c.codes[1]), (c.cache.k_scale, c.scale[0]),
                 (c.cache.v_scale, c.scale[1])):
        t.copy_(torch.from_numpy(x).to(DEV).to(t.dtype))


def scale_values(c, n, exps):
    """Values of position j of sequence n times 2^exps[j]."""
    for j, e in enumerate(exps):
        c.scale[1][c.table[n, j // c.page], :, j % c.page] *= np.float32(2.0 ** int(e))


def set_keys(c, n, j, rows):
    """Keys of position j: rows [Hkv, D]."""
    u, s, b = kv4.quantise(rows.astype(np.float32))
    at = c.table[n, j // c.page]
    c.codes[0][at, :, j % c.page] = kv4.pack(u)
    c.scale[0][at, :, j % c.page, :, 0], c.scale[0][at, :, j % c.page, :, 1] = s, b


def float32_form(c, n, q, scale):
    """O and LSE of the last rows of sequence n, causal, in float32 on the device."""
    k, v = (torch.from_numpy(sum(kv4.parts(*c.rows(n, w))).astype(np.float32)).to(DEV) for w in (0, 1))
    group, t, length = q.shape[0] // c.Hkv, q.shape[1], c.lens[n]
    k, v = k.repeat_interleave(group, 0), v.repeat_interleave(group, 0)
    tf32, torch.backends.cuda.matmul.allow_tf32 = torch.backends.cuda.matmul.allow_tf32, False
    s = (q.to(DEV) @ k.transpose(1, 2)) * scale
    late = torch.arange(length, device=DEV)[None] > length - t + torch.arange(t, device=DEV)[:, None]
    s = s.masked_fill(late, -np.inf)
    m = s.amax(-1, True)
    p = torch.exp(s - m)
    total = p.sum(-1, True)
    o, lse = (p @ v) / total, (torch.log(total) + m)[..., 0]
    torch.backends.cuda.matmul.allow_tf32 = tf32
    return o.double().cpu().numpy(), lse.double().cpu().numpy()


def check(c, Hq, t, dtype, scale, seed, q=None, sharp=None):
    """One call, causal.  sharp: the bound has to be below that part of the largest |O| of each row."""
    if q is None:
        q = torch.randn(len(c.lens), Hq, t, c.D, generator=torch.Generator().manual_seed(seed))
    q = q.to(DT[dtype])
    o, lse = attn_fwd_kv4(q.to(DEV), c.cache, c.table_dev, c.lens_dev, scale=scale)
    assert get_status() == 0
    o, lse, qd = o.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().numpy()
    group = Hq // c.Hkv
    for n, length in enumerate(c.lens):
        ku, vu = c.rows(n, 0), c.rows(n, 1)
        kp, vp = kv4.parts(*ku), kv4.parts(*vu)
        ro, rl, A, R, W = kv4.attend(qd[n], kp, vp, ku[1], scale, True)
        d = (c.D + 16) * EPS * W + length * EPS + 2.0 ** -21
        largest = np.zeros((Hq, t, c.D))  # of a row's p s in each group
        for h in range(Hq):
            x = scale * (qd[n, h] @ (kp[0] + kp[1])[h // group].T)
            x[np.arange(length)[None] > length - t + np.arange(t)[:, None]] = -np.inf
            p = np.exp(x - rl[h][:, None])
            largest[h] = np.repeat((p[:, :, None] * vu[1][h // group][None]).max(1), 64, -1)
        if dtype == "bf16":
            tol = 2 * d[..., None] * A + 2.0 ** -11 * R + length * 2.0 ** -26 * largest + 2.0 ** -8 * np.abs(ro) * (1 + 2.0 ** -8)
        else:
            tol = 2 * d[..., None] * A + 2 * EPS * (R + np.abs(ro)) + length * 2.0 ** -38 * largest
        err, lerr = np.abs(o[n] - ro), np.abs(lse[n] - rl)
        print(f"O {np.max(err / tol):.3f} of the bound, bound {np.max(np.median(tol, -1) / np.abs(ro).max(-1)):.1e} of O")
        assert np.all(err <= tol), f"sequence {n}: {np.max(err / tol):.3f}"
        assert np.all(lerr <= d + 4 * EPS * np.abs(rl)), f"sequence {n}: LSE"
        if sharp is not None:
            assert np.all(np.median(tol, -1) < sharp * np.abs(ro).max(-1))
        if dtype == "f32":
            fo, fl = float32_form(c, n, q[n], scale)
            rms = lambda x, axis: np.sqrt(np.mean(x * x, axis))  # noqa: E731
            for got, plain, size, half in ((rms(err, (1, 2)), rms(fo - ro, (1, 2)), np.abs(ro).max((1, 2)), 1),
                                           (rms(lerr, 1), rms(fl - rl, 1), np.abs(rl).max(1), 4)):
                print(f"  {np.max(got / size):.2e} of the largest, float32 form {np.max(plain / size):.2e}")
                assert np.all(got <= 4 * plain + half * EPS * size), (got, plain, size)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D, Hq, t", [(64, 4, 1), (128, 4, 3), (128, 16, 1), (64, 24, 1), (256, 4, 1), (256, 4, 3)])
@pytest.mark.parametrize("small", [6, 12, 20, 28])
def test_weight_on_a_position_with_small_values(small, D, Hq, t, dtype):
    """One position takes all the weight but 2^-40 and its values are 2^small times smaller than the others':
    the first position, one in the middle, or a late one, which lowers what all before it weigh."""
    lens = [1500, 700, 900]
    c = Paged(lens, 1, D, 16, seed=small + D)
    g = torch.Generator().manual_seed(small)
    q = torch.randn(3, 1, 1, D, generator=g) + 0.2 * torch.randn(3, Hq, t, D, generator=g)
    for n, at in enumerate((0, 333, 890)):
        scale_values(c, n, np.where(np.arange(lens[n]) == at, -small, 0))
        along = q[n, 0, 0].numpy()
        set_keys(c, n, at, (along * 45 / (along @ along) * np.sqrt(D))[None])  # a score of about 45
    upload(c)
    check(c, Hq, t, dtype, 1.0 / np.sqrt(D), 0, q=q, sharp=2.0 ** -4)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D, Hq, t", [(64, 4, 1), (128, 20, 1), (256, 8, 2)])
def test_a_late_score_that_leaves_nothing_of_the_others(D, Hq, t, dtype):
    """A score of about 150 behind others of a few: they weigh 2^-200, less than float32 holds, and the position's
    values are 2^25 times smaller than theirs."""
    c = Paged([800], 1, D, 16, seed=D + 1)
    g = torch.Generator().manual_seed(D)
    q = torch.randn(1, 1, 1, D, generator=g) + 0.05 * torch.randn(1, Hq, t, D, generator=g)
    scale_values(c, 0, np.where(np.arange(800) == 700, -25, 0))
    along = q[0, 0, 0].numpy()
    set_keys(c, 0, 700, (along * 150 / (along @ along) * np.sqrt(D))[None])
    upload(c)
    check(c, Hq, t, dtype, 1.0 / np.sqrt(D), 0, q=q, sharp=2.0 ** -4)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D, Hq, t", [(64, 2, 1), (128, 8, 2), (128, 6, 4), (256, 2, 5)])
def test_values_that_grow_fall_and_jump(D, Hq, t, dtype):
    """Sizes over 2^-30 .. 2^30: rising with the position, falling, at random, and one that is far
    above all others but has no weight to speak of."""
    lens = [1100, 1100, 1100, 600]
    c = Paged(lens, 1, D, 32, seed=D)
    r = np.random.default_rng(3)
    for n, exps in enumerate((np.arange(1100) // 18 - 30, 30 - np.arange(1100) // 18, r.integers(-30, 31, 1100),
                              np.where(np.arange(600) == 300, 50, 0))):
        scale_values(c, n, exps)
    set_keys(c, 3, 300, np.zeros((1, D)))
    upload(c)
    check(c, Hq, t, dtype, 1.0 / np.sqrt(D), D)


@pytest.mark.parametrize("D, Hq, t, length", [(64, 1, 1, 30000), (64, 2, 5, 21000), (128, 2, 1, 21000), (256, 1, 1, 20011)])
def test_float32_rows_over_a_long_context(D, Hq, t, length):
    c = Paged([length], 1, D, 64, seed=length)
    check(c, Hq, t, "f32", 1.0 / np.sqrt(D), 3)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("scale, spread", [(1.0, 1.0), (-0.2, 1.0), (0.0, 1.0), (0.1, 1e-20), (0.1, 1e18)])
def test_float32_extreme_scores(scale, spread, D):
    """Scores in the hundreds, of the other sign, all equal; queries far from 1."""
    c = Paged([300, 137], 2, D, 16, seed=27)
    q = torch.randn(2, 4, 2, D, generator=torch.Generator().manual_seed(2)) * spread
    check(c, 4, 2, "f32", scale / spread, 0, q=q)
