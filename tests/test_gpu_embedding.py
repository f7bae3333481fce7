"""The embedding table on the GPU: lookup with scaling and the gradient by sorted tokens,
against the float64 oracle.

Tolerances, with u = 2^-24: the lookup is one float32 product (u) rounded to the type (finfo.eps / 2).
A word's gradient is a sum of float32 terms.  Up to 512 tokens: at most 128 one after the other, then four sums.
More: at most 64 one after the other in a piece of 16 or more, and then one partial sum for each piece that the word
reaches, an eighth of them one after the other where they are more than 17, and eight sums: at most
64 + 17 + tokens / 128 + 8 additions.  The scale and (with `out`) the old value are two
more operations: (140 + tokens / 32) u sum|terms| covers both, and eps / 2 of the result's type.
"""

import ctypes

import numpy as np
import pytest
import torch

from bwd_flashattention_fwd_sm_gb300 import _lib, embedding, embedding_bwd, get_status
from bwd_flashattention_fwd_sm_gb300._lib import EmbeddingParamsC
from oracle import rows as R

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24


def words(tokens, vocab, kind, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "uniform":
        return torch.randint(0, vocab, (tokens,), generator=g)
    if kind == "one":
        return torch.full((tokens,), vocab - 1)
    if kind == "each":  # every word once, then again
        return torch.arange(tokens) % vocab
    u = torch.rand(tokens, generator=g, dtype=torch.float64)  # a few words often
    return torch.randperm(vocab, generator=g)[(torch.exp(u * np.log(vocab + 1.0)).long() - 1).clamp(0, vocab - 1)]


def check_lookup(got, weight, ids, scale):
    ref = R.embedding(weight.double().cpu().numpy(), ids.cpu().numpy(), scale)
    tol = (torch.finfo(weight.dtype).eps / 2 + 2 * U) * np.abs(ref)
    assert got.shape == (*ids.shape, weight.shape[1])
    assert np.all(np.abs(got.double().cpu().numpy() - ref) <= tol)


def check_grad(got, dy, ids, vocab, scale, padding_id=None, old=None):
    ref, size = R.embedding_bwd(dy.double().cpu().numpy(), ids.cpu().numpy(), vocab, scale, padding_id)
    if old is not None:
        ref, size = ref + old.double().cpu().numpy(), size + np.abs(old.double().cpu().numpy())
    tol = (140 + ids.numel() / 32) * U * size + torch.finfo(got.dtype).eps / 2 * np.abs(ref)
    assert np.all(np.abs(got.double().cpu().numpy() - ref) <= tol)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 5, 7), (100, 10, 8), (64, 1000, 2), (33, 17, 130), (300, 70000, 64),
                                   (2000, 100, 513), (17, 300, 4096), (5, 9, 8200)], ids=str)
def test_lookup(shape, dtype):
    tokens, vocab, dim = shape
    g = torch.Generator().manual_seed(tokens)
    w = torch.randn(vocab, dim, generator=g).to(DTYPES[dtype]).cuda()
    ids = words(tokens, vocab, "uniform", 1).cuda()
    for i in (ids, ids.int()):
        check_lookup(embedding(w, i), w, i, 1.0)
        check_lookup(embedding(w, i, scale=-2.75), w, i, -2.75)


GRADS = [(1, 1, 1, "one"), (3, 5, 7, "uniform"), (31, 4, 8, "few"), (32, 4, 16, "one"), (33, 2, 24, "each"),
         (64, 1, 130, "one"), (100, 1000, 4, "few"), (1000, 10, 72, "uniform"), (1025, 511, 40, "few"),
         (2048, 512, 64, "each"), (2049, 3, 33, "uniform"), (5000, 70000, 16, "few"), (9000, 300000, 8, "uniform"),
         (9000, 1, 12, "one"), (20001, 60, 6, "few"), (300, 50, 4096, "few"), (70, 9, 8200, "one"),
         (40000, 2000, 32, "few"), (512, 300, 520, "few"), (512, 9000, 24, "one"), (513, 300, 520, "few"),
         (511, 100000, 10, "uniform")]


@pytest.mark.parametrize("dtype, grad", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("shape", GRADS, ids=str)
def test_gradient(shape, dtype, grad):
    tokens, vocab, dim, kind = shape
    g = torch.Generator().manual_seed(tokens)
    dy = torch.randn(tokens, dim, generator=g).to(DTYPES[dtype]).cuda()
    ids = words(tokens, vocab, kind, 2).cuda()
    got = embedding_bwd(dy, ids, vocab, scale=1.5, dtype=DTYPES[grad])
    assert got.dtype == DTYPES[grad] and got.shape == (vocab, dim)
    check_grad(got, dy, ids, vocab, 1.5)
    pad = int(ids[0])
    got = embedding_bwd(dy, ids.int(), vocab, padding_id=pad, dtype=DTYPES[grad])
    check_grad(got, dy, ids, vocab, 1.0, pad)
    assert not got[pad].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 131])
@pytest.mark.parametrize("tokens", [300, 700])
def test_gradient_added_to_another(tokens, dim, dtype):
    g = torch.Generator().manual_seed(3)
    dy = torch.randn(tokens, dim, generator=g).to(DTYPES[dtype]).cuda()
    ids = words(tokens, 400, "few", 4).cuda()
    old = torch.randn(400, dim, generator=g).to(DTYPES[dtype]).cuda()
    out = old.clone()
    assert embedding_bwd(dy, ids, 400, scale=0.5, padding_id=int(ids[5]), out=out) is out
    check_grad(out, dy, ids, 400, 0.5, int(ids[5]), old)
    named = torch.zeros(400, dtype=torch.bool, device="cuda")
    named[ids] = True
    named[ids[5]] = False
    assert torch.equal(out[~named], old[~named])  # rows that no token names, bit for bit
    wide = torch.full((400, dim + 16), 7.0, dtype=DTYPES[dtype], device="cuda")
    wide[:, :dim] = old
    embedding_bwd(dy, ids, 400, scale=0.5, padding_id=int(ids[5]), out=wide[:, :dim])
    assert torch.equal(wide[:, :dim], out) and bool((wide[:, dim:] == 7).all())
    with pytest.raises(ValueError, match="out"):
        embedding_bwd(dy, ids, 400, out=torch.empty(dim, 400, dtype=DTYPES[dtype], device="cuda").t())
    with pytest.raises(ValueError, match="dtype"):
        embedding_bwd(dy, ids, 400, out=out, dtype=torch.float16)


@pytest.mark.parametrize("dtype, dim", [("bf16", 1000), ("f32", 777)])
@pytest.mark.parametrize("tokens, kind", [(600, "few"), (3000, "uniform"), (9000, "few")])
def test_gradient_of_a_large_table(tokens, kind, dtype, dim):
    """Tables whose zeros take longer than the sort, over memory that holds NaN;
    float64 sums on the GPU."""
    vocab, dt = 150000, DTYPES[dtype]
    g = torch.Generator().manual_seed(tokens)
    dy = torch.randn(tokens, dim, generator=g).to(dt).cuda()
    ids = words(tokens, vocab, kind, 3).cuda()
    ids[:4] = torch.tensor([0, vocab - 1, vocab - 1, 0], device="cuda")
    del_me = torch.full((vocab, dim), float("nan"), dtype=dt, device="cuda")
    at = del_me.data_ptr()
    del del_me
    got = embedding_bwd(dy, ids, vocab, scale=0.5)
    assert got.data_ptr() == at  # the same memory: every row has been written
    ref = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda").index_add_(0, ids, 0.5 * dy.double())
    size = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda").index_add_(0, ids, 0.5 * dy.double().abs())
    tol = (140 + tokens / 32) * U * size + torch.finfo(dt).eps / 2 * ref.abs()
    assert bool(((got.double() - ref).abs() <= tol).all())


def test_ids_outside_the_table():
    """They give rows of zeros and no gradient, and are recorded; everything else is as without them."""
    g = torch.Generator().manual_seed(5)
    w, dy = torch.randn(50, 24, generator=g).cuda(), torch.randn(900, 24, generator=g).cuda()
    for dtype, bad, n in ((torch.int64, [-1, 50, 2 ** 40, -2 ** 63], 200), (torch.int32, [-1, 50, 2 ** 31 - 1, -2 ** 31], 200),
                          (torch.int64, [-1, 50, 2 ** 40, -2 ** 63], 900)):
        ids = torch.randint(0, 50, (n,), generator=g).to(dtype)
        ids[torch.tensor([0, 63, 64, n - 1])] = torch.tensor(bad, dtype=dtype)
        ids = ids.cuda()
        assert get_status() == 0
        check_lookup(embedding(w, ids), w, ids, 1.0)
        assert get_status() == _lib.ATTN_ERR_DEVICE_BOUNDS
        check_grad(embedding_bwd(dy[:n], ids, 50), dy[:n], ids, 50, 1.0)
        assert get_status() == _lib.ATTN_ERR_DEVICE_BOUNDS
    for n in (100, 900):
        every = torch.full((n,), 77, device="cuda")
        assert not embedding(w, every).any() and not embedding_bwd(dy[:n], every, 50).any()
    assert get_status() == _lib.ATTN_ERR_DEVICE_BOUNDS and get_status() == 0


def test_empty():
    w = torch.ones(5, 8, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert embedding(w, none).shape == (0, 8)
    assert not embedding_bwd(torch.empty(0, 8, device="cuda"), none, 5).any()
    out = w.clone()
    assert torch.equal(embedding_bwd(torch.empty(0, 8, device="cuda"), none, 5, out=out), w)
    assert embedding(torch.empty(5, 0, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")).shape == (3, 0)
    assert embedding_bwd(torch.empty(3, 0, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda"), 5).shape == (5, 0)


@pytest.mark.parametrize("tokens", [100, 1000])
def test_nan_stays_with_its_word(tokens):
    dy = torch.ones(tokens, 16, device="cuda")
    ids = torch.arange(tokens, device="cuda") % 10
    dy[13] = float("nan")
    got = embedding_bwd(dy, ids, 12)
    assert torch.isnan(got[3]).all()
    got[3] = 0
    assert torch.isfinite(got).all()
    got = embedding_bwd(dy, ids, 12, padding_id=3)  # a padding row's NaN goes nowhere
    assert torch.isfinite(got).all() and not got[3].any()


def test_same_bits_every_time_and_on_any_workspace():
    g = torch.Generator().manual_seed(6)
    dy = torch.randn(30000, 40, generator=g).cuda()
    ids = words(30000, 5000, "few", 7).cuda()
    a = embedding_bwd(dy, ids, 5000)
    ws = torch.full((1 << 25,), 0xFF, dtype=torch.uint8, device="cuda")
    for kw in ({}, {"workspace": ws}, {"workspace": ws}):
        assert torch.equal(a, embedding_bwd(dy, ids, 5000, **kw))


def test_views():
    g = torch.Generator().manual_seed(8)
    w, dy = torch.randn(30, 96, generator=g).cuda(), torch.randn(4, 25, 96, generator=g).cuda()
    ids = torch.randint(0, 30, (4, 25), generator=g).cuda()
    for cols in (slice(0, 64), slice(32, 96), slice(1, 60)):
        check_lookup(embedding(w[:, cols], ids), w[:, cols], ids, 1.0)
        check_grad(embedding_bwd(dy[..., cols], ids, 30), dy[..., cols], ids, 30, 1.0)
    check_lookup(embedding(w.t().contiguous().t(), ids.t()), w, ids.t(), 1.0)
    check_grad(embedding_bwd(dy.transpose(0, 1), ids.t(), 30), dy.transpose(0, 1), ids.t(), 30, 1.0)


def test_c_entry_writes_nothing_behind_its_buffers():
    """A table with gaps between its rows and a pattern around it, a workspace of exactly the size asked for."""
    lib = _lib.load()
    for tokens, vocab, dim, step in ((1000, 300, 40, 48), (77, 300, 41, 45), (4097, 7, 256, 256)):
        g = torch.Generator().manual_seed(tokens)
        dy = torch.randn(tokens, dim, generator=g).cuda()
        ids = words(tokens, vocab, "few", 9).cuda()
        buf = torch.full((vocab * step + 64,), 7.0, device="cuda")
        table = buf[32:32 + vocab * step].view(vocab, step)
        p = EmbeddingParamsC(tokens, vocab, dim, dim, step, 1.0, _lib.ATTN_F32, _lib.ATTN_F32, 1, 0, -1)
        need = lib.attn_embedding_bwd_workspace_size(p)
        ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
        code = lib.attn_embedding_bwd(p, dy.data_ptr(), ids.data_ptr(), table.data_ptr(), ws.data_ptr(), need,
                                      ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert code == 0
        torch.cuda.synchronize()
        assert bool((ws[need:] == 0x5A).all())
        assert bool((buf[:32] == 7).all()) and bool((buf[32 + vocab * step:] == 7).all())
        assert bool((table[:, dim:] == 7).all())
        check_grad(table[:, :dim], dy, ids, vocab, 1.0)


def test_a_table_beyond_31_bits():
    """Rows at offsets that pass 2^31 elements, and 2^32 bytes of gradient."""
    vocab, dim = (1 << 31) // 4096 + 9, 4096
    w = torch.zeros(vocab, dim, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([vocab - 1, 0, vocab - 2, vocab - 1], device="cuda")
    w[ids] = torch.randn(4, dim, device="cuda").to(torch.bfloat16)
    assert torch.equal(embedding(w, ids), w[ids])
    dy = torch.randn(4, dim, device="cuda").to(torch.bfloat16)
    w.fill_(1)
    got = embedding_bwd(dy, ids, vocab)
    assert torch.equal(got[0], dy[1]) and torch.equal(got[vocab - 2], dy[2])
    assert torch.equal(got[vocab - 1], (dy[0].float() + dy[3].float()).to(torch.bfloat16))
    assert int(got.any(1).sum()) == 3
    del got
    # the same by sorting
    dy = torch.randn(600, dim, device="cuda").to(torch.bfloat16)
    dy[4:] = 0
    got = embedding_bwd(dy, torch.cat([ids, ids.repeat(149)]), vocab)
    assert torch.equal(got[0], dy[1]) and torch.equal(got[vocab - 2], dy[2])
    assert torch.equal(got[vocab - 1], (dy[0].float() + dy[3].float()).to(torch.bfloat16))
    assert int(got.any(1).sum()) == 3


def test_streams_and_graphs():
    """Two gradients at once on two streams; a captured call follows new ids and values."""
    g = torch.Generator().manual_seed(10)
    jobs = []
    for tokens, vocab, dim in ((20000, 3000, 256), (9000, 20000, 128)):
        jobs.append((torch.randn(tokens, dim, generator=g).cuda(), words(tokens, vocab, "few", tokens).cuda(), vocab))
    ref = [embedding_bwd(*j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(3):
        got = [embedding_bwd(*j, stream=s) for j, s in zip(jobs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    dy, ids, vocab = (t.clone() if torch.is_tensor(t) else t for t in jobs[0])
    w = torch.randn(vocab, 256, generator=g).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, dw = embedding(w, ids), embedding_bwd(dy, ids, vocab)
    for shift in (0, 1):
        ids.copy_((jobs[0][1] + shift) % vocab)
        graph.replay()
        assert torch.equal(y, w[ids])
        assert torch.equal(dw, embedding_bwd(dy, ids, vocab))
    assert get_status() == 0


def test_refuses_a_padding_token_below_zero():
    """It would name no token, nor the table's last row."""
    dy, ids = torch.ones(3, 8, device="cuda"), torch.tensor([0, 3, 1], device="cuda")
    for pad in (-1, -100):
        with pytest.raises(ValueError, match="padding_id"):
            embedding_bwd(dy, ids, 4, padding_id=pad)
    check_grad(embedding_bwd(dy, ids, 4, padding_id=3), dy, ids, 4, 1.0, 3)
