"""Row operators of a training step: dropout, residual add and LayerNorm with their
gradients, and the embedding table with its gradient.

Dropout.  The mask of a [rows, cols] tensor (leading axes taken together) is never
stored; it follows from a seed, an offset and an element's place.  Philox4x32 with 7
rounds (Salmon, Moraes, Dror, Shaw: Parallel random numbers: as easy as 1, 2, 3; 2011)
with the key (seed low, seed high) and the counter (col / 8, row, offset low, offset
high) gives four 32-bit words; element col has the 16 bits number col % 8 of them,
lowest first.  With t = round(65536 p) an element whose 16 bits are below t becomes 0
(whatever it held), another is multiplied by 65536 / (65536 - t).  seed and offset are
the sums, modulo 2^64, of numbers of the call and of a pair `rng` on the device.

LayerNorm.  h = D(x) + r with D the dropout, and per row
    mean = sum(h) / cols,  rstd = 1 / sqrt(sum((h - mean)^2) / cols + eps),
    y = (h - mean) rstd gamma + beta.
Its backward pass takes dy, the stored h, mean and rstd and, where h also goes on as
the residual stream, the gradient dh that arrives there.  With xh = (h - mean) rstd
and g = dy gamma,
    dr = dh + rstd (g - sum(g) / cols - xh sum(g xh) / cols),   dx = D(dr),
    dgamma = sum over rows of dy xh,   dbeta = sum over rows of dy.
Without dropout dx and dr are one.

Embedding.  y_i = s W[id_i].  The gradient is dW[v] = s times the sum of dy_i over the
places i with id_i = v; rows of W that no place names get 0, and so does the row of
the padding token.
"""

import math

import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _rows(name, op, dtype, rows, cols, p, stream):
    """op: "ln_fwd", "ln_bwd", "dropout" over [rows, cols]; p: dropout's probability;
    stream: x is added to a residual (ln_fwd), a gradient dh arrives at h (ln_bwd)."""
    return {"name": name, "op": op, "dtype": dtype, "rows": rows, "cols": cols, "p": p, "stream": stream}


def _table(name, op, dtype, tokens, vocab, dim, pad, ids, grad="same"):
    """op: "embed", "embed_bwd"; pad: share of the places that hold the padding token;
    ids: the places' type; grad: the type of dW, dy's own or "f32"."""
    return {"name": name, "op": op, "dtype": dtype, "tokens": tokens, "vocab": vocab, "dim": dim, "pad": pad,
            "ids": ids, "grad": grad}


def listed():
    return [
        # two sequences of 8192 tokens through one sublayer's dropout, add and norm
        _rows("ln_fwd_stream", "ln_fwd", "bf16", 16384, 4096, 0.1, True),
        # float32, rows that are no whole vectors, a high rate
        _rows("ln_fwd_f32_odd", "ln_fwd", "f32", 777, 2049, 0.25, True),
        # a short sequence of a small model: latency
        _rows("ln_bwd_short", "ln_bwd", "bf16", 128, 1024, 0.1, True),
        # the backward pass of ln_fwd_stream
        _rows("ln_bwd_stream", "ln_bwd", "bf16", 16384, 4096, 0.1, True),
        # a norm before the products, without dropout; the widest rows
        _rows("ln_bwd_wide", "ln_bwd", "bf16", 2047, 16384, 0.0, True),
        # many narrow rows (a norm of heads), float32
        _rows("ln_bwd_f32_narrow", "ln_bwd", "f32", 100003, 128, 0.0, False),
        # dropout of an inner layer's activations
        _rows("dropout_inner", "dropout", "bf16", 16384, 8192, 0.1, False),
        # float32, odd sizes
        _rows("dropout_f32_odd", "dropout", "f32", 1501, 1003, 0.5, False),
        # the tokens of a batch of prompts
        _table("embed_batch", "embed", "bf16", 16384, 50000, 4096, 0.1, "i64"),
        # one decoding step of a serving batch: latency
        _table("embed_step", "embed", "f32", 64, 32000, 2048, 0.0, "i32"),
        # the table's gradient after a batch: few words come often, most of the table not at all
        _table("embed_bwd_batch", "embed_bwd", "bf16", 16384, 50000, 4096, 0.1, "i64"),
        # many tokens on a small table, half of them padding, float32
        _table("embed_bwd_f32_small", "embed_bwd", "f32", 40001, 1000, 513, 0.5, "i32"),
    ]


def draw(rng):
    def log_int(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))

    op = rng.choice(["ln_fwd", "ln_bwd", "ln_bwd", "ln_bwd", "dropout", "embed", "embed_bwd", "embed_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])

    def width(lo, hi):
        n = log_int(lo, hi)
        return n if rng.random() < 0.5 else max(8, n // 64 * 64)

    if op in ("ln_fwd", "ln_bwd", "dropout"):
        cols = width(1 if op == "dropout" else 16, 16384)
        rows = log_int(1, max(1, (1 << 25) // cols))
        c = _rows("", op, dtype, rows, cols, rng.choice([0.0, 0.1, 0.1, 0.25, 0.5]), rng.random() < 0.7)
        if op == "dropout":
            c["p"], c["stream"] = c["p"] or 0.3, False
    else:
        dim = width(1, 8192)
        tokens = log_int(1, min(65536, (1 << 25) // dim))
        vocab = log_int(2, min(262144, (1 << 26) // dim))
        c = _table("", op, dtype, tokens, vocab, dim, rng.choice([0.0, 0.1, 0.5]), rng.choice(["i64", "i32"]),
                   rng.choice(["same", "f32"]) if op == "embed_bwd" else "same")
    del c["name"]
    return c


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------


class State:
    pass


PADDING = 1  # the padding token of a table


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    c, st = case, State()
    dtype = DTYPES[c["dtype"]]
    st.case, st.dtype = c, dtype

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if c["op"] in ("embed", "embed_bwd"):
        N, V, dim = c["tokens"], c["vocab"], c["dim"]
        st.scale = math.sqrt(dim)
        # the k-th most frequent word with a share near 1 / k, words in any order in the table
        u = torch.rand(N, generator=g, device=dev, dtype=torch.float64)
        rank = torch.exp(u * math.log(V + 1.0)).long().sub(1).clamp(0, V - 1)
        ids = torch.randperm(V, generator=g, device=dev)[rank]
        padded = torch.arange(N, device=dev) % 1024 >= 1024 - int(1024 * c["pad"])  # the ends of sequences
        ids = torch.where(padded, torch.full_like(ids, PADDING), ids)
        st.ids = ids.to(torch.int64 if c["ids"] == "i64" else torch.int32)
        if c["op"] == "embed":
            st.weight = (normal(V, dim) / math.sqrt(dim)).to(dtype)
        else:
            st.dy = (normal(N, dim) * 1e-2).to(dtype)
            st.grad = dtype if c["grad"] == "same" else DTYPES[c["grad"]]
            st.padding = PADDING if c["pad"] > 0 else None
        return st

    rows, cols = c["rows"], c["cols"]
    # the pair on the device that a training loop advances, and the number of this layer
    st.rng = torch.randint(-(2 ** 63), 2 ** 63 - 1, (2,), generator=g, device=dev)
    st.layer = 7
    if c["op"] == "dropout":
        st.x = normal(rows, cols).to(dtype)
        return st
    st.gamma, st.beta = 1.0 + 0.5 * normal(cols), 0.1 * normal(cols)
    if c["op"] == "ln_fwd":
        st.x = normal(rows, cols).to(dtype)
        st.r = (2.0 * normal(rows, cols) + 0.5).to(dtype) if c["stream"] else None
        return st
    # a few channels of the residual stream are much larger than the others, as in trained models
    st.h = ((2.0 * normal(rows, cols) + 0.5) * (1.0 + 9.0 * (torch.rand(cols, generator=g, device=dev) < 0.01))).to(dtype)
    h = st.h.double()
    mean = h.mean(1)
    st.mean = mean.float()
    st.rstd = (1.0 / torch.sqrt((h - mean[:, None]).square().mean(1) + EPS)).float()
    st.dy = (1e-2 * normal(rows, cols)).to(dtype)
    st.dh = (1e-2 * normal(rows, cols)).to(dtype) if c["stream"] else None
    return st


# ----------------------------------------------------------------------------
# The operators
# ----------------------------------------------------------------------------

LOW = 0xFFFFFFFF


def _product(a, b):
    """High and low 32 bits of a number a times a tensor b of numbers below 2^32, without passing 63 bits."""
    low, high = a * (b & 0xFFFF), a * (b >> 16)
    return (high + (low >> 16)) >> 16, (((high & 0xFFFF) << 16) + low) & LOW


def _kept(st):
    """The mask, and the factor of the elements that stay."""
    c, dev = st.case, st.rng.device
    rows, cols = c["rows"], c["cols"]
    t = round(65536 * c["p"])
    groups = -(-cols // 8)
    offset = st.rng[1] + st.layer
    k0, k1 = st.rng[0] & LOW, (st.rng[0] >> 32) & LOW
    c0 = torch.arange(groups, device=dev)[None, :].expand(rows, groups)
    c1 = torch.arange(rows, device=dev)[:, None].expand(rows, groups)
    c2, c3 = (offset & LOW).expand(rows, groups), ((offset >> 32) & LOW).expand(rows, groups)
    for _ in range(7):
        h0, l0 = _product(0xD2511F53, c0)
        h1, l1 = _product(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & LOW, (k1 + 0xBB67AE85) & LOW
    words = torch.stack([c0, c1, c2, c3], -1)
    u = torch.stack([words & 0xFFFF, words >> 16], -1).flatten(1)[:, :cols]
    return u >= t, 65536.0 / (65536 - t) if t < 65536 else 0.0


def _dropped(st, x):
    if st.case["p"] == 0.0:
        return x
    keep, factor = _kept(st)
    return torch.where(keep, x * factor, 0.0)


def run(state):
    st, c = state, state.case
    if own:
        import bwd_flashattention_fwd_sm_gb300 as G

        if c["op"] == "embed":
            return G.embedding(st.weight, st.ids, scale=st.scale)
        if c["op"] == "embed_bwd":
            return G.embedding_bwd(st.dy, st.ids, c["vocab"], scale=st.scale, padding_id=st.padding, dtype=st.grad)
        if c["op"] == "dropout":
            return G.dropout(st.x, c["p"], offset=st.layer, rng=st.rng)
        if c["op"] == "ln_fwd":
            return G.layernorm_residual(st.x, st.r, st.gamma, st.beta, eps=EPS, return_stats=True, dropout_p=c["p"],
                                        offset=st.layer, rng=st.rng)
        return G.layernorm_residual_bwd(st.dy, st.h, st.mean, st.rstd, st.gamma, st.dh, dropout_p=c["p"],
                                        offset=st.layer, rng=st.rng)
    if c["op"] == "embed":
        return (st.weight[st.ids].float() * st.scale).to(st.dtype)
    if c["op"] == "embed_bwd":
        dy = st.dy.float()
        if st.padding is not None:
            dy = dy.masked_fill((st.ids == st.padding)[:, None], 0.0)
        dw = torch.zeros(c["vocab"], c["dim"], device=dy.device).index_add_(0, st.ids, dy)
        return (dw * st.scale).to(st.grad)
    if c["op"] == "dropout":
        return _dropped(st, st.x.float()).to(st.dtype)
    if c["op"] == "ln_fwd":
        h = _dropped(st, st.x.float())
        if st.r is not None:
            h = h + st.r.float()
        mean = h.mean(1, keepdim=True)
        d = h - mean
        rstd = 1.0 / torch.sqrt(d.square().mean(1, keepdim=True) + EPS)
        y = d * rstd * st.gamma + st.beta
        return y.to(st.dtype), h.to(st.dtype), mean.flatten(), rstd.flatten()
    dy, rstd = st.dy.float(), st.rstd[:, None]
    xh = (st.h.float() - st.mean[:, None]) * rstd
    g = dy * st.gamma
    dr = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    if st.dh is not None:
        dr = dr + st.dh.float()
    dgamma, dbeta = (dy * xh).sum(0), dy.sum(0)
    out = dr.to(st.dtype)
    return (_dropped(st, dr).to(st.dtype) if c["p"] > 0 else out), out, dgamma, dbeta


def _distinct(tokens, vocab):
    """How many different words `tokens` draws name, on average."""
    log_all, total, k = math.log(vocab + 1.0), 0.0, 0
    while k < vocab:
        n = min(vocab - k, 1 + k // 64)  # words of nearly one share together
        share = math.log((k + 1.0 + n) / (k + 1.0)) / log_all / n
        total += n * -math.expm1(tokens * math.log1p(-min(share, 1 - 1e-12)))
        k += n
    return total


def work(case):
    c, size = case, DTYPES[case["dtype"]].itemsize
    if c["op"] in ("embed", "embed_bwd"):
        N, dim = c["tokens"], c["dim"]
        pads = int(1024 * c["pad"])  # of each 1024 places, the last ones
        real = N - N // 1024 * pads - max(0, N % 1024 - (1024 - pads))
        held = N * (8 if c["ids"] == "i64" else 4)
        if c["op"] == "embed":
            return {"bytes": int(held + size * dim * (N + _distinct(real, c["vocab"]))), "flops": N * dim}
        out = DTYPES[c["grad"]].itemsize if c["grad"] != "same" else size
        return {"bytes": held + size * dim * real + out * dim * c["vocab"], "flops": dim * (real + c["vocab"])}
    n = c["rows"] * c["cols"]
    drops = c["p"] > 0
    if c["op"] == "dropout":
        return {"bytes": 2 * n * size + 16, "flops": n}
    if c["op"] == "ln_fwd":
        moved = (4 if c["stream"] else 3) * n * size
        return {"bytes": moved + 8 * (c["rows"] + c["cols"]), "flops": n * (8 + drops + c["stream"])}
    moved = (3 + c["stream"] + drops) * n * size
    return {"bytes": moved + 8 * c["rows"] + 12 * c["cols"], "flops": n * (14 + drops + c["stream"])}


# ----------------------------------------------------------------------------
# In 64 bits, from the definitions alone
# ----------------------------------------------------------------------------


def _bits_64(case, seed, offset, device):
    """The 16 bits of every element, for a seed and an offset as Python's whole numbers."""
    rows, cols = case["rows"], case["cols"]
    groups = (cols + 7) // 8
    mask = (1 << 32) - 1
    at = torch.arange(rows * groups, device=device)
    # a counter as one row of 32-bit words; products modulo 2^64 in the signed type's own arithmetic
    x = [at % groups, at // groups, torch.full_like(at, offset & mask), torch.full_like(at, offset >> 32)]
    key = [seed & mask, seed >> 32]
    for i in range(7):
        p0, p1 = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57
        k = [(key[0] + i * 0x9E3779B9) & mask, (key[1] + i * 0xBB67AE85) & mask]
        x = [((p1 >> 32) & mask) ^ x[1] ^ k[0], p1 & mask, ((p0 >> 32) & mask) ^ x[3] ^ k[1], p0 & mask]
    u = torch.empty(rows, groups * 8, dtype=torch.int32, device=device)
    for i in range(8):
        u[:, i::8] = ((x[i // 2] >> (16 * (i % 2))) & 0xFFFF).reshape(rows, groups)
    return u[:, :cols]


def _dropout_64(st, x):
    p = st.case["p"]
    if p == 0:
        return x
    pair = [int(v) % 2 ** 64 for v in st.rng.tolist()]
    u = _bits_64(st.case, pair[0], (pair[1] + st.layer) % 2 ** 64, x.device)
    t = int(math.floor(65536 * p + 0.5))
    return torch.zeros_like(x).masked_scatter_(u >= t, x[u >= t] * (65536 / (65536 - t)))


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        return torch.index_select(st.weight.double(), 0, st.ids.long()) * math.sqrt(case["dim"])
    if op == "embed_bwd":
        # the places in the order of their tokens; a token's sum from differences of its own rows alone
        order = torch.argsort(st.ids.long(), stable=True)
        ids = st.ids.long()[order]
        words, counts = torch.unique_consecutive(ids, return_counts=True)
        out = torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device=st.dy.device)
        begin = 0
        for n, w in zip(counts.tolist(), words.tolist()):
            if st.padding is None or w != st.padding:
                out[w] = st.dy[order[begin:begin + n]].double().sum(0) * math.sqrt(case["dim"])
            begin += n
        return out
    if op == "dropout":
        return _dropout_64(st, st.x.double())
    if op == "ln_fwd":
        h = _dropout_64(st, st.x.double()) + (0 if st.r is None else st.r.double())
        var, mean = torch.var_mean(h, 1, correction=0)
        rstd = (var + EPS) ** -0.5
        y = torch.addcmul(st.beta.double(), (h - mean[:, None]) * rstd[:, None], st.gamma.double())
        return y, h, mean, rstd
    dy, rstd = st.dy.double(), st.rstd.double()
    xh = (st.h.double() - st.mean.double()[:, None]) * rstd[:, None]
    g, n = dy * st.gamma.double(), case["cols"]
    a, b = g.sum(1) / n, torch.einsum("rc,rc->r", g, xh) / n
    dr = (g - a[:, None] - xh * b[:, None]) * rstd[:, None] + (0 if st.dh is None else st.dh.double())
    return _dropout_64(st, dr), dr, torch.einsum("rc,rc->c", dy, xh), dy.sum(0)
