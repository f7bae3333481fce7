"""The 4-bit key/value cache: quantising keys and values as they are written, reading
them back, and attention over the cache.

The cache.  Pages of `page` positions, one page list (a row of `table`) per
sequence; `lens` counts a sequence's positions.  Each row of head_dim values is cut
into groups of 64.  With lo and hi a group's least and largest value,
    s = bf16((hi - lo) / 15)  (0 if below 2^-126),   b = bf16(lo + 8 s),
    u = clamp(round((x - b) (1 / s)) + 8, 0, 15)     (8 if s = 0),
every difference, product and quotient rounded to float32 and halves to the even
code, so that a value next to a border has one code.  The group then stands for
the values s (u - 8) + b.  Scales are stored as (s, b) pairs [pages, heads, page,
groups, 2], codes as bytes [pages, heads, page, head_dim / 2]: seen as 32-bit words
[8, groups], word (i, g) holds the values 8 i .. 8 i + 7 of group g, the first in its
lowest 4 bits.

The n newest tokens of a sequence (all three operators take or give those) are its
positions len - n .. len - 1.  Attention: query i of n sits at position len - n + i,
sees the positions up to its own (all of them where `causal` is false), and gives
O = softmax(scale Q K^T) V and the log of the softmax's sum.

`run` returns what the cache holds as the values that it stands for.
"""

import math

import torch

own = False

GROUP = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _case(name, op, dtype, batch, heads_q, heads_kv, head_dim, page, new, length, ragged, packed, causal=True):
    """op: "write" (write the new tokens, then read them back), "read" (the newest
    `new` tokens), "attend".  ragged: lengths spread over the range up to `length`.
    packed: the new tokens' counts differ too (up to `new`) and their rows stand
    one after the other, [tokens, heads, head_dim]; else [batch, heads, new, head_dim]."""
    return {"name": name, "op": op, "dtype": dtype, "batch": batch, "heads_q": heads_q, "heads_kv": heads_kv,
            "head_dim": head_dim, "page": page, "new": new, "length": length, "ragged": ragged, "packed": packed,
            "causal": causal}


def listed():
    return [
        # one decoding step's new token of each sequence: latency
        _case("write_token", "write", "bf16", 32, 32, 8, 128, 16, 1, 4096, True, False),
        # prompts of different lengths, packed: the cache's bulk write
        _case("write_prompts", "write", "bf16", 16, 32, 32, 128, 64, 8192, 8192, True, True),
        # float32 keys and values, head dim 64, an odd length
        _case("write_f32_d64", "write", "f32", 2, 16, 16, 64, 32, 2047, 4096, False, False),
        # a whole long context back into bf16, for a pass on the tensor cores
        _case("read_long", "read", "bf16", 1, 32, 8, 128, 256, 131072, 131072, False, False),
        # short contexts of different lengths, head dim 256
        _case("read_d256", "read", "bf16", 8, 16, 16, 256, 16, 600, 600, True, True),
        # one sequence, a short context: latency
        _case("decode_one", "attend", "bf16", 1, 32, 8, 128, 16, 1, 777, False, False),
        # a serving batch, ragged contexts, grouped heads
        _case("decode_batch", "attend", "bf16", 64, 32, 8, 128, 64, 1, 8192, True, False),
        # one sequence with a long context: the key axis is all there is to split
        _case("decode_long", "attend", "bf16", 1, 32, 8, 128, 256, 1, 131072, False, False),
        # float32 queries, one query head for each key head, head dim 64
        _case("decode_f32_d64", "attend", "f32", 8, 16, 16, 64, 32, 1, 8192, True, False),
        # head dim 256, ragged
        _case("decode_d256", "attend", "bf16", 16, 16, 16, 256, 128, 1, 4100, True, False),
        # a few proposed tokens of each sequence checked at once
        _case("verify_tokens", "attend", "bf16", 16, 32, 8, 128, 16, 5, 4096, True, False),
        # a chunk of each prompt over what the cache already holds
        _case("prompt_chunk", "attend", "bf16", 2, 32, 8, 128, 64, 512, 8192, True, False),
    ]


def draw(rng):
    def log_int(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))

    op = rng.choice(["write", "read", "attend", "attend", "attend"])
    heads_q, heads_kv = rng.choice([(32, 8), (16, 16), (32, 32), (16, 2), (8, 1), (4, 2), (12, 4)])
    head_dim = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    length = log_int(1, 131072)
    batch = log_int(1, 64)
    ragged, packed = rng.random() < 0.6, rng.random() < 0.4
    row = heads_kv * head_dim
    if op == "attend":
        new = min(length, rng.choice([1, 1, 1, log_int(2, 16), log_int(17, 512)]))
        most = (1 << 28) // row  # half of the rows of a ragged decode_batch's longest
        while batch > 1 and (batch * length > most or batch * new * length * heads_q * head_dim > 1 << 30):
            batch //= 2
        length = max(1, min(length, most, (1 << 30) // (new * heads_q * head_dim)))
        new = min(new, length)
    else:
        new = min(length, 1 if op == "write" and rng.random() < 0.3 else log_int(1, length))
        most = (1 << 27) // row
        while batch > 1 and batch * length > most:
            batch //= 2
        length = min(length, most)
        new = min(new, length)
    c = _case("", op, rng.choice(["bf16", "bf16", "f32"]), batch, heads_q, heads_kv, head_dim, page, new, length,
              ragged, packed, rng.random() < 0.8)
    del c["name"]
    return c


def _spread(n, lo, hi):
    """n whole numbers spread evenly over lo .. hi (multiples of the golden ratio, modulo 1)."""
    return [lo + int((hi - lo + 1) * (((i + 1) * 0.6180339887498949) % 1.0)) for i in range(n)]


def _shape(case):
    """Per sequence: the new tokens and the whole length, as lists."""
    b = case["batch"]
    new = _spread(b, 1 + (case["new"] - 1) // 64, case["new"]) if case["packed"] else [case["new"]] * b
    length = _spread(b, 1 + (case["length"] - 1) // 64, case["length"]) if case["ragged"] else [case["length"]] * b
    return new, [max(n, t) for n, t in zip(new, length)]


# ----------------------------------------------------------------------------
# The cache's format
# ----------------------------------------------------------------------------


def _pack(u):
    """Codes 0 .. 15 [..., head_dim] to bytes [..., head_dim / 2]."""
    w = u.to(torch.uint8).unflatten(-1, (-1, 8, 8)).transpose(-3, -2)  # [..., 8 (i), groups, 8]
    return (w[..., 0::2] | (w[..., 1::2] << 4)).flatten(-3)


def _unpack(p):
    """The other way round."""
    n = p.shape[-1] // (GROUP // 2)
    w = p.unflatten(-1, (8, n, 4)).transpose(-3, -2)  # [..., groups, 8 (i), 4]
    return torch.stack([w & 15, w >> 4], -1).flatten(-4)


def _quantise(x):
    """x float32 [..., head_dim]: codes as bytes, and (s, b) as bf16 [..., groups, 2]."""
    g = x.unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1, True), g.amax(-1, True)
    s = ((hi - lo) / torch.full_like(hi, 15.0)).to(torch.bfloat16).float()
    s = torch.where(s < 2.0 ** -126, 0.0, s)
    b = (lo + 8.0 * s).to(torch.bfloat16).float()
    u = ((g - b) * torch.where(s > 0, 1.0 / s, 0.0)).round().add(8.0).clamp(0.0, 15.0)
    return _pack(u.flatten(-2)), torch.cat([s, b], -1).to(torch.bfloat16)


def _values(codes, scale, dtype=torch.float32):
    """The values that codes [..., head_dim / 2] with scales [..., groups, 2] stand for."""
    u = _unpack(codes).to(dtype).unflatten(-1, (-1, GROUP))
    return ((u - 8.0) * scale[..., :1].to(dtype) + scale[..., 1:].to(dtype)).flatten(-2)


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------


class State:
    pass


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    c, st = case, State()
    dtype, D, Hq, Hkv, page = DTYPES[c["dtype"]], c["head_dim"], c["heads_q"], c["heads_kv"], c["page"]
    new, length = _shape(c)
    st.case, st.new, st.length, st.dtype = c, new, length, dtype
    st.scale = 1.0 / math.sqrt(D)
    rows = max(-(-n // page) for n in length)
    pages = sum(-(-n // page) for n in length) + 3  # a few that no sequence has
    # the new tokens of each sequence, and where the rows of a packed batch begin
    st.starts = [sum(new[:i]) for i in range(len(new) + 1)]
    st.new_dev = torch.tensor(new, device=dev)
    st.starts_dev = torch.tensor(st.starts, device=dev)
    st.lens = torch.tensor(length, dtype=torch.int32, device=dev)
    # the pages of a sequence lie anywhere in the cache, as after many requests came and went
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    st.table = torch.zeros(c["batch"], rows, dtype=torch.int32, device=dev)
    have = torch.arange(rows, device=dev)[None, :] * page < st.lens[:, None]
    st.table[have] = order[: int(have.sum())]

    # keys with a few stronger channels, as trained models have them
    strong = 1.0 + 3.0 * (torch.rand(Hkv, 1, D, generator=g, device=dev) < 0.04)

    def values(*shape, factor=None):
        x = torch.randn(*shape, generator=g, device=dev)
        return x if factor is None else x * factor

    if c["op"] == "write":
        shape = (c["batch"], Hkv, c["new"], D)
        k, v = values(*shape, factor=strong).to(dtype), values(*shape).to(dtype)
        if c["packed"]:
            keep = torch.arange(c["new"], device=dev)[None, :] < st.new_dev[:, None]
            k, v = (x.transpose(1, 2)[keep].contiguous() for x in (k, v))
        st.k, st.v = k, v
        st.codes = [torch.zeros(pages, Hkv, page, D // 2, dtype=torch.uint8, device=dev) for _ in "kv"]
        st.scales = [torch.zeros(pages, Hkv, page, D // GROUP, 2, dtype=torch.bfloat16, device=dev) for _ in "kv"]
    else:
        (kc, ks), (vc, vs) = _quantise(values(pages, Hkv, page, D, factor=strong)), _quantise(values(pages, Hkv, page, D))
        st.codes, st.scales = [kc, vc], [ks, vs]
    if c["op"] == "attend":
        q = values(c["batch"], Hq, c["new"], D).to(dtype)
        if c["packed"]:
            keep = torch.arange(c["new"], device=dev)[None, :] < st.new_dev[:, None]
            q = q.transpose(1, 2)[keep].contiguous()
        st.q = q
    if own:  # the handles that a program keeps: the cache, and the packed batch's row starts
        from bwd_flashattention_fwd_sm_gb300 import Kv4Cache, SeqLens

        st.cache = Kv4Cache(st.codes[0], st.codes[1], st.scales[0], st.scales[1])
        st.seqlens = SeqLens(st.starts, device=dev) if c["packed"] else None
    return st


# ----------------------------------------------------------------------------
# The operators
# ----------------------------------------------------------------------------


def _places(st):
    """Page and row in it of every new token, sequence after sequence."""
    dev = st.table.device
    seq = torch.repeat_interleave(torch.arange(len(st.new), device=dev), st.new_dev, output_size=st.starts[-1])
    i = torch.arange(len(seq), device=dev) - st.starts_dev[seq]
    pos = st.lens.long()[seq] - st.new_dev[seq] + i
    return st.table.long()[seq, pos // st.case["page"]], pos % st.case["page"]


def _packed_rows(st, x):
    """[batch, heads, new, D] or packed rows as [tokens, heads, D]."""
    return x if st.case["packed"] else x.transpose(1, 2).flatten(0, 1)


def _plain_write(st):
    page, at = _places(st)
    for x, codes, scale in zip((st.k, st.v), st.codes, st.scales):
        c, s = _quantise(_packed_rows(st, x).float())
        codes[page, :, at], scale[page, :, at] = c, s


def _plain_read(st):
    page, at = _places(st)
    out = [_values(codes[page, :, at], scale[page, :, at]).to(st.dtype) for codes, scale in zip(st.codes, st.scales)]
    if st.case["packed"]:
        return out
    return [x.unflatten(0, (st.case["batch"], -1)).transpose(1, 2) for x in out]


def _all_keys(st, codes, scale, dtype):
    """Every sequence's rows, [batch, heads, positions, D] (as many as the longest list of pages has)."""
    t = st.table.long()
    return _values(codes[t], scale[t], dtype).transpose(1, 2).flatten(2, 3)


def _allowed(st, positions):
    """[batch, 1, 1, new, positions]: whether a query (right-aligned where the batch is packed) sees a position."""
    dev, n = st.table.device, st.case["new"]
    j = torch.arange(positions, device=dev)
    at = st.lens.long()[:, None] - n + torch.arange(n, device=dev)[None, :]
    ok = j[None, None, :] < st.lens.long()[:, None, None]
    if st.case["causal"]:
        ok = ok & (j[None, None, :] <= at[:, :, None])
    return ok[:, None, None]


def _attend(st, q, dtype):
    c = st.case
    B, Hq, Hkv, n = c["batch"], c["heads_q"], c["heads_kv"], c["new"]
    if c["packed"]:  # right-aligned: a sequence's last token last
        keep = torch.arange(n, device=q.device)[None, :] >= n - st.new_dev[:, None]
        full = torch.zeros(B, n, Hq, c["head_dim"], dtype=q.dtype, device=q.device)
        full[keep] = q
        q = full.transpose(1, 2)
    k = _all_keys(st, st.codes[0], st.scales[0], dtype)
    v = _all_keys(st, st.codes[1], st.scales[1], dtype)
    q = q.to(dtype).unflatten(1, (Hkv, Hq // Hkv)).flatten(2, 3)  # the queries of one key head together
    s = (torch.matmul(q, k.transpose(-1, -2)) * st.scale).unflatten(2, (Hq // Hkv, n))
    s = s.masked_fill(~_allowed(st, k.shape[2]), -math.inf)
    m = s.amax(-1, True)
    m = torch.where(m > -math.inf, m, 0.0)
    p = torch.exp(s - m)
    total = p.sum(-1, True)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (Hq // Hkv, n))
    o = torch.where(total > 0, o / total, 0.0).flatten(1, 2)
    lse = (torch.log(total) + m).squeeze(-1).flatten(1, 2)
    if c["packed"]:
        return o.transpose(1, 2)[keep], lse.transpose(1, 2)[keep].transpose(0, 1).contiguous()
    return o, lse


def run(state):
    st, op = state, state.case["op"]
    if own:
        from bwd_flashattention_fwd_sm_gb300 import attn_fwd_kv4, kv4_read, kv4_write

        if op == "attend":
            return attn_fwd_kv4(st.q, st.cache, st.table, st.lens, causal=st.case["causal"], scale=st.scale,
                                seqlens=st.seqlens)
        if op == "write":
            kv4_write(st.cache, st.k, st.v, st.table, st.lens, seqlens=st.seqlens)
        return kv4_read(st.cache, st.table, st.lens, None if st.case["packed"] else st.case["new"],
                        seqlens=st.seqlens, dtype=st.dtype)
    if op == "attend":
        o, lse = _attend(st, st.q, torch.float32)
        return o.to(st.dtype), lse
    if op == "write":
        _plain_write(st)
    return tuple(_plain_read(st))


def work(case):
    new, length = _shape(case)
    D, Hq, Hkv = case["head_dim"], case["heads_q"], case["heads_kv"]
    size = DTYPES[case["dtype"]].itemsize
    held = D // 2 + 4 * (D // GROUP)  # bytes of one row in the cache
    if case["op"] == "attend":
        rows = sum(new) * Hq
        if case["causal"]:
            pairs = sum(n * t - n * (n - 1) // 2 for n, t in zip(new, length))
        else:
            pairs = sum(n * t for n, t in zip(new, length))
        return {"bytes": 2 * held * Hkv * sum(length) + rows * (2 * D * size + 4), "flops": 4 * D * Hq * pairs}
    rows = 2 * sum(new) * Hkv
    moved = rows * (held + D * size)
    if case["op"] == "read":
        return {"bytes": moved, "flops": 2 * rows * D}
    return {"bytes": 2 * moved, "flops": 8 * rows * D}


# ----------------------------------------------------------------------------
# In 64 bits, from the definitions alone
# ----------------------------------------------------------------------------


def _f32_64(x):
    """x (float64) rounded to float32: where the definition rounds."""
    return x.float().double()


def _bf16_64(x):
    """x (float64) rounded to the nearest number of 8 significant bits, ties to even."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(torch.ldexp(m, torch.full_like(e, 8))), e - 8)


def _held_64(x):
    """What the cache then stands for: x (float64, [..., D]) through the format's definition."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    lo, hi = g.min(-1, keepdim=True).values, g.max(-1, keepdim=True).values
    s = _bf16_64(_f32_64(_f32_64(hi - lo) / 15))
    s = s * (s >= 2.0 ** -126)
    b = _bf16_64(_f32_64(lo + 8 * s))
    u = torch.round(_f32_64(_f32_64(g - b) * _f32_64(1 / s.masked_fill(s == 0, math.inf)))) + 8
    return (s * (u.clamp(0, 15) - 8) + b).reshape(x.shape)


def _rows_64(codes, scale):
    """One sequence's rows [heads, positions, D] as float64: word (i, g) of a row holds the values 8 i .. of group g."""
    n = scale.shape[-2]
    word = codes.contiguous().view(torch.int32).reshape(*codes.shape[:-1], 8, n).long()
    u = torch.stack([(word >> (4 * e)) & 15 for e in range(8)], -1)  # [..., i, g, e]
    u = u.movedim(-2, -3).reshape(*codes.shape[:-1], n, GROUP).double()
    return (scale[..., 0, None].double() * (u - 8) + scale[..., 1, None].double()).reshape(*codes.shape[:-1], n * GROUP)


def exact(case, seed):
    st = prepare(case, seed)
    c, page = case, case["page"]
    Hq, Hkv = c["heads_q"], c["heads_kv"]
    first, lse_all = [], []
    second = []
    for b in range(c["batch"]):
        n, t = st.new[b], st.length[b]
        rows = slice(st.starts[b], st.starts[b + 1])
        ids = st.table[b, : -(-t // page)].long()
        if c["op"] == "write":
            k, v = ((x[rows] if c["packed"] else x[b].transpose(0, 1)).double() for x in (st.k, st.v))
            first.append(_held_64(k))
            second.append(_held_64(v))
            continue
        k, v = (_rows_64(codes[ids], scale[ids]).transpose(0, 1).reshape(Hkv, -1, c["head_dim"])[:, :t]
                for codes, scale in zip(st.codes, st.scales))
        if c["op"] == "read":
            first.append(k[:, t - n:].transpose(0, 1))
            second.append(v[:, t - n:].transpose(0, 1))
            continue
        q = (st.q[rows] if c["packed"] else st.q[b].transpose(0, 1)).double()  # [n, Hq, D]
        q = q.reshape(n, Hkv, Hq // Hkv, -1).permute(1, 2, 0, 3)
        s = (q.flatten(1, 2) @ k.transpose(1, 2)).reshape(Hkv, Hq // Hkv, n, t) / math.sqrt(c["head_dim"])
        if c["causal"]:
            late = torch.arange(t, device=s.device)[None, :] > t - n + torch.arange(n, device=s.device)[:, None]
            s = s.masked_fill(late, -math.inf)
        lse = torch.logsumexp(s, -1)
        o = torch.exp(s - lse[..., None]).flatten(1, 2) @ v
        first.append(o.reshape(Hq, n, -1).transpose(0, 1))
        lse_all.append(lse.reshape(Hq, n))
    if c["packed"]:
        a = torch.cat(first)
        return (a, torch.cat(lse_all, 1)) if c["op"] == "attend" else (a, torch.cat(second))
    a = torch.stack(first).transpose(1, 2)
    return (a, torch.stack(lse_all)) if c["op"] == "attend" else (a, torch.stack(second).transpose(1, 2))
