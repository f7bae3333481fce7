"""A prompt written to the 4-bit cache and attended over there, against the full attention in float32 on the
values read back in float32 (which are what the cache stands for, but for one float32 rounding).

Bounds as in test_gpu_kv4.py, with d for both sides: each p is off by d = (D + 16) eps W + n eps + 2^-21 on
either side and by 2 eps W for the rounding of the keys read back; O by 4 d A, the weights' rounding 2^-11 A
(bfloat16), and its own.
"""

import pytest
import torch

from bwd_flashattention_fwd_sm_gb300 import Kv4Cache, attn_fwd, attn_fwd_kv4, get_status, kv4_read, kv4_write

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
EPS = 2.0 ** -24


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D, prompt", [(64, 45), (128, 300), (256, 129)])
def test_prompt_over_the_cache_is_the_full_attention(D, prompt, dtype):
    B, Hq, Hkv, page = 2, 8, 2, 16
    g = torch.Generator(device=DEV).manual_seed(D)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV).to(dtype)  # noqa: E731
    per = -(-prompt // page)
    cache = Kv4Cache.empty(2 * per + 3, Hkv, page, D, device=DEV)
    table = torch.randperm(2 * per + 3, generator=g, device=DEV)[: 2 * per].to(torch.int32).view(2, per)
    lens = torch.full((B,), prompt, dtype=torch.int32, device=DEV)
    q = rand(B, Hq, prompt, D)
    kv4_write(cache, rand(B, Hkv, prompt, D), rand(B, Hkv, prompt, D), table, lens)
    o, lse = attn_fwd_kv4(q, cache, table, lens)
    k, v = kv4_read(cache, table, lens, prompt, dtype=torch.float32)
    ro, rl = attn_fwd(q.float(), k, v, causal=True)
    # W: scale sum |q| (16 s + |b|), the largest over the keys; A from the sizes |s (u - 8)| + |b|
    group = lambda x: x.repeat_interleave(Hq // Hkv, 1)  # noqa: E731
    sb = [s[table.long()].float().transpose(1, 2).flatten(2, 3)[:, :, :prompt] for s in (cache.k_scale, cache.v_scale)]
    s, b = ([x[..., i].repeat_interleave(64, -1) for x in sb] for i in (0, 1))
    W = (q.float().abs().double() @ group(16 * s[0] + b[0].abs()).double().transpose(2, 3)).amax(-1) * D ** -0.5
    size = (v - b[1]).abs() + b[1].abs()
    A = attn_fwd(q.float(), k, size, causal=True)[0].double()
    R = attn_fwd(q.float(), k, (v - b[1]).abs(), causal=True)[0].double()
    torch.cuda.synchronize()
    assert get_status() == 0
    d = (D + 16) * EPS * W + prompt * EPS + 2.0 ** -21 + EPS * W
    if dtype == torch.bfloat16:
        own = 2.0 ** -11 * A + 2.0 ** -8 * ro.double().abs() * (1 + 2.0 ** -8)
    else:
        own = 2 * EPS * (R + ro.double().abs())
    # the weights' far end (2^-32 of the largest step and offset, 8 codes) is below d n here
    assert torch.all((o.double() - ro.double()).abs() <= 4 * d[..., None] * A + own)
    assert torch.all((lse.double() - rl.double()).abs() <= 2 * d + 8 * EPS * rl.double().abs())
