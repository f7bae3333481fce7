"""The training loop that README.md shows, run with stand-ins for the operators: no mask comes twice, and a
backward pass gets the seed and offset of its forward pass."""

import os
import re
import sys
import types

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = "bwd_flashattention_fwd_sm_gb300"


class Value:
    """Any tensor; remembers which dropout made it."""
    shape = (1,)

    def __init__(self, drop=None):
        self.drop = drop


def test_every_dropout_of_every_step_has_a_mask_of_its_own(monkeypatch):
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = [b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "layernorm_residual_bwd" in b]
    assert len(blocks) == 1
    forward, backward = [], []

    def key(rng, offset, seed=0):
        return (rng[0] + seed) % 2 ** 64, (rng[1] + offset) % 2 ** 64

    def layernorm_residual(*_, rng, offset, **kw):
        forward.append(key(rng, offset))
        return Value(), Value(), Value(), Value()

    def layernorm_residual_bwd(*_, rng, offset, **kw):
        backward.append(key(rng, offset))
        return Value(), Value(), Value(), Value()

    def dropout(x, p, *, rng, offset, **kw):
        # the first use of a sum is the forward pass
        (backward if key(rng, offset) in forward else forward).append(key(rng, offset))
        return x

    fake = types.ModuleType(PACKAGE)
    fake.__dict__.update(layernorm_residual=layernorm_residual, layernorm_residual_bwd=layernorm_residual_bwd,
                         dropout=dropout, embedding=lambda *_, **kw: Value(), embedding_bwd=lambda *_, **kw: Value())
    monkeypatch.setitem(sys.modules, PACKAGE, fake)
    torch = types.SimpleNamespace(tensor=lambda v, device=None: list(v))
    names = {n: Value() for n in ("table", "ids", "residual", "gamma", "beta", "dy", "dh", "z", "dz")}
    steps = 5
    exec(blocks[0], dict(names, torch=torch, seed=123, steps=steps, step=0))
    assert len(forward) >= 2 * steps and len(set(forward)) == len(forward)
    assert sorted(backward) == sorted(forward)
