"""A row operator's call on a stream of the caller's that is refused leaves the current device and stream as they were."""

import pytest
import torch

from bwd_flashattention_fwd_sm_gb300 import (dropout, embedding, embedding_bwd, layernorm_residual,
                                             layernorm_residual_bwd, rows)

CUDA0 = torch.device("cuda", 0)


class Context:
    """Stands for torch.cuda.device and torch.cuda.stream."""
    inside = 0

    def __init__(self, _):
        pass

    def __enter__(self):
        Context.inside += 1

    def __exit__(self, *error):
        Context.inside -= 1


class Stream:
    device = CUDA0


class Tensor:
    device = CUDA0

    def __init__(self, error=None):
        self.error, self.on = error, []

    def record_stream(self, stream):
        if self.error:
            raise self.error
        assert Context.inside == 0
        self.on.append(stream)


def test_what_is_refused_leaves_no_stream_current(monkeypatch):
    monkeypatch.setattr(torch.cuda, "device", Context)
    monkeypatch.setattr(torch.cuda, "stream", Context)
    s, good = Stream(), Tensor()
    with rows.elsewhere(CUDA0, s, (good, None)):
        assert Context.inside == 2 and good.on == [s]
    assert Context.inside == 0
    for bad, error in ((Tensor(RuntimeError("no such stream")), RuntimeError), (torch.zeros(1), ValueError)):
        with pytest.raises(error):
            with rows.elsewhere(CUDA0, s, (good, bad)):
                pass
        assert Context.inside == 0


@pytest.mark.gpu
def test_host_tensors_with_a_stream():
    """A pair or a workspace on the host is refused as it is without a stream, and the stream stays what it was."""
    x = torch.randn(700, 64, device="cuda")
    one = torch.ones(700, device="cuda")
    ids = torch.zeros(700, dtype=torch.int64, device="cuda")
    rng, ws = torch.zeros(2, dtype=torch.int64), torch.zeros(1 << 22, dtype=torch.uint8)
    before, side = torch.cuda.current_stream(), torch.cuda.Stream()
    for stream in (None, side):
        for call in (lambda: dropout(x, 0.1, rng=rng, stream=stream),
                     lambda: layernorm_residual(x, dropout_p=0.1, rng=rng, stream=stream),
                     lambda: layernorm_residual_bwd(x, x, one, one, dropout_p=0.1, rng=rng, stream=stream),
                     lambda: layernorm_residual_bwd(x, x, one, one, workspace=ws, stream=stream),
                     lambda: embedding_bwd(x, ids, 5, workspace=ws, stream=stream)):
            with pytest.raises(ValueError):
                call()
            assert torch.cuda.current_stream() == before
    for call in (lambda s: embedding(x, ids, stream=s), lambda s: dropout(x, 0.1, stream=s)):
        assert torch.equal(call(None), call(before)) and torch.cuda.current_stream() == before
