"""A row operator's call on a stream of the caller's that is refused leaves the current device and stream as they were."""

import pytest
import torch

from bwd_flashattention_fwd_sm_gb300 import (dropout, embedding, embedding_bwd, layernorm_residual,
                                             layernorm_residual_bwd, rows)

CUDA0 = torch.device("cuda", 0)


class Now:
    """Stands for the current stream of a device, (stream_id, device_index, device_type)."""
    stream = (0, 0, 1)

    @staticmethod
    def make(*stream):
        Now.stream = stream


class Stream:
    device, stream_id, device_index, device_type = CUDA0, 77, 0, 1


class Tensor:
    device = CUDA0

    def __init__(self, error=None):
        self.error, self.on = error, []

    def record_stream(self, stream):
        if self.error:
            raise self.error
        assert Now.stream == (0, 0, 1)
        self.on.append(stream)


def test_what_is_refused_leaves_no_stream_current(monkeypatch):
    monkeypatch.setattr(rows, "current_device", lambda: 0)
    monkeypatch.setattr(rows, "_get_stream", lambda index: Now.stream)
    monkeypatch.setattr(rows, "_make_current", Now.make)
    s, good = Stream(), Tensor()
    with rows.elsewhere(CUDA0, s, (good, None)):
        assert Now.stream == (77, 0, 1) and good.on == [s]
    assert Now.stream == (0, 0, 1)
    with pytest.raises(KeyError):
        with rows.elsewhere(CUDA0, s, (good,)):
            raise KeyError
    assert Now.stream == (0, 0, 1)
    for bad, error in ((Tensor(RuntimeError("no such stream")), RuntimeError), (torch.zeros(1), ValueError)):
        with pytest.raises(error):
            with rows.elsewhere(CUDA0, s, (good, bad)):
                pass
        assert Now.stream == (0, 0, 1)


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


@pytest.mark.gpu
def test_a_call_runs_and_allocates_on_its_stream():
    """Nested in another current stream, too; afterwards that one is current again."""
    x = torch.randn(700, 64, device="cuda")
    ref = dropout(x, 0.3, seed=1)
    torch.cuda.synchronize()
    outer, side = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(outer):
        for _ in range(20):
            torch.cuda._sleep(100000)  # what the call must not wait for
            done = torch.cuda.Event()
            y = dropout(x, 0.3, seed=1, stream=side)
            done.record(side)
            done.synchronize()
            assert torch.cuda.current_stream() == outer
            assert torch.equal(y.cpu(), ref.cpu())
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    external = torch.cuda.ExternalStream(side.cuda_stream)
    y = dropout(x, 0.3, seed=1, stream=external)
    external.synchronize()
    assert torch.equal(y, ref) and torch.cuda.current_stream() == torch.cuda.default_stream()
