"""LayerNorm without dropout from host threads at once: each launch finds its kernel's limit of shared memory as it needs it."""

import ctypes
import threading

import pytest
import torch

from bwd_flashattention_fwd_sm_gb300 import _lib, layernorm_residual
from bwd_flashattention_fwd_sm_gb300._lib import LnParamsC

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype, few, many", [("bfloat16", 4104, 8192), ("float32", 2052, 4096), ("bfloat16", 8200, 16384)])
@pytest.mark.parametrize("residual", [False, True])
def test_threads_without_dropout(dtype, few, many, residual):
    """The same kernel with rows of two lengths, hence with two sizes of its ring of stages.  The C entry with
    arguments made before, so that the threads spend their time in it, where none holds the interpreter."""
    lib, dt = _lib.load(), getattr(torch, dtype)
    work = []
    for cols in (few, many, few, many):
        x = torch.randn(3, cols, device="cuda").to(dt)
        y = torch.empty_like(x)
        p = LnParamsC(3, cols, cols, cols, cols, cols, 1e-5, _lib.ATTN_BF16 if dt == torch.bfloat16 else _lib.ATTN_F32)
        stream = torch.cuda.Stream()
        args = (p, x.data_ptr(), x.data_ptr() if residual else None, None, None, y.data_ptr(), None, None, None,
                ctypes.c_void_p(stream.cuda_stream))
        work.append((args, stream, x, y, layernorm_residual(x, x if residual else None, return_sum=False)))
    torch.cuda.synchronize()
    codes, together = set(), threading.Barrier(len(work))

    def calls(args):
        together.wait()
        codes.update({lib.ln_residual_fwd(*args) for _ in range(5000)})

    threads = [threading.Thread(target=calls, args=(w[0],)) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == {_lib.ATTN_OK}
    assert all(torch.equal(y, ref) for *_, y, ref in work)
