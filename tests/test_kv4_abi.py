"""The 4-bit cache's C entries without a GPU: refusals before any device work, and the
index arithmetic that the kernels check on the device, compiled for the host."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from bwd_flashattention_fwd_sm_gb300 import Kv4Cache, _lib, build
from bwd_flashattention_fwd_sm_gb300._lib import Kv4ParamsC

FAKE = 1 << 20  # an aligned non-NULL address; never dereferenced by host validation
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def params(**kw):
    p = Kv4ParamsC(batch=2, heads_q=8, heads_kv=2, head_dim=128, page_size=16, n_pages=10, max_pages=4, seqlen=3,
                   block_table=FAKE, table_stride=4, lens=FAKE, x_stride_b=8 * 3 * 128, x_stride_h=3 * 128,
                   x_stride_s=128, y_stride_b=8 * 3 * 128, y_stride_h=3 * 128, y_stride_s=128, scale=0.1,
                   dtype=_lib.ATTN_BF16, causal=1)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def calls(lib, p, ptr=FAKE, ws_bytes=1 << 40):
    return (lib.attn_kv4_write(p, ptr, FAKE, FAKE, FAKE, FAKE, FAKE, None),
            lib.attn_kv4_read(p, FAKE, FAKE, FAKE, FAKE, ptr, FAKE, None),
            lib.attn_fwd_kv4(p, ptr, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, ws_bytes, None))


def test_valid_calls_fail_only_for_want_of_a_gpu(lib):
    assert calls(lib, params()) == (_lib.ATTN_ERR_CUDA,) * 3
    assert calls(lib, params(dtype=_lib.ATTN_F32)) == (_lib.ATTN_ERR_CUDA,) * 3


@pytest.mark.parametrize("change, code", [
    ({"dtype": 7}, _lib.ATTN_ERR_INVALID_ARG),
    ({"heads_kv": 0}, _lib.ATTN_ERR_INVALID_ARG),
    ({"head_dim": 96}, _lib.ATTN_ERR_UNSUPPORTED),
    ({"page_size": 0}, _lib.ATTN_ERR_INVALID_ARG),
    ({"page_size": 24}, _lib.ATTN_ERR_INVALID_ARG),
    ({"batch": -1}, _lib.ATTN_ERR_INVALID_ARG),
    ({"max_pages": -1}, _lib.ATTN_ERR_INVALID_ARG),
    ({"lens": None}, _lib.ATTN_ERR_INVALID_ARG),
    ({"block_table": None}, _lib.ATTN_ERR_INVALID_ARG),
    ({"table_stride": 3}, _lib.ATTN_ERR_INVALID_ARG),
    ({"x_stride_s": 100}, _lib.ATTN_ERR_INVALID_ARG),
    ({"y_stride_h": -128}, _lib.ATTN_ERR_INVALID_ARG),
    ({"seqlen": 1 << 30}, _lib.ATTN_ERR_UNSUPPORTED),
])
def test_refusals(lib, change, code):
    assert calls(lib, params(**change)) == (code,) * 3
    assert lib.attn_last_error() != b""


def test_refusals_of_the_attention(lib):
    for change in ({"heads_q": 0}, {"heads_q": 7}, {"scale": float("nan")}):
        p = params(**change)
        assert calls(lib, p)[2] == _lib.ATTN_ERR_INVALID_ARG
        assert lib.attn_kv4_workspace_size(p) == _lib.SIZE_MAX
    need = lib.attn_kv4_workspace_size(params())
    if need:
        assert calls(lib, params(), ws_bytes=need - 1)[2] == _lib.ATTN_ERR_WORKSPACE
        assert lib.attn_fwd_kv4(params(), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, need,
                                None) == _lib.ATTN_ERR_WORKSPACE
        assert lib.attn_fwd_kv4(params(), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE + 16, need,
                                None) == _lib.ATTN_ERR_WORKSPACE
    assert lib.attn_fwd_kv4(params(), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, 1 << 40,
                            None) == _lib.ATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    {"n_pages": 1 << 27},                                              # 2^32 rows
    {"n_pages": (1 << 31) - 1, "page_size": 1 << 30, "max_pages": 1},  # and far more
    {"max_pages": (1 << 26) + 1, "table_stride": 1 << 27},             # 2^30 + 16 positions of a sequence
    {"max_pages": (1 << 31) - 1, "table_stride": 1 << 31, "page_size": 1 << 30},
    {"seqlen": 1 << 27, "batch": 1, "heads_q": 10},                    # more than 2^30 query rows
])
def test_sizes_that_the_attention_refuses(lib, change):
    p = params(**change)
    assert calls(lib, p) == (_lib.ATTN_ERR_CUDA, _lib.ATTN_ERR_CUDA, _lib.ATTN_ERR_UNSUPPORTED)
    assert lib.attn_kv4_workspace_size(p) == _lib.SIZE_MAX
    near = params(n_pages=(1 << 27) - 1, max_pages=1 << 26, table_stride=1 << 27)
    assert calls(lib, near)[2] == _lib.ATTN_ERR_CUDA


def test_pointers(lib):
    assert calls(lib, params(), ptr=None) == (_lib.ATTN_ERR_INVALID_ARG,) * 3
    assert calls(lib, params(), ptr=FAKE + 8) == (_lib.ATTN_ERR_INVALID_ARG,) * 3


def test_packed_batches(lib):
    def packed(cu, **kw):
        cu = np.asarray(cu, np.int32)
        p = params(cu_seqlens=FAKE, cu_seqlens_host=cu.ctypes.data, batch=len(cu) - 1, **kw)
        return calls(lib, p), cu

    assert packed([0, 3, 5])[0] == (_lib.ATTN_ERR_CUDA,) * 3
    assert packed([1, 3, 5])[0] == (_lib.ATTN_ERR_INVALID_ARG,) * 3  # does not start at 0
    assert packed([0, 3, 2])[0] == (_lib.ATTN_ERR_INVALID_ARG,) * 3  # decreases
    assert packed([0, 1, 5])[0] == (_lib.ATTN_ERR_INVALID_ARG,) * 3  # 4 rows, seqlen 3
    assert packed([0, 0, 0])[0] == (_lib.ATTN_OK,) * 3               # no row at all
    assert calls(lib, params(cu_seqlens=FAKE)) == (_lib.ATTN_ERR_INVALID_ARG,) * 3


def test_nothing_to_do_is_no_work(lib):
    for change in ({"batch": 0}, {"seqlen": 0}):
        p = params(**change)
        assert lib.attn_kv4_workspace_size(p) == 0
        assert lib.attn_kv4_write(p, *[None] * 7) == _lib.ATTN_OK
        assert lib.attn_kv4_read(p, *[None] * 7) == _lib.ATTN_OK
        assert lib.attn_fwd_kv4(p, *[None] * 8, 0, None) == _lib.ATTN_OK


def test_the_binding_has_no_cpu_path():
    codes = torch.zeros(2, 1, 16, 64, dtype=torch.uint8)
    scale = torch.zeros(2, 1, 16, 2, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        Kv4Cache(codes, codes, scale, scale)


def test_device_side_checks_on_the_host(tmp_path):
    """Pages, lengths and packed rows that the kernels refuse, through the very functions they call."""
    nvcc = build.nvcc()
    if not shutil.which(nvcc) and not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path / "kv4_index")
    src = os.path.join(ROOT, "tests", "kv4_index_host.cu")
    r = subprocess.run([nvcc, "-std=c++17", "-I", build.CSRC, "-I", build.INCLUDE, src, "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
