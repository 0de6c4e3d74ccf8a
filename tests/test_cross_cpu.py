"""pa_cross_attention's refusals, on a machine without a GPU: bad arguments return a status before any CUDA call, and
the binding refuses tensors that the library cannot take."""
import ctypes

import pytest
import torch

from paged_kv_cache_456_b200 import ops

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_456_b200 import build
    build.build()
    return ops.library()


def call(lib, **kw):
    a = dict(out=P(16), q=P(16), kc=P(16), vc=P(16), tables=P(16), lens=P(16), qs=P(16), S=3, T=9, Hq=8, Hkv=2, D=64, bs=16,
             B=10, N=40, max_len=100, scale=0.125, dt=ops.PA_BF16, ws=P(16), bytes=1 << 20)
    a.update(kw)
    return lib.pa_cross_attention(a["out"], a["q"], a["kc"], a["vc"], a["tables"], a["lens"], a["qs"], a["S"], a["T"], a["Hq"],
                                  a["Hkv"], a["D"], a["bs"], a["B"], a["N"], a["max_len"], a["scale"], a["dt"], a["ws"],
                                  a["bytes"], None, None)


@pytest.mark.parametrize("bad", [
    dict(S=-1), dict(T=-1), dict(S=0), dict(Hq=0), dict(Hkv=0), dict(Hq=7), dict(D=0), dict(bs=0), dict(B=0), dict(N=0),
    dict(max_len=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(dt=7), dict(out=None), dict(q=None),
    dict(kc=None), dict(vc=None), dict(tables=None), dict(lens=None), dict(qs=None), dict(out=P(24)), dict(q=P(20)),
    dict(kc=P(8)), dict(vc=P(18))])
def test_invalid_arguments(lib, bad):
    assert call(lib, **bad) == ops.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("far", [
    dict(D=32), dict(D=256), dict(Hq=6), dict(Hq=32), dict(bs=32), dict(T=1 << 30), dict(N=1 << 27),
    dict(B=1 << 30, max_len=(1 << 31) - 1)])
def test_unsupported_shapes(lib, far):
    assert call(lib, **far) == ops.PA_ERR_UNSUPPORTED


def test_no_rows_is_fine(lib):
    assert call(lib, T=0) == ops.PA_OK
    assert call(lib, T=0, S=0, q=None, out=None) == ops.PA_OK


def test_workspace_size_refuses(lib):
    n = ctypes.c_size_t(0)
    f = lib.pa_cross_attention_workspace_size
    assert f(2, 4, 8, 2, 64, 100, ops.PA_BF16, None) == ops.PA_ERR_INVALID_ARG
    assert f(-1, 4, 8, 2, 64, 100, ops.PA_BF16, ctypes.byref(n)) == ops.PA_ERR_INVALID_ARG
    assert f(2, -4, 8, 2, 64, 100, ops.PA_BF16, ctypes.byref(n)) == ops.PA_ERR_INVALID_ARG
    assert f(2, 4, 8, 2, 80, 100, ops.PA_BF16, ctypes.byref(n)) == ops.PA_ERR_UNSUPPORTED
    assert f(2, 4, 12, 4, 64, 100, ops.PA_F32, ctypes.byref(n)) == ops.PA_ERR_UNSUPPORTED


def test_the_binding_refuses_host_tensors():
    q, c = torch.zeros(3, 4, 64), torch.zeros(2, 2, 16, 64)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ops.cross_attention(q, q, c, c, i[:, None], i, torch.zeros(3, dtype=torch.int32), scale=1.0, max_context_len=16,
                            workspace=torch.zeros(64, dtype=torch.uint8))
