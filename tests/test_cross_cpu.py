"""pa_cross_attention's refusals, on a machine without a GPU: bad arguments return a status before any CUDA call, and
the binding refuses tensors that the library cannot take."""
import ctypes
import os
import re
import struct
import subprocess

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


@pytest.mark.parametrize("args", [dict(T=0), dict(S=-1), dict(Hq=7), dict(D=32), dict(bs=32), dict(N=1 << 27), dict(dt=7),
                                  dict(scale=float("nan")), dict(max_len=-1), dict(qs=None), dict(out=24), dict(B=0)])
def test_the_packed_call_is_the_same_call(lib, args):
    a = dict(out=16, q=16, kc=16, vc=16, tables=16, lens=16, qs=16, ws=16, bytes=1 << 20, err=0, S=3, T=9, Hq=8, Hkv=2, D=64,
             bs=16, B=10, N=40, max_len=100, scale=0.125, dt=ops.PA_BF16, stream=0)
    a.update(args)
    fields = "out q kc vc tables lens qs ws bytes err S T Hq Hkv D bs B N max_len scale dt stream".split()
    assert lib.pa_cross_attention_packed(ops._CROSS_ARGS.pack(*(a[f] or 0 for f in fields))) == call(lib, **args)
    assert lib.pa_cross_attention_packed(None) == ops.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("name,layout", [("pa_rope_append_args", ops._ROPE_ARGS), ("pa_cross_attention_args", ops._CROSS_ARGS)])
def test_the_struct_is_laid_out_as_in_c(tmp_path, name, layout):
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    fields = re.search(r"typedef struct " + name + r" \{(.*?)\}", open(os.path.join(header, "paged_attention.h")).read(), re.S)[1]
    fields = re.findall(r"(\w+)\s*[,;]", fields)
    src = (f'#include <stdio.h>\n#include "paged_attention.h"\n#define P(f) '
           f'printf("%zu %zu\\n", offsetof({name}, f), sizeof((({name}*)0)->f))\n'
           f'int main(void) {{ {"".join(f"P({f});" for f in fields)} return 0; }}\n')
    exe = str(tmp_path / "offsets")
    subprocess.run(["gcc", "-std=c99", "-I", header, "-x", "c", "-", "-o", exe], input=src, text=True, check=True)
    c = [tuple(map(int, line.split())) for line in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines()]
    codes = [ch for n, ch in re.findall(r"(\d*)([A-Za-z])", layout.format) for _ in range(int(n or 1))]
    assert len(codes) == len(c) == len(fields)
    for i, (ch, (offset, size)) in enumerate(zip(codes, c)):
        assert struct.calcsize("".join(codes[:i + 1])) == offset + size and struct.calcsize(ch) == size, fields[i]
