"""pa_rope_append's refusals, on a machine without a GPU: bad arguments return a status before any CUDA call, and the
binding refuses tensors that the library cannot take."""
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
    a = dict(q_out=P(16), q=P(16), key=P(16), value=P(16), kc=P(16), vc=P(16), slots=P(16), pos=P(16), freq=P(16), axis=None,
             axes=1, rot=64, style=0, rot_scale=1.0, os=512, qs=512, ks=128, vs=128, T=4, Hq=8, Hkv=2, D=64, bs=16, N=10,
             dt=ops.PA_BF16)
    a.update(kw)
    return lib.pa_rope_append(a["q_out"], a["q"], a["key"], a["value"], a["kc"], a["vc"], a["slots"], a["pos"], a["freq"],
                              a["axis"], a["axes"], a["rot"], a["style"], a["rot_scale"], a["os"], a["qs"], a["ks"], a["vs"],
                              a["T"], a["Hq"], a["Hkv"], a["D"], a["bs"], a["N"], a["dt"], None, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(axes=0), dict(axes=9), dict(rot=0), dict(rot=80), dict(rot=-16), dict(D=0), dict(style=2), dict(dt=5),
    dict(rot_scale=float("nan")), dict(rot_scale=float("inf")), dict(Hq=0), dict(Hkv=0), dict(bs=0), dict(N=0),
    dict(q=None), dict(q_out=None), dict(key=None), dict(value=None), dict(kc=None), dict(vc=None), dict(slots=None),
    dict(pos=None), dict(freq=None), dict(q=P(24)), dict(q_out=P(8)), dict(key=P(18)), dict(value=P(20)), dict(kc=P(8)),
    dict(vc=P(8)), dict(qs=500), dict(qs=504), dict(qs=-512), dict(os=256), dict(ks=64), dict(vs=0), dict(ks=130),
    dict(os=1024),                                                              # in place with two strides
    dict(q_out=None, q=None, key=None, value=None, kc=None, vc=None, slots=None),  # nothing to do, with tokens
    dict(D=20, rot=16), dict(D=66, rot=64, dt=ops.PA_F32)])                     # rows that are not whole 16-byte chunks
def test_invalid_arguments(lib, bad):
    assert call(lib, **bad) == ops.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("far", [dict(rot=24), dict(rot=8), dict(D=8192, Hq=1, Hkv=1), dict(Hq=1 << 16, qs=1 << 22, os=1 << 22)])
def test_unsupported_shapes(lib, far):
    assert call(lib, **far) == ops.PA_ERR_UNSUPPORTED


def test_no_tokens_is_fine(lib):
    assert call(lib, T=0) == ops.PA_OK
    assert call(lib, T=0, q=None, q_out=None, key=None, value=None) == ops.PA_OK


def test_the_binding_refuses():
    T, D = 3, 64
    q, k = torch.zeros(T, 4, D), torch.zeros(T, 2, D)
    cache, slots = torch.zeros(2, 2, 16, D), torch.zeros(T, dtype=torch.int64)
    pos, freq = torch.zeros(T, dtype=torch.int64), torch.ones(32)
    with pytest.raises(ValueError, match="CUDA"):                       # host memory
        ops.rope_append(q, q, k, k, cache, cache, slots, pos, freq)
    with pytest.raises(ValueError, match="together"):
        ops.rope_append(None, q, k, k, cache, cache, slots, pos, freq)
    with pytest.raises(ValueError, match="together"):
        ops.rope_append(q, q, k, None, cache, cache, slots, pos, freq)
    with pytest.raises(ValueError, match="needs"):
        ops.rope_append(None, None, None, None, None, None, None, pos, freq)


@pytest.mark.parametrize("name,t,shape,dtype", [
    ("rows of another shape", torch.zeros(3, 4, 64), (3, 2, 64), torch.float32),
    ("rows of another type", torch.zeros(3, 4, 64), (3, 4, 64), torch.bfloat16),
    ("heads apart", torch.zeros(3, 64, 4).transpose(1, 2), (3, 4, 64), torch.float32),
    ("every other head", torch.zeros(3, 8, 64)[:, ::2], (3, 4, 64), torch.float32)])
def test_rows_the_library_cannot_take(name, t, shape, dtype):
    with pytest.raises(ValueError):
        ops._rows_ptr(name, t, shape, dtype)


def test_rows_may_lie_apart():
    t = torch.zeros(3, 400)[:, 8:264].view(3, 4, 64)
    assert ops._rows_ptr("t", t, (3, 4, 64), torch.float32) == (t.data_ptr(), 400)
    with pytest.raises(ValueError):
        ops._array_ptr("a", torch.zeros(4, 6)[:, :3], (4, 3), torch.float32)


FIELDS = "q_out q key value kc vc slots pos freq axis os qs ks vs err axes rot style rot_scale T Hq Hkv D bs N dt stream".split()


@pytest.mark.parametrize("args", [dict(T=0), dict(axes=9), dict(rot=24), dict(rot_scale=float("nan")), dict(bs=0),
                                  dict(ks=64), dict(vs=0), dict(dt=5), dict(pos=None), dict(Hq=1 << 16, qs=1 << 22, os=1 << 22)])
def test_the_packed_call_is_the_same_call(lib, args):
    a = dict(q_out=16, q=16, key=16, value=16, kc=16, vc=16, slots=16, pos=16, freq=16, axis=None, axes=1, rot=64, style=0,
             rot_scale=1.0, os=512, qs=512, ks=128, vs=128, T=4, Hq=8, Hkv=2, D=64, bs=16, N=10, dt=ops.PA_BF16, err=None,
             stream=None)
    a.update(args)
    want = call(lib, **args)
    assert lib.pa_rope_append_packed(ops._ROPE_ARGS.pack(*(a[f] or 0 for f in FIELDS))) == want
    assert lib.pa_rope_append_packed(None) == ops.PA_ERR_INVALID_ARG


def test_an_argument_out_of_its_range_is_refused(lib):
    for bad in (dict(T=1 << 31), dict(D=-(1 << 31) - 1), dict(ks=1 << 63)):
        a = dict.fromkeys(FIELDS, 0) | bad
        with pytest.raises(ValueError, match="range"):
            ops._call_on(0, lib.pa_rope_append_packed, "pa_rope_append", 0, ops._ROPE_ARGS, *(a[f] for f in FIELDS[:-1]))
