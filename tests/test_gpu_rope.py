"""Rotary append (pa_rope_append) on the GPU against its definition in 64 bits.

Tolerance, element by element.  The kernel turns a pair (a, b) in fp32 and rounds each result once to the element
type (relative error at most eps / 2).  In fp32: the angle is a fraction of a turn rounded once (2^-25 of at most
one half turn: pi 2^-25 < 1e-7 rad), cos and sin carry at most one unit more (2^-24 < 6e-8), the factor rot_scale
another 2^-24, the two products and their sum 3 x 2^-24 < 1.8e-7: less than 4e-7 in all, times
|rot_scale| (|a| + |b|).
"""
import numpy as np
import pytest
import torch

from paged_kv_cache_456_b200 import ops

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_456_b200 import build
    build.build()
    ops.library()


def turned(x, positions, inv_freq, pair_axis, adjacent, rot_scale):
    """The definition in 64 bits: (result, the fp32 error allowed before the last rounding)."""
    x = x.detach().cpu().double()
    half = inv_freq.numel()
    axis = torch.zeros(half, dtype=torch.long) if pair_axis is None else pair_axis.cpu().long()
    pos = positions.cpu().double().reshape(-1, x.shape[0])
    theta = (pos[axis] * inv_freq.cpu().double()[:, None]).t()[:, None]          # [T][1][half]
    ia = torch.arange(half) * 2 if adjacent else torch.arange(half)
    ib = ia + 1 if adjacent else ia + half
    a, b = x[..., ia], x[..., ib]
    out, slack = x.clone(), torch.zeros_like(x)
    out[..., ia] = rot_scale * (a * theta.cos() - b * theta.sin())
    out[..., ib] = rot_scale * (a * theta.sin() + b * theta.cos())
    slack[..., ia] = slack[..., ib] = 4e-7 * abs(rot_scale) * (a.abs() + b.abs())
    return out, slack


def assert_turned(got, want, slack):
    half_step = torch.finfo(got.dtype).eps / 2
    err = (got.detach().cpu().double() - want).abs()
    bound = half_step * (want.abs() + slack) + slack
    assert (err <= bound).all(), f"worst error / bound {(err / bound.clamp_min(1e-300)).max():.3f}"


def bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def inputs(T, Hq, Hkv, D, rot, *, dtype="bf16", axes=1, bs=16, far=5000, seed=0, padding=0):
    g = torch.Generator().manual_seed(seed + 131 * T + D)
    dt = DT[dtype]
    rand = lambda *s: torch.randn(*s, generator=g).to(dt).cuda()  # noqa: E731
    N = -(-T // bs) + 3
    slots = torch.randperm(N * bs, generator=g)[:T]
    if padding:
        slots[torch.randperm(T, generator=g)[:padding]] = -1
    positions = torch.randint(0, far, (axes, T), generator=g)
    pair_axis = torch.randint(0, axes, (rot // 2,), generator=g).int().cuda() if axes > 1 else None
    inv_freq = (10000.0 ** (-torch.arange(rot // 2).double() / (rot // 2))).float().cuda()
    return dict(q=rand(T, Hq, D), key=rand(T, Hkv, D), value=rand(T, Hkv, D), k_cache=rand(N, Hkv, bs, D),
                v_cache=rand(N, Hkv, bs, D), slots=slots.cuda(), positions=positions.cuda(), inv_freq=inv_freq,
                pair_axis=pair_axis)


def call(x, q_out, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops.rope_append(q_out, x["q"], x["key"], x["value"], x["k_cache"], x["v_cache"], x["slots"], x["positions"],
                    x["inv_freq"], pair_axis=x["pair_axis"], err_flag=err, **kw)
    torch.cuda.synchronize()
    return int(err.item())


def check(x, adjacent=False, rot_scale=1.0, q_out=None):
    k0, v0 = x["k_cache"].clone(), x["v_cache"].clone()
    want_q, slack_q = turned(x["q"], x["positions"], x["inv_freq"], x["pair_axis"], adjacent, rot_scale)
    want_k, slack_k = turned(x["key"], x["positions"], x["inv_freq"], x["pair_axis"], adjacent, rot_scale)
    q_out = torch.full_like(x["q"], float("nan"), memory_format=torch.contiguous_format) if q_out is None else q_out
    assert call(x, q_out, adjacent=adjacent, rot_scale=rot_scale) == 0
    assert_turned(q_out, want_q, slack_q)
    slots = x["slots"].cpu()
    live = torch.nonzero(slots >= 0).flatten()
    bs = k0.shape[2]
    blk, off = slots[live] // bs, slots[live] % bs
    k, v = x["k_cache"].cpu(), x["v_cache"].cpu()
    assert_turned(k[blk, :, off], want_k[live], slack_k[live])
    assert torch.equal(bits(v[blk, :, off]), bits(x["value"].cpu()[live]))
    # dims that are not rotated: bit for bit; every other slot as it was
    rot = 2 * x["inv_freq"].numel()
    assert torch.equal(bits(q_out[..., rot:].contiguous()), bits(x["q"][..., rot:].contiguous()))
    assert torch.equal(bits(k[blk, :, off][..., rot:].contiguous()), bits(x["key"].cpu()[live][..., rot:].contiguous()))
    keep = torch.ones(k.shape[0], bs, dtype=torch.bool)
    keep[blk, off] = False
    for new, old in ((k, k0.cpu()), (v, v0.cpu())):
        assert torch.equal(bits(new.transpose(1, 2)[keep]), bits(old.transpose(1, 2)[keep]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,axes", [
    (1, 4, 2, 64, 64, 1), (1, 32, 32, 128, 128, 1), (2, 1, 1, 64, 16, 1), (17, 6, 3, 80, 48, 1), (33, 8, 8, 96, 96, 2),
    (130, 5, 1, 256, 64, 3), (300, 12, 4, 128, 128, 3), (2000, 2, 1, 64, 32, 1), (5001, 3, 1, 128, 128, 8),
    (700, 16, 2, 72, 64, 1), (3, 2, 1, 4096, 1024, 1)])
def test_matches_the_definition(dtype, adjacent, T, Hq, Hkv, D, rot, axes):
    check(inputs(T, Hq, Hkv, D, rot, dtype=dtype, axes=axes, padding=T // 7), adjacent)


@pytest.mark.parametrize("bs", [1, 7, 16, 64])
def test_block_sizes(bs):
    check(inputs(75, 4, 2, 64, 64, bs=bs))


@pytest.mark.parametrize("rot_scale", [0.75, -2.0, 0.0])
def test_rot_scale(rot_scale):
    check(inputs(40, 4, 2, 64, 32), rot_scale=rot_scale)


@pytest.mark.parametrize("far", [1 << 22, 1 << 31, 1 << 40])
@pytest.mark.parametrize("sign", [1, -1])
def test_far_positions_keep_their_angle(far, sign):
    x = inputs(64, 2, 2, 64, 64, dtype="f32")
    x["positions"] = sign * (far - torch.arange(64, device="cuda").view(1, -1))
    # 64 bits hold an angle of `far` radians to far * 2^-53, in the test as in the kernel (three roundings each)
    if far * 2.0 ** -53 * 6 > 1e-8:
        q_out = torch.empty_like(x["q"])
        assert call(x, q_out) == 0
        want, _ = turned(x["q"], x["positions"], x["inv_freq"], None, False, 1.0)
        pairs = x["q"].cpu().double().abs()
        slack = (4e-7 + 6 * far * 2.0 ** -53) * (pairs + pairs.roll(32, -1))
        assert_turned(q_out, want, slack)
    else:
        check(x)


def test_one_dimensional_positions_and_position_zero():
    x = inputs(50, 3, 1, 64, 64)
    x["positions"] = torch.zeros(50, dtype=torch.int64, device="cuda")
    q_out = torch.empty_like(x["q"])
    assert call(x, q_out) == 0
    assert torch.equal(q_out, x["q"])


def test_strided_views_of_one_projection():
    T, Hq, Hkv, D = 200, 8, 2, 64
    x = inputs(T, Hq, Hkv, D, D)
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D + 24, device="cuda").bfloat16()
    x["q"], x["key"], x["value"] = (t.view(T, -1, D) for t in
                                    qkv[:, :-24].split((Hq * D, Hkv * D, Hkv * D), dim=1))
    check(x)
    # and into a wider buffer: the bytes between its rows stay
    wide = torch.full((T, Hq * D + 40), 7.0, device="cuda", dtype=torch.bfloat16)
    check(x, q_out=wide[:, :Hq * D].view(T, Hq, D))
    assert (wide[:, Hq * D:] == 7).all()


@pytest.mark.parametrize("adjacent", [False, True])
def test_in_place(adjacent):
    x = inputs(333, 8, 2, 128, 64)
    apart = torch.empty_like(x["q"])
    assert call(x, apart, adjacent=adjacent) == 0
    assert call(x, x["q"], adjacent=adjacent) == 0
    assert torch.equal(bits(x["q"]), bits(apart))


def test_only_q_and_only_append():
    x = inputs(90, 4, 2, 64, 64)
    both = torch.empty_like(x["q"])
    assert call(x, both) == 0
    k, v = x["k_cache"].clone(), x["v_cache"].clone()
    alone = ops.rope_append(torch.empty_like(both), x["q"], None, None, None, None, None, x["positions"], x["inv_freq"])
    assert torch.equal(bits(alone), bits(both))
    k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
    assert ops.rope_append(None, None, x["key"], x["value"], k2, v2, x["slots"], x["positions"], x["inv_freq"]) is None
    blk, off = x["slots"] // 16, x["slots"] % 16
    assert torch.equal(bits(k2[blk, :, off]), bits(k[blk, :, off]))
    assert torch.equal(bits(v2[blk, :, off]), bits(v[blk, :, off]))


def test_zero_frequencies_equal_the_slot_write():
    """Frequencies of zero turn nothing: the caches are those of pa_reshape_and_cache, bit for bit."""
    x = inputs(61, 2, 2, 64, 64, padding=5)
    x["inv_freq"].zero_()
    k, v = x["k_cache"].clone(), x["v_cache"].clone()
    assert call(x, torch.empty_like(x["q"])) == 0
    ops.reshape_and_cache(x["key"], x["value"], k, v, x["slots"])
    assert torch.equal(bits(x["k_cache"]), bits(k)) and torch.equal(bits(x["v_cache"]), bits(v))


@pytest.mark.parametrize("T", [3, 3000])
def test_a_slot_past_the_cache_is_skipped(T):
    x = inputs(T, 4, 2, 64, 64)
    want, slack = turned(x["q"], x["positions"], x["inv_freq"], None, False, 1.0)
    N, bs = x["k_cache"].shape[0], 16
    x["slots"][1] = N * bs
    x["slots"][2] = 1 << 62
    k0 = x["k_cache"].clone()
    q_out = torch.empty_like(x["q"])
    assert call(x, q_out) == ops.ERRBIT_SLOT
    assert_turned(q_out, want, slack)                 # its q row is turned all the same
    changed = (bits(x["k_cache"]) != bits(k0)).any(dim=3).any(dim=1).sum().item()
    assert changed <= T - 2


def test_a_pair_without_an_axis_is_not_turned():
    x = inputs(20, 2, 1, 64, 64, axes=2)
    x["pair_axis"][5], x["pair_axis"][9] = 2, -1
    q_out = torch.empty_like(x["q"])
    assert call(x, q_out) == ops.ERRBIT_AXIS
    for p in (5, 9, 37, 41):
        assert torch.equal(q_out[..., p], x["q"][..., p])
    x["inv_freq"][[5, 9]] = 0.0
    x["pair_axis"][[5, 9]] = 0
    want, slack = turned(x["q"], x["positions"], x["inv_freq"], x["pair_axis"], False, 1.0)
    assert_turned(q_out, want, slack)


def test_non_finite_values_stay_in_their_pair():
    x = inputs(10, 2, 1, 64, 64, dtype="f32")
    x["q"][3, 1, 7] = float("nan")
    x["q"][4, 0, 40] = float("inf")
    q_out = torch.empty_like(x["q"])
    assert call(x, q_out) == 0
    fine = torch.ones_like(q_out, dtype=torch.bool)
    fine[3, 1, [7, 39]] = False
    fine[4, 0, [8, 40]] = False
    assert torch.isfinite(q_out[fine]).all() and q_out[3, 1, 7].isnan() and q_out[3, 1, 39].isnan()


def test_no_tokens():
    x = inputs(1, 2, 1, 64, 64)
    for k in ("q", "key", "value", "slots"):
        x[k] = x[k][:0]
    x["positions"] = x["positions"][:, :0]
    k0 = x["k_cache"].clone()
    assert call(x, torch.empty_like(x["q"])) == 0
    assert torch.equal(bits(k0), bits(x["k_cache"]))


def test_on_another_stream_and_in_a_graph():
    x = inputs(100, 4, 2, 64, 64)
    want = torch.empty_like(x["q"])
    assert call(x, want) == 0
    k_want = x["k_cache"].clone()
    got = torch.zeros_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    args = (x["q"], x["key"], x["value"], x["k_cache"], x["v_cache"], x["slots"], x["positions"], x["inv_freq"])
    x["k_cache"].zero_()
    s.wait_stream(torch.cuda.current_stream())
    ops.rope_append(got, *args, stream=s)
    s.synchronize()
    assert torch.equal(bits(got), bits(want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.rope_append(got, *args)
    for _ in range(2):
        got.zero_()
        x["k_cache"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(got), bits(want))
    blk, off = x["slots"] // 16, x["slots"] % 16
    assert torch.equal(bits(x["k_cache"][blk, :, off]), bits(k_want[blk, :, off]))


def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements per tensor (8 GiB each in bf16), written at its far end."""
    N, Hkv, D = (1 << 32) // (16 * 8 * 128) + 64, 8, 128
    x = inputs(40, 8, Hkv, D, D)
    small_k, small_v = x["k_cache"], x["v_cache"]
    assert call(x, torch.empty_like(x["q"])) == 0
    shift = (N - small_k.shape[0]) * 16
    big_k = torch.zeros(N, Hkv, 16, D, dtype=torch.bfloat16, device="cuda")
    big_v = torch.zeros_like(big_k)
    ops.rope_append(torch.empty_like(x["q"]), x["q"], x["key"], x["value"], big_k, big_v, x["slots"] + shift,
                    x["positions"], x["inv_freq"])
    blk, off = x["slots"] // 16, x["slots"] % 16
    far = blk + N - small_k.shape[0]
    assert torch.equal(bits(big_k[far, :, off]), bits(small_k[blk, :, off]))
    assert torch.equal(bits(big_v[far, :, off]), bits(small_v[blk, :, off]))
    assert not big_k[:64].any()
