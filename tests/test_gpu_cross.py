"""Cross attention over the paged cache (pa_cross_attention) against its definition in 64 bits.

Tolerance, element by element, with u = 2^-24 (fp32) and A = sum_i p_i |V_i| / sum_i p_i:

* A score is a dot product of D terms accumulated in fp32 (u a term, 2 u where a tensor core truncates) and scaled
  once: |dx| <= 2 (D + 2) u X with X = |scale| max_i sum_d |q_d K_id|.  The exponent's argument x - m is rounded twice
  more, at most 4 u X, and the exponential itself carries 4 u.  A weight's relative error is then at most
  e = 2 (D + 4) u X + 4 u, which the output sees twice (in the weights, and in their sum): 2 e A.
* n products are added up in fp32, and the weights beside them: 2 * 2 (n + 64) u A.
* bf16: a weight is rounded once for its product with V (at most half a step, 2^-8): 2^-8 A.
* The result is rounded once to the element type: half a step of its value.
"""
import math

import pytest
import torch

from paged_kv_cache_456_b200 import ops

from tests.test_gpu_rope import assert_turned, turned

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24
BLOCK = 16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_456_b200 import build
    build.build()
    ops.library()


class Case:
    """Sequences of ``rows`` rows and ``keys`` keys; slots that hold no key are NaN, table entries past the last block
    are not ids, ``before`` and ``behind`` rows belong to no sequence."""

    def __init__(self, rows, keys, *, dtype="bf16", hkv=2, G=4, D=128, seed=0, before=0, behind=0, std=1.5, spare=3,
                 tables_width=None):
        g = torch.Generator("cuda").manual_seed(seed + 977 * len(rows) + 31 * sum(rows) + sum(keys))
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.rows, self.keys, self.hkv, self.G, self.D, self.dt = rows, keys, hkv, G, D, DT[dtype]
        self.scale = 1 / math.sqrt(D)
        S, need = len(rows), [-(-n // BLOCK) for n in keys]
        N = sum(need) + spare
        order = torch.randperm(N, generator=g, device="cuda").int()
        self.tables = torch.full((S, tables_width or max(max(need), 1)), -7, dtype=torch.int32, device="cuda")
        self.tables[:, 1::2] = N + 100
        live = torch.zeros(N, BLOCK, dtype=torch.bool, device="cuda")
        at = 0
        for s, n in enumerate(need):
            self.tables[s, :n] = order[at:at + n]
            pos = torch.arange(keys[s], device="cuda")
            live[order[at:at + n].long()[pos // BLOCK], pos % BLOCK] = True
            at += n
        dead = ~live[:, None, :, None]
        self.k = rand(N, hkv, BLOCK, D).masked_fill_(dead, math.nan).to(self.dt)
        self.v = (rand(N, hkv, BLOCK, D) + 0.5).masked_fill_(dead, math.nan).to(self.dt)
        self.T = before + sum(rows) + behind
        self.q = (rand(self.T, hkv * G, D) * std).to(self.dt)
        self.starts = [before + sum(rows[:s]) for s in range(S + 1)]
        self.qs = torch.tensor(self.starts, dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(keys, dtype=torch.int32, device="cuda")
        self.max_keys = max(keys)

    def workspace(self):
        return ops.make_cross_attention_workspace(len(self.rows), self.T, self.hkv * self.G, self.hkv, self.D, self.max_keys,
                                                  dtype=self.dt)

    def call(self, out=None, ws=None, **kw):
        out = torch.full_like(self.q, 7.0) if out is None else out
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        ops.cross_attention(out, self.q, self.k, self.v, self.tables, self.lens, self.qs, scale=self.scale,
                            max_context_len=self.max_keys, workspace=self.workspace() if ws is None else ws, err_flag=err,
                            **kw)
        torch.cuda.synchronize()
        return out, int(err.item())

    def expected(self, s):
        """(definition, tolerance) of sequence s's rows, in 64 bits."""
        Q, n, G, D = self.rows[s], self.keys[s], self.G, self.D
        r0 = self.starts[s]
        if n == 0:
            z = torch.zeros(Q, self.hkv * G, D, dtype=torch.float64, device="cuda")
            return z, z
        ids = self.tables[s, :-(-n // BLOCK)].long()
        k, v = (x[ids].transpose(0, 1).reshape(self.hkv, -1, D)[:, :n].double() for x in (self.k, self.v))
        q = self.q[r0:r0 + Q].double().view(Q, self.hkv, G, D).permute(1, 2, 0, 3).reshape(self.hkv, G * Q, D)
        p = torch.softmax(self.scale * (q @ k.transpose(1, 2)), dim=-1)
        out, a = p @ v, p @ v.abs()
        x = abs(self.scale) * (q.abs() @ k.abs().transpose(1, 2)).amax(-1, keepdim=True)
        e = 2 * (D + 4) * U * x + 4 * U
        half = torch.finfo(self.dt).eps / 2
        tol = (2 * e + 4 * (n + 64) * U + (half if self.dt == torch.bfloat16 else 0)) * a
        tol = tol + half * (out.abs() + tol)
        back = lambda t: t.view(self.hkv, G, Q, D).permute(2, 0, 1, 3).reshape(Q, self.hkv * G, D)  # noqa: E731
        return back(out), back(tol)

    def check(self, out, skip=()):
        covered = torch.zeros(self.T, dtype=torch.bool, device="cuda")
        for s, Q in enumerate(self.rows):
            r0 = self.starts[s]
            covered[r0:r0 + Q] = True
            if Q == 0 or s in skip:
                continue
            want, tol = self.expected(s)
            err = (out[r0:r0 + Q].double() - want).abs()
            assert (err <= tol).all(), (f"sequence {s} ({Q} rows, {self.keys[s]} keys): worst error / tolerance "
                                        f"{(err / tol.clamp_min(1e-300)).nan_to_num(nan=math.inf).max():.3f}")
        assert (out[~covered] == 7.0).all(), "rows of no sequence were written"


SHAPES = [(dt, D, G) for dt in ("bf16", "f32") for D in (64, 128) for G in (1, 2, 4, 8)]
BATCHES = [((1,), (1,)), ((1, 1, 1, 1, 1), (1500, 7, 0, 16, 333)), ((5, 0, 17, 1, 64, 130), (33, 50, 0, 700, 128, 65)),
           ((300, 129), (1000, 257)), ((2,), (5000,)), ((700, 3), (3, 64)), ((33, 1, 32), (127, 129, 2049))]


@pytest.mark.parametrize("dtype,D,G", SHAPES, ids=str)
@pytest.mark.parametrize("rows,keys", BATCHES, ids=lambda x: "-".join(map(str, x)))
def test_matches_the_definition(dtype, D, G, rows, keys):
    c = Case(rows, keys, dtype=dtype, D=D, G=G, before=2, behind=3)
    out, err = c.call()
    assert err == 0
    c.check(out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hkv,G", [(1, 1), (16, 1), (3, 8), (8, 4)])
def test_head_layouts(dtype, hkv, G):
    for rows, keys in (((1, 1, 1), (100, 1000, 17)), ((40, 7), (300, 900))):
        c = Case(rows, keys, dtype=dtype, hkv=hkv, G=G, D=64)
        out, err = c.call()
        assert err == 0
        c.check(out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257])
def test_lengths_around_the_tiles(dtype, n):
    for rows in ((1,), (9,), (70,)):
        c = Case(rows, (n,), dtype=dtype, G=2)
        out, err = c.call()
        assert err == 0
        c.check(out)


@pytest.mark.parametrize("Q", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257])
def test_rows_around_the_tiles(Q):
    for dtype in ("bf16", "f32"):
        c = Case((Q, 1), (77, 300), dtype=dtype, hkv=1, G=1, D=64)
        out, err = c.call()
        assert err == 0
        c.check(out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [(1, 1), (40, 2), (200, 150)])
@pytest.mark.parametrize("scale", [-0.125, 0.0, 3.0])
def test_scales(dtype, rows, scale):
    c = Case(rows, (150, 700), dtype=dtype, std=0.5)
    c.scale = scale
    out, err = c.call()
    assert err == 0
    c.check(out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [(1, 1), (40, 2), (200, 150)])
def test_scores_that_grow_along_the_keys(dtype, rows):
    """The running maximum grows by more than any threshold from tile to tile."""
    c = Case(rows, (900, 500), dtype=dtype, D=64)
    c.q[:] = c.q.abs()
    for s, n in enumerate(c.keys):
        pos = torch.arange(n, device="cuda")
        ids = c.tables[s].long()[pos // BLOCK]
        c.k[ids, :, pos % BLOCK] = (c.k[ids, :, pos % BLOCK].float().abs() * (pos[:, None, None] / 60)).to(c.dt)
    out, err = c.call()
    assert err == 0
    c.check(out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 3, 20, 40, 200, 300])
def test_one_item_over_every_worker(dtype, rows):
    """One KV head's keys cut into as many pieces as there are workers, of one sequence or beside short ones."""
    for keys in ((40000,), (3, 30001, 17)):
        c = Case((rows,) * len(keys), keys, dtype=dtype, hkv=1, G=1, D=64)
        ws = c.workspace()
        for _ in range(2):
            out, err = c.call(ws=ws)
            assert err == 0
            c.check(out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [(1, 2, 1), (90, 300, 2)])
def test_infinite_scores(dtype, rows):
    """Keys whose scores are -inf weigh nothing; rows that see nothing else are NaN, as the softmax is."""
    c = Case(rows, (300, 700, 40), dtype=dtype, hkv=1, G=2, D=64)
    c.q[:] = c.q.abs() + 0.1
    pos = torch.arange(0, 700, 3, device="cuda")
    c.k[c.tables[1].long()[pos // BLOCK], 0, pos % BLOCK, 5] = -math.inf
    pos = torch.arange(40, device="cuda")
    c.k[c.tables[2].long()[pos // BLOCK], 0, pos % BLOCK, 5] = -math.inf
    out, err = c.call()
    assert err == 0
    assert out[c.starts[2]:c.starts[3]].isnan().all()
    c.check(out, skip=(1, 2))
    ids = c.tables[1, :44].long()
    k, v = (x[ids, 0].reshape(-1, 64)[:700].double() for x in (c.k, c.v))
    seen = torch.ones(700, dtype=torch.bool, device="cuda")
    seen[::3] = False
    q = c.q[c.starts[1]:c.starts[2]].double()
    p = torch.softmax(c.scale * (q @ k[seen].t()), dim=-1)
    want, a = p @ v[seen], p @ v[seen].abs()
    x = c.scale * (q.abs() @ k[seen].abs().t()).amax(-1, keepdim=True)
    half = torch.finfo(c.dt).eps / 2
    tol = (2 * (2 * 68 * U * x + 4 * U) + 4 * 764 * U + (half if dtype == "bf16" else 0)) * a
    assert ((out[c.starts[1]:c.starts[2]].double() - want).abs() <= tol + half * (want.abs() + tol)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_batch_of_many_sequences(dtype):
    """More sequences than the plan keeps on chip, one row or none each, most of them without keys or short."""
    g = torch.Generator().manual_seed(5)
    S = 4200
    rows = tuple(int(x) for x in torch.randint(0, 2, (S,), generator=g))
    keys = tuple(int(x) for x in torch.randint(0, 40, (S,), generator=g))
    c = Case(rows, keys, dtype=dtype, hkv=1, G=2, D=64, behind=4)
    out, err = c.call()
    assert err == 0
    some = set(torch.randint(0, S, (300,), generator=g).tolist())
    c.check(out, skip=set(range(S)) - some)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [(1, 1, 1), (5, 9, 3), (300, 200, 64)])
def test_repeated_calls_are_bit_identical(dtype, rows):
    c = Case(rows, (900, 1700, 64), dtype=dtype)
    ws = c.workspace()
    first, _ = c.call(ws=ws)
    for _ in range(3):
        again, err = c.call(ws=ws)
        assert err == 0 and torch.equal(first.view(torch.uint8), again.view(torch.uint8))


def test_one_workspace_for_different_calls():
    cases = [Case(r, k, hkv=4) for r, k in (((300, 900), (500, 20)), ((1, 1), (4000, 3)), ((64,) * 9, (100,) * 9))]
    ws = max((c.workspace() for c in cases), key=lambda w: w.numel())
    for c in cases * 2:
        out, err = c.call(ws=ws)
        assert err == 0
        c.check(out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [(1, 1, 1), (20, 30, 10), (400, 300, 100)])
def test_bad_blocks_and_lengths_zero_their_sequence_only(dtype, rows):
    for what, bit in (("id", ops.ERRBIT_BLOCK_ID), ("negative id", ops.ERRBIT_BLOCK_ID),
                      ("length", ops.ERRBIT_CONTEXT_LEN), ("negative length", ops.ERRBIT_CONTEXT_LEN)):
        c = Case(rows, (200, 1500, 90), dtype=dtype, before=1, behind=1, tables_width=130)
        if "id" in what:
            c.tables[1, 87] = -1 if "negative" in what else c.k.shape[0]
        else:
            c.lens[1] = -1 if "negative" in what else 1501
        out, err = c.call()
        assert err == bit, what
        assert (out[c.starts[1]:c.starts[2]] == 0).all()
        c.check(out, skip=(1,))


def test_a_sequence_without_rows_is_not_checked():
    c = Case((4, 0, 6), (50, 80, 70))
    c.tables[1, 2] = 1 << 20
    c.lens[1] = -5
    out, err = c.call()
    assert err == 0
    c.check(out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_out_of_order(dtype):
    c = Case((5, 7, 4), (60, 70, 80), dtype=dtype)
    for bad in ([0, 5, 3, 16], [0, 5, 17, 20], [-1, 5, 12, 16]):
        c.qs.copy_(torch.tensor(bad, dtype=torch.int32))
        out, err = c.call()
        assert err == ops.ERRBIT_QUERY
        if bad[:2] == [0, 5]:
            want, tol = c.expected(0)
            assert ((out[:3].double() - want[:3]).abs() <= tol[:3]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [(1, 1), (64, 40)])
def test_a_nan_stays_in_its_head(dtype, rows):
    c = Case(rows, (300, 100), dtype=dtype, hkv=2, G=2, D=64)
    ref, _ = c.call()
    c.v[c.tables[0, 3].long(), 1, 5, 10] = math.nan
    out, err = c.call()
    assert err == 0
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[:rows[0], 2:, 10] = True
    assert out[hit].isnan().all()
    assert torch.equal(out[~hit], ref[~hit])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [(1, 1, 1), (30, 50, 1)])
def test_on_another_stream_and_in_a_graph(dtype, rows):
    """Captured once, replayed with other queries, lengths and tables; two graphs share the workspace."""
    a, b = (Case(rows, (300, 100, 700), dtype=dtype, seed=s) for s in (1, 2))
    ws, outs = a.workspace(), [torch.full_like(a.q, 7.0), torch.full_like(b.q, 7.0)]
    a.call(), b.call()
    stream = torch.cuda.Stream()
    graphs = []
    for c, out in zip((a, b), outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            ops.cross_attention(out, c.q, c.k, c.v, c.tables, c.lens, c.qs, scale=c.scale, max_context_len=c.max_keys,
                                workspace=ws)
        graphs.append(graph)
    for _ in range(2):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    a.check(outs[0])
    b.check(outs[1])
    a.keys = (300, 0, 650)
    a.lens.copy_(torch.tensor(a.keys))
    a.q.neg_()
    graphs[0].replay()
    torch.cuda.synchronize()
    a.check(outs[0])


def test_no_rows_and_no_keys():
    c = Case((0, 0), (30, 20))
    out, err = c.call()
    assert err == 0 and out.shape[0] == 0
    c = Case((3, 0), (0, 0), behind=2)
    out, err = c.call()
    assert err == 0
    c.check(out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [(1,), (70,)])
def test_offsets_past_32_bits(dtype, rows):
    """A cache of more than 2^32 bytes, the blocks attended to at its end."""
    c = Case(rows, (100,), dtype=dtype, hkv=8, G=1, D=128)
    N = (1 << 32) // (8 * BLOCK * 128 * c.dt.itemsize) + 50
    k, v = (torch.empty(N, 8, BLOCK, 128, dtype=c.dt, device="cuda") for _ in range(2))
    ids = c.tables[0, :7].long()
    k[N - 7:], v[N - 7:] = c.k[ids], c.v[ids]
    c.k, c.v = k, v
    c.tables[0, :7] = torch.arange(N - 7, N, device="cuda").int()
    out, err = c.call()
    assert err == 0
    c.check(out)


def test_the_binding_refuses_on_the_device():
    c = Case((4,), (40,))
    ws = c.workspace()
    with pytest.raises(ops.PagedAttentionError) as e:
        c.call(ws=ws[:ws.numel() - 512])
    assert e.value.status == ops.PA_ERR_WORKSPACE
    with pytest.raises(ops.PagedAttentionError):
        c.call(ws=ws[8:])


def wrong(t):
    """The tensor as the binding must not take it: on the host, of another type, shape or layout."""
    other = {torch.bfloat16: torch.float32, torch.float32: torch.float64, torch.int32: torch.int64,
             torch.int64: torch.int32, torch.uint8: torch.uint8}[t.dtype]
    yield t.cpu()
    if other is not t.dtype:
        yield t.to(other)
        yield t[None]
        yield t[:0] if t.shape[0] else t
    yield torch.stack((t, t), dim=-1)[..., 0] if t.numel() > 1 else t.cpu()


@pytest.mark.parametrize("name", ["out", "q", "k", "v", "tables", "lens", "qs", "ws", "err"])
def test_the_binding_refuses_each_tensor(name):
    c = Case((4, 2), (40, 50), G=2, D=64)
    good = dict(out=torch.empty_like(c.q), q=c.q, k=c.k, v=c.v, tables=c.tables, lens=c.lens, qs=c.qs, ws=c.workspace(),
                err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    for bad in wrong(good[name]):
        if name == "err" and bad.is_cuda and bad.dtype is torch.int32 and bad.numel():
            continue  # (an error word of any shape will do)
        x = dict(good, **{name: bad})
        with pytest.raises((ValueError, TypeError)):
            ops.cross_attention(x["out"], x["q"], x["k"], x["v"], x["tables"], x["lens"], x["qs"], scale=1.0,
                                max_context_len=50, workspace=x["ws"], err_flag=x["err"])


@pytest.mark.parametrize("name", ["q_out", "q", "key", "value", "k", "v", "slots", "pos", "freq", "axis", "err"])
def test_the_rotary_binding_refuses_each_tensor(name):
    T, dev = 6, "cuda"
    r = lambda *s: torch.randn(*s, device=dev).bfloat16()  # noqa: E731
    good = dict(q_out=r(T, 4, 64), q=r(T, 4, 64), key=r(T, 2, 64), value=r(T, 2, 64), k=r(3, 2, 16, 64), v=r(3, 2, 16, 64),
                slots=torch.arange(T, device=dev), pos=torch.arange(2 * T, device=dev).view(2, T),
                freq=torch.ones(32, device=dev), axis=torch.zeros(32, dtype=torch.int32, device=dev),
                err=torch.zeros(1, dtype=torch.int32, device=dev))
    for bad in wrong(good[name]):
        if name == "err" and bad.is_cuda and bad.dtype is torch.int32 and bad.numel():
            continue
        x = dict(good, **{name: bad})
        with pytest.raises((ValueError, TypeError, ops.PagedAttentionError)):
            ops.rope_append(x["q_out"], x["q"], x["key"], x["value"], x["k"], x["v"], x["slots"], x["pos"], x["freq"],
                            pair_axis=x["axis"], err_flag=x["err"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_run_of_the_operators_together(dtype):
    """Encoder states written once with their rotary positions, then prompts of several rows and generated rows that
    attend to them, each rotated on the way."""
    rows, keys, hkv, G, D = (6, 11, 1), (200, 35, 500), 2, 4, 64
    c = Case(rows, keys, dtype=dtype, hkv=hkv, G=G, D=D)
    dev, n = "cuda", sum(keys)
    freq = (100.0 ** (-torch.arange(16).double() / 16)).float().to(dev)
    gen = torch.Generator(dev).manual_seed(3)
    states = torch.randn(n, 2 * hkv * D, generator=gen, device=dev).to(c.dt)
    key, value = (x.view(n, hkv, D) for x in states.split(hkv * D, dim=1))
    pos = torch.cat([torch.arange(m, device=dev) for m in keys])
    slots = torch.cat([c.tables[s].long()[torch.arange(m, device=dev) // BLOCK] * BLOCK
                       + torch.arange(m, device=dev) % BLOCK for s, m in enumerate(keys)])
    ops.rope_append(None, None, key, value, c.k, c.v, slots, pos, freq)
    ws = c.workspace()
    for step in range(3):  # a prompt, then two generated rows of each sequence
        if step:
            c.rows = (1, 1, 1)
            c.starts = [0, 1, 2, 3]
            c.T = 3
            c.qs = torch.tensor(c.starts, dtype=torch.int32, device=dev)
        x = torch.randn(c.T, hkv * G, D, generator=gen, device=dev).to(c.dt)
        at = torch.cat([torch.arange(r, device=dev) for r in c.rows]) + 7 * step
        c.q = torch.empty_like(x)
        ops.rope_append(c.q, x, None, None, None, None, None, at, freq)
        # (a cos - b sin may cancel, so the rotation's fp32 error follows |a| + |b|, 4e-7 of it by the count in
        # test_gpu_rope, and not the result: the helper there allows that and the last rounding)
        assert_turned(c.q, *turned(x, at, freq, None, False, 1.0))
        out, err = c.call(ws=ws if step == 0 else None)
        assert err == 0
        c.check(out)
