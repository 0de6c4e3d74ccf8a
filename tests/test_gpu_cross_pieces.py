"""pa_cross_attention where a CTA's share holds several pieces: what one piece leaves in shared memory, in the counters
or in the workspace must not reach another.  Tolerances as in test_gpu_cross, whose 64-bit definition this uses."""
import pytest
import torch

from paged_kv_cache_456_b200 import ops

from tests.test_gpu_cross import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_456_b200 import build
    build.build()
    ops.library()


def beside_a_load(c, repeats):
    """The outputs of ``repeats`` calls while another stream keeps part of the SMs busy, so that CTAs start late and
    unevenly."""
    ws = c.workspace()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [torch.full_like(c.q, 7.0) for _ in range(repeats)]
    x = torch.randn(1024, 1024, device="cuda")
    y = torch.empty_like(x)
    load = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        with torch.cuda.stream(load):
            for n in range(1 + i % 3):
                torch.matmul(x[:256 * (1 + (i + n) % 4)], x, out=y[:256 * (1 + (i + n) % 4)])
        ops.cross_attention(out, c.q, c.k, c.v, c.tables, c.lens, c.qs, scale=c.scale, max_context_len=c.max_keys,
                            workspace=ws, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return outs


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,long_rows,short_rows", [(2, 9, 3), (2, 5, 4), (1, 10, 8), (2, 1, 1), (4, 1, 3), (1, 1, 1)])
@pytest.mark.parametrize("pairs,keys", [(20, 2000), (30, 9000), (4, 60000), (60, 1100)])
def test_few_columns_a_merge_and_then_a_short_piece(D, G, long_rows, short_rows, pairs, keys):
    """Items cut into 2 to 31 pieces, some of them of two columns, each followed by sequences of 1 to 128 keys, whose
    pieces begin while slower warps may still be merging: up to 16 columns a (sequence, KV head) on average."""
    rows, lens = [], []
    for i in range(pairs):
        rows += [long_rows, short_rows]
        lens += [keys - 7 * i, (1, 16, 17, 100, 128)[i % 5]]
    c = Case(tuple(rows), tuple(lens), hkv=2, G=G, D=D, behind=1)
    outs = beside_a_load(c, 12)
    c.check(outs[0])
    for out in outs[1:]:
        assert torch.equal(out.view(torch.int16), outs[0].view(torch.int16))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,rows", [(1, 40), (4, 40), (8, 100)])
@pytest.mark.parametrize("seqs,keys", [(90, 200), (100, 300), (37, 1000), (8, 5000), (200, 129)])
def test_many_columns_a_cut_item_and_then_a_piece_of_one_tile(D, G, rows, seqs, keys):
    """More than 32 columns: shares of one to a few tiles of 128 keys, so that a cut item's end is followed at once by
    the first tile of the next cut item."""
    c = Case(tuple(rows - i % 7 for i in range(seqs)), tuple(keys - i % 3 * 64 for i in range(seqs)), hkv=2, G=G, D=D)
    outs = beside_a_load(c, 12)
    c.check(outs[0])
    for out in outs[1:]:
        assert torch.equal(out.view(torch.int16), outs[0].view(torch.int16))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,G,rows", [(128, 4, 256), (64, 1, 64), (64, 8, 8), (128, 1, 33)])
def test_a_workspace_for_the_largest_batch_does_for_what_is_left_of_it(dtype, D, G, rows):
    """Sized once for many sequences, used as sequences leave and the same rows, or fewer, fall to fewer sequences."""
    ws = ops.make_cross_attention_workspace(64, rows, 2 * G, 2, D, 500, dtype=torch.bfloat16 if dtype == "bf16"
                                            else torch.float32)
    for seqs in (64, 17, 8, 4, 2, 1):
        for part in (1, 3):
            share = [max(rows // part // seqs, 1)] * min(seqs, rows // part)
            c = Case(tuple(share), tuple(500 - 5 * i for i in range(len(share))), dtype=dtype, hkv=2, G=G, D=D)
            assert c.T <= rows
            out, err = c.call(ws=ws)
            assert err == 0
            c.check(out)


def repeated(rows, keys, heads, D, dtype, period=64):
    """Sequences whose tables list ``period`` blocks over and over, one query head a KV head: a few cached tokens stand
    for contexts of millions."""
    c = Case(rows, (period * 16,) * len(rows), dtype=dtype, hkv=heads, G=1, D=D)
    c.tables = c.tables[:, torch.arange(-(-max(keys) // 16), device="cuda") % period].contiguous()
    c.lens.copy_(torch.tensor(keys, dtype=torch.int32))
    c.max_keys = max(keys)
    return c


def test_a_column_tile_left_out_for_longer_than_one_wait_may_last():
    """Eight sequences of 2^24 keys and 40 rows occupy every CTA for 1.4 s, in which the second column tile has nothing
    to do; then come items of 200 rows.  (The limit of a wait for one tile's work is 1 s.)"""
    period = 64
    c = repeated((40,) * 8 + (200,), (1 << 24,) * 8 + (300,), 148, 64, "bf16", period)
    out, err = c.call()
    assert err == 0
    assert torch.isfinite(out.float()).all()
    c.keys = (period * 16,) * 8 + (300,)
    c.check(out, skip=range(8))


@pytest.mark.parametrize("dtype,rows", [("bf16", 1), ("bf16", 12), ("bf16", 40), ("f32", 1), ("f32", 40)])
def test_a_million_keys_of_one_item_on_one_cta(dtype, rows):
    """2^20 keys a KV head, as many KV heads as CTAs that hold them.  Beside the tolerance of the period's own sums (the
    weights and their products repeat exactly), n keys are added up: fp32 n 2^-24 of A in the products and as much in
    the weights; bf16 one truncation of at most 2^-23 for every 16 keys in the products, and sums of at least 16
    weights rounded to nearest (2^-24) in the weights."""
    n, period = 1 << 20, 64
    c = repeated((rows,), (n,), 148, 64, dtype, period)
    out, err = c.call()
    assert err == 0
    c.keys = (period * 16,)
    want, tol = c.expected(0)
    ids = c.tables[0, :period].long()
    k, v = (x[ids].transpose(0, 1).reshape(148, -1, 64).double() for x in (c.k, c.v))
    p = torch.softmax(c.scale * (c.q.double().transpose(0, 1) @ k.transpose(1, 2)), dim=-1)
    a = (p @ v.abs()).transpose(0, 1)
    sums = n * 2.0 ** -23 if dtype == "f32" else n / 16 * (2.0 ** -23 + 2.0 ** -24)
    bound = tol + sums * a * (1 + torch.finfo(c.dt).eps / 2)
    worst = ((out.double() - want).abs() / bound).max()
    assert worst <= 1, f"worst error / tolerance {worst:.3f}"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seqs,T", [(64, 300), (130, 300), (40, 9), (40, 900), (2000, 40)])
def test_query_starts_that_go_back_and_forth_are_refused(dtype, seqs, T):
    """0, T, 0, T, ...: every other pair is in order and covers all rows.  The call must not do their work over."""
    c = Case((1,) * seqs, (100,) * seqs, dtype=dtype, hkv=1, G=4, D=64)
    c.T = T
    c.q = torch.randn(T, 4, 64, device="cuda").to(c.dt)
    c.qs.copy_(torch.tensor([T * (s % 2) for s in range(seqs + 1)], dtype=torch.int32))
    ws = c.workspace()
    out, err = c.call(ws=ws)
    assert err == ops.ERRBIT_QUERY
    assert (out == 7.0).all()
    # and the workspace is ready for a call that is in order
    d = Case((T // 2, T - T // 2), (900, 70), dtype=dtype, hkv=1, G=4, D=64)
    out, err = d.call(ws=ws)
    assert err == 0
    d.check(out)


def poisoned(ws):
    """A workspace as it must be before its first use where it is read without having been written: the counters zero
    (the first 16 KB), all else NaN."""
    ws[16384:] = 255
    return ws


@pytest.mark.parametrize("dtype,rows", [("bf16", 2), ("bf16", 6), ("bf16", 28), ("f32", 2), ("f32", 28)])
@pytest.mark.parametrize("seqs", [31, 33, 64, 127, 128, 129, 600])
def test_numbers_of_sequences(dtype, rows, seqs):
    """Up to 32 sequences every lane of a warp lays one out, up to 128 several, above the whole CTA: on each kernel (8,
    24 and 112 columns a sequence at most), some sequences without rows and some without keys."""
    g = torch.Generator().manual_seed(seqs + rows)
    r = [int(x) for x in torch.randint(rows - rows // 4, rows + 1, (seqs,), generator=g)]
    n = [int(x) for x in torch.randint(1, 260, (seqs,), generator=g)]
    for i in range(0, seqs, 9):
        r[i] = 0
    for i in range(4, seqs, 11):
        n[i] = 0
    r[-1], n[-1], n[seqs // 2] = rows, 700, 3000
    c = Case(tuple(r), tuple(n), dtype=dtype, hkv=2, G=4, D=64, before=1, behind=2)
    ws = poisoned(c.workspace())
    outs = [c.call(ws=ws) for _ in range(2)]
    assert [err for _, err in outs] == [0, 0]
    c.check(outs[0][0])
    assert torch.equal(outs[0][0].view(torch.uint8), outs[1][0].view(torch.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,G", [(64, 1), (64, 4), (128, 2), (128, 8)])
@pytest.mark.parametrize("rows", [1, 3, 7, 12, 40, 150])
@pytest.mark.parametrize("keys", [(40000,), (5000, 60, 2500)])
def test_no_partial_is_read_that_was_not_stored(dtype, D, G, rows, keys):
    """Cut items over a workspace that is NaN but for its counters."""
    c = Case((rows,) * len(keys), keys, dtype=dtype, hkv=2, G=G, D=D)
    out, err = c.call(ws=poisoned(c.workspace()))
    assert err == 0
    c.check(out)


@pytest.mark.parametrize("first,second", [(("bf16", 1), ("bf16", 60)), (("bf16", 60), ("f32", 30)), (("f32", 1), ("bf16", 3)),
                                          (("bf16", 60), ("bf16", 60))])
def test_two_calls_at_once(first, second):
    """On two streams, each with a workspace of its own."""
    cases = [Case((rows,) * 5, (3000, 200, 17, 1111, 640), dtype=dtype, G=2, D=64, seed=i)
             for i, (dtype, rows) in enumerate((first, second))]
    alone = [c.call()[0] for c in cases]
    streams, spaces = [torch.cuda.Stream() for _ in cases], [c.workspace() for c in cases]
    outs = [[torch.full_like(c.q, 7.0) for _ in range(10)] for c in cases]
    torch.cuda.synchronize()
    for i in range(10):
        for c, s, ws, out in zip(cases, streams, spaces, outs):
            ops.cross_attention(out[i], c.q, c.k, c.v, c.tables, c.lens, c.qs, scale=c.scale, max_context_len=c.max_keys,
                                workspace=ws, stream=s)
    torch.cuda.synchronize()
    for c, want, out in zip(cases, alone, outs):
        c.check(want)
        for o in out:
            assert torch.equal(o.view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [(1, 2), (9, 4)])
def test_thousands_of_heads(dtype, D, rows):
    c = Case(rows, (40, 21), dtype=dtype, hkv=2050, G=8, D=D, behind=1)
    out, err = c.call()
    assert err == 0
    c.check(out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 12, 90])
@pytest.mark.parametrize("at", [0, 700, 2499])
def test_one_bad_block_poisons_every_piece_of_its_sequence(dtype, rows, at):
    """A bad id in the first, a middle or the last piece of cut items: the sequence's rows are zeros, the others' right."""
    c = Case((rows, rows, 3), (300, 40000, 129), dtype=dtype, hkv=2, G=2, D=64)
    ws = poisoned(c.workspace())
    good = int(c.tables[1, at])
    for bad in (c.k.shape[0], -1, good):
        c.tables[1, at] = bad
        out, err = c.call(ws=ws)
        if bad == good:
            assert err == 0
            c.check(out)
        else:
            assert err == ops.ERRBIT_BLOCK_ID
            assert (out[c.starts[1]:c.starts[2]] == 0).all()
            c.check(out, skip=(1,))
