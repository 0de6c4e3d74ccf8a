"""The cases on which the rotary append and the cross attention of the paged cache are measured.

``run`` makes one pass through an operator: in its plain form (elementary torch operations, 32 bits) or, where
``own`` is true, through the library's entry points.  Lengths of a ragged batch are a fixed function of the case;
values, block tables and slots come from the seed.
"""
import math
import random

import torch

own = False

BLOCK = 16
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one generated token of one sequence: pure latency
        _rope("rope one token", tokens=1, hq=32, hkv=8, d=128, rot=128),
        # a decode step of 64 sequences, as many KV heads as query heads
        _rope("rope decode 64", tokens=64, hq=32, hkv=32, d=128, rot=128),
        # a chunk of prompts, 8 query heads a KV head, q/k/v views of one fused projection
        _rope("rope chunk 2048", tokens=2048, hq=64, hkv=8, d=128, rot=128, fused=True),
        # image and video tokens: three position axes (time, height, width), padding at the end
        _rope("rope video 16384", tokens=16384, hq=32, hkv=8, d=128, rot=128, axes=3, padding=96),
        # fp32, half of each head rotated, adjacent pairs, an odd number of tokens far into their sequences
        _rope("rope f32 far 1023", tokens=1023, hq=12, hkv=4, d=64, rot=32, dtype="f32", adjacent=True, far=1 << 20),
        # one generated token of one sequence against 1500 encoder states: latency
        _cross("cross one row", seqs=1, rows=1, keys=1500, hq=16, hkv=16, d=64),
        # a decode step of 64 sequences, each against its own encoder states
        _cross("cross decode 64", seqs=64, rows=1, keys=1500, hq=16, hkv=16, d=64),
        # 5 candidates of each of two sequences against long documents: few rows, a long axis
        _cross("cross long 5x2", seqs=2, rows=5, keys=32768, hq=32, hkv=8, d=128),
        # ragged prompts against ragged encoder states, some of them empty
        _cross("cross ragged 16", seqs=16, rows=333, keys=1100, hq=32, hkv=8, d=128, ragged=True),
        # whole images: many rows against many states
        _cross("cross full 4x4096", seqs=4, rows=4096, keys=4096, hq=32, hkv=8, d=128),
        # fp32, ragged, two query heads a KV head
        _cross("cross f32 ragged 6", seqs=6, rows=150, keys=700, hq=8, hkv=4, d=64, dtype="f32", ragged=True),
    ]


def _rope(name=None, *, tokens, hq, hkv, d, rot, axes=1, dtype="bf16", adjacent=False, fused=False, padding=0, far=4096):
    c = dict(op="rope_append", tokens=tokens, hq=hq, hkv=hkv, d=d, rot=rot, axes=axes, dtype=dtype, adjacent=adjacent,
             fused=fused, padding=padding, far=far)
    return dict(c, name=name) if name else c


def _cross(name=None, *, seqs, rows, keys, hq, hkv, d, dtype="bf16", ragged=False):
    c = dict(op="cross_attention", seqs=seqs, rows=rows, keys=keys, hq=hq, hkv=hkv, d=d, dtype=dtype, ragged=ragged)
    return dict(c, name=name) if name else c


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    dtype = rng.choice(("bf16", "bf16", "f32"))
    d = rng.choice((64, 128))
    hkv = rng.choice((1, 2, 4, 8, 16))
    group = rng.choice((1, 2, 4, 8))
    if rng.random() < 0.5:
        tokens = _log_int(rng, 1, 16384)
        return _rope(tokens=tokens, hq=min(64, hkv * rng.choice((1, 2, 3, 4, 5, 8))) // hkv * hkv, hkv=hkv, d=d,
                     rot=rng.choice((d, d, d // 2, d // 4)), axes=rng.choice((1, 1, 2, 3)), dtype=dtype,
                     adjacent=rng.random() < 0.4, fused=rng.random() < 0.4, padding=rng.randrange(tokens // 8 + 1),
                     far=rng.choice((4096, 131072, 1 << 22)))
    while True:
        seqs, rows, keys = _log_int(rng, 1, 64), _log_int(rng, 1, 4096), _log_int(rng, 1, 32768)
        hq = hkv * group
        # no dearer than the largest listed case, and the plain form's scores fit the card three times over
        scores = seqs * rows * keys * hq
        if scores <= (1 << 31 if dtype == "bf16" else 1 << 28) and seqs * keys * hkv * d <= 1 << 27:
            return _cross(seqs=seqs, rows=rows, keys=keys, hq=hq, hkv=hkv, d=d, dtype=dtype, ragged=rng.random() < 0.5)


def _lengths(case):
    """(rows, keys) of each sequence: all alike, or spread between an eighth of the largest and the largest, with one
    sequence of no rows and one of no keys where the batch has four or more."""
    S, Q, N = case["seqs"], case["rows"], case["keys"]
    if not case["ragged"]:
        return [Q] * S, [N] * S
    r = random.Random("%d %d %d" % (S, Q, N))
    rows = [max(1, round(Q * r.uniform(0.125, 1.0))) for _ in range(S)]
    keys = [max(1, round(N * r.uniform(0.125, 1.0))) for _ in range(S)]
    if S >= 4:
        rows[1], keys[2] = 0, 0
    return rows, keys


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return (_prepare_rope if case["op"] == "rope_append" else _prepare_cross)(case, g)


def _normal(g, *shape, dtype, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _prepare_rope(c, g):
    T, Hq, Hkv, D, dt = c["tokens"], c["hq"], c["hkv"], c["d"], DTYPES[c["dtype"]]
    if c["fused"]:  # the rows of one projection's output
        qkv = _normal(g, T, (Hq + 2 * Hkv) * D, dtype=dt)
        q, k, v = (x.view(T, -1, D) for x in qkv.split((Hq * D, Hkv * D, Hkv * D), dim=1))
    else:
        q, k, v = (_normal(g, T, h, D, dtype=dt) for h in (Hq, Hkv, Hkv))
    # block 0 belongs to no sequence; the tokens' slots are scattered over whole blocks of the pool, in order inside a block
    used = -(-T // BLOCK)
    N = used + max(4, used // 4)
    blocks = 1 + torch.randperm(N - 1, generator=g, device="cuda")[:used]
    slots = (blocks[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")).reshape(-1)[:T].contiguous()
    if c["padding"]:
        slots[T - c["padding"]:] = -1
    # positions: runs of consecutive tokens, each run from a place of its own; other axes: a grid's rows and columns
    run = 256
    start = torch.randint(0, c["far"], (-(-T // run),), generator=g, device="cuda")
    t = torch.arange(T, device="cuda")
    pos = [start[t // run] + t % run, start[t // run] + t % run // 16, start[t // run] + t % 16]
    positions = torch.stack(pos[:c["axes"]]).contiguous()
    half = c["rot"] // 2
    inv_freq = (10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)).float()
    # the pairs go to the axes in contiguous sections: a quarter to the first, the others alike
    pair_axis = None
    if c["axes"] > 1:
        first = half // 4
        rest = torch.arange(half - first, device="cuda") * (c["axes"] - 1) // (half - first)
        pair_axis = torch.cat([torch.zeros(first, dtype=torch.int64, device="cuda"), 1 + rest]).int()
    return dict(case=c, q=q, key=k, value=v, slots=slots, positions=positions, inv_freq=inv_freq, pair_axis=pair_axis,
                q_out=torch.empty(T, Hq, D, dtype=dt, device="cuda"),
                k_cache=_normal(g, N, Hkv, BLOCK, D, dtype=dt), v_cache=_normal(g, N, Hkv, BLOCK, D, dtype=dt))


def _prepare_cross(c, g):
    rows, keys = _lengths(c)
    S, Hq, Hkv, D, dt = c["seqs"], c["hq"], c["hkv"], c["d"], DTYPES[c["dtype"]]
    T = sum(rows)
    need = [-(-n // BLOCK) for n in keys]
    N = sum(need) + max(4, sum(need) // 8)
    order = torch.randperm(N, generator=g, device="cuda").int()
    tables = torch.full((S, max(max(need), 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = order[at:at + n]
        at += n
    k_cache = _normal(g, N, Hkv, BLOCK, D, dtype=dt)
    # values have a mean of their own in each channel, as projections of encoder states have
    v_cache = (torch.randn(N, Hkv, BLOCK, D, generator=g, device="cuda")
               + 0.5 * torch.randn(Hkv, 1, D, generator=g, device="cuda")).to(dt)
    starts = [sum(rows[:s]) for s in range(S + 1)]
    state = dict(case=c, q=_normal(g, T, Hq, D, dtype=dt, std=1.5), k_cache=k_cache, v_cache=v_cache, tables=tables,
                 lens=torch.tensor(keys, dtype=torch.int32, device="cuda"),
                 starts=torch.tensor(starts, dtype=torch.int32, device="cuda"),
                 out=torch.empty(T, Hq, D, dtype=dt, device="cuda"), scale=1.0 / math.sqrt(D),
                 max_rows=max(rows), max_keys=max(keys), workspace=None)
    if own:
        from paged_kv_cache_456_b200 import ops
        state["workspace"] = ops.make_cross_attention_workspace(S, T, Hq, Hkv, D, max(keys), dtype=dt)
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    return (_plain_rope if state["case"]["op"] == "rope_append" else _plain_cross)(state)


def _run_own(s):
    from paged_kv_cache_456_b200 import ops
    c = s["case"]
    if c["op"] == "rope_append":
        ops.rope_append(s["q_out"], s["q"], s["key"], s["value"], s["k_cache"], s["v_cache"], s["slots"], s["positions"],
                        s["inv_freq"], pair_axis=s["pair_axis"], adjacent=c["adjacent"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    ops.cross_attention(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["starts"], scale=s["scale"],
                        max_context_len=s["max_keys"], workspace=s["workspace"])
    return s["out"]


def _rotate(x, cos, sin, rot, adjacent):
    """x [T][H][D] in 32 bits; cos, sin [T][1][rot / 2]."""
    if adjacent:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((turned, x[..., rot:]), dim=-1)


def _plain_rope(s):
    c = s["case"]
    pos = s["positions"].double()  # far positions: the angle needs more than 32 bits
    pos = pos[0][:, None] if s["pair_axis"] is None else pos[s["pair_axis"].long()].t()
    angle = pos * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    dt = s["q"].dtype
    q_out = _rotate(s["q"].float(), cos, sin, c["rot"], c["adjacent"]).to(dt)
    k = _rotate(s["key"].float(), cos, sin, c["rot"], c["adjacent"]).to(dt)
    # a padding token puts back what block 0 holds
    live = (s["slots"] >= 0)[:, None, None]
    slot = s["slots"].clamp_min(0)
    block, off = slot // BLOCK, slot % BLOCK
    for cache, new in ((s["k_cache"], k), (s["v_cache"], s["value"])):
        cache[block, :, off] = torch.where(live, new, cache[block, :, off])
    return q_out, s["k_cache"], s["v_cache"]


def _plain_cross(s):
    c = s["case"]
    S, Q, N, Hq, Hkv, D = c["seqs"], s["max_rows"], s["max_keys"], c["hq"], c["hkv"], c["d"]
    T = s["q"].shape[0]
    # the sequences' states side by side, padded to the longest
    blocks = s["tables"][:, :-(-N // BLOCK)].clamp_min(0).long()
    k, v = (x[blocks].transpose(1, 2).reshape(S, Hkv, -1, D)[:, :, :N].float() for x in (s["k_cache"], s["v_cache"]))
    # the rows of each sequence, padded to the most
    first, last = s["starts"][:-1, None].long(), s["starts"][1:, None].long()
    row = first + torch.arange(Q, device="cuda")
    q = s["q"][row.clamp_max(T - 1)].float()                                       # [S][Q][Hq][D]
    q = q.view(S, Q, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(S, Hkv, -1, D)
    logits = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])                 # [S][Hkv][G Q][N]
    hidden = torch.arange(N, device="cuda") >= s["lens"][:, None]
    logits.masked_fill_(hidden[:, None, None], -math.inf)
    top = logits.amax(-1, keepdim=True).clamp_min(-3e38)                           # (no keys: -inf)
    p = logits.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / total.masked_fill(total == 0, 1.0)
    o = o.view(S, Hkv, Hq // Hkv, Q, D).permute(0, 3, 1, 2, 4).reshape(S * Q, Hq, D)
    # back to rows one behind the other: row r is row r - starts[s] of the sequence s that holds it
    r = torch.arange(T, device="cuda")
    seq = torch.searchsorted(s["starts"][1:].long(), r, right=True)
    return o[seq * Q + r - s["starts"].long()[seq]].to(s["q"].dtype)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    eb = 2 if case["dtype"] == "bf16" else 4
    Hq, Hkv, D = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rope_append":
        T, live = case["tokens"], case["tokens"] - case["padding"]
        # q in and out; k and v of the tokens that have a slot in and out; positions, slots
        moved = 2 * T * Hq * D * eb + 4 * live * Hkv * D * eb + 8 * T * (case["axes"] + 1)
        return {"bytes": moved, "flops": 3 * (T * Hq + live * Hkv) * case["rot"]}
    rows, keys = _lengths(case)
    moved = 2 * sum(rows) * Hq * D * eb + sum(n for q, n in zip(rows, keys) if q) * Hkv * 2 * D * eb
    return {"bytes": moved, "flops": 4 * sum(q * n for q, n in zip(rows, keys)) * Hq * D}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rope(s) if case["op"] == "rope_append" else _exact_cross(s)


def _exact_rope(s):
    c = s["case"]
    half = c["rot"] // 2
    pairs = ([(2 * i, 2 * i + 1) for i in range(half)] if c["adjacent"] else [(i, i + half) for i in range(half)])
    axis = [0] * half if s["pair_axis"] is None else s["pair_axis"].tolist()
    caches = [s["k_cache"].double(), s["v_cache"].double()]
    turned = [s["q"].double(), s["key"].double()]
    for i, (a, b) in enumerate(pairs):
        theta = s["positions"][axis[i]].double() * s["inv_freq"][i].double()
        turn = torch.polar(torch.ones_like(theta), theta)[:, None]
        for x in turned:
            z = torch.complex(x[..., a], x[..., b]) * turn
            x[..., a], x[..., b] = z.real, z.imag
    live = torch.nonzero(s["slots"] >= 0).flatten()
    at = s["slots"][live]
    for cache, new in zip(caches, (turned[1], s["value"].double())):
        flat = cache.permute(0, 2, 1, 3).reshape(-1, c["hkv"], c["d"]).clone()
        flat[at] = new[live]
        cache.copy_(flat.view(-1, BLOCK, c["hkv"], c["d"]).permute(0, 2, 1, 3))
    return turned[0], caches[0], caches[1]


def _exact_cross(s):
    c = s["case"]
    group = c["hq"] // c["hkv"]
    rows, keys = _lengths(c)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for i, (Q, n) in enumerate(zip(rows, keys)):
        blocks = s["tables"][i, :-(-n // BLOCK)].long()
        for h in range(c["hq"] if Q and n else 0):
            k, v = (x[blocks, h // group].reshape(-1, c["d"])[:n].double() for x in (s["k_cache"], s["v_cache"]))
            weights = torch.softmax(s["q"][at:at + Q, h].double() @ k.t() * s["scale"], dim=-1)
            out[at:at + Q, h] = weights @ v
        at += Q
    return out
