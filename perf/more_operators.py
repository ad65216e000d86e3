"""Timed cases of the paged cache's prompt side: rotary positions with the append, attention
of several query tokens a sequence, and forked block tables.

Three operators that a serving step with prompts and samples runs next to the decode:

  rope     pa_rope_append: rotates queries and keys by their positions and writes keys and
           values through the slot map into the paged cache
  attend   pa_attend: attention of a ragged batch of query tokens over the paged cache:
           cross attention to states of another length, few tokens a sequence, and chunks
           of prompts with a causal mask; with the rows' log-sum-exp
  fork     pa_fork_tables: new block tables that go on from rows of the old ones (samples
           of a prompt, beams, finished requests), with the blocks' extra references,
           the free list and the copies of half-filled last blocks

`run` computes them in their plain form (elementary torch operations in 32 bits; angles in
64), or, with `own` set, through the package's entry points.  `exact` gives the same results
from the definitions in 64 bits, a sequence at a time.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DTYPE_BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ----------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # a decode step of 64 sequences, grouped heads (a rope of latency only)
        {"name": "rope_step_bf16", "op": "rope", "dtype": "bf16", "hq": 64, "hkv": 8, "d": 128, "b": 16, "rot": 128,
         "interleaved": False, "scaling": "none", "tokens": 64, "far": 32768, "fused": False},
        # prompts and chunks of a long-context model, its positions scaled by bands
        {"name": "rope_prompts_bf16", "op": "rope", "dtype": "bf16", "hq": 32, "hkv": 8, "d": 128, "b": 32, "rot": 128,
         "interleaved": False, "scaling": "yarn", "tokens": 32768, "far": 131072, "fused": True},
        # odd sizes: half of each head turned, pairs side by side, far positions, fp32
        {"name": "rope_chunks_f32", "op": "rope", "dtype": "f32", "hq": 39, "hkv": 3, "d": 64, "b": 16, "rot": 32,
         "interleaved": True, "scaling": "linear", "tokens": 1171, "far": 1000003, "fused": True},
        # a question of seven tokens to fifty states (the smallest: latency only)
        {"name": "cross_tiny_f32", "op": "attend", "dtype": "f32", "hq": 8, "hkv": 8, "d": 64, "b": 16, "seqs": 1,
         "new_lo": 7, "new_hi": 7, "kind": "uniform", "lo": 50, "hi": 50, "causal": False},
        # cross attention of ragged decoder chunks to encoder states, multi-head
        {"name": "cross_f16", "op": "attend", "dtype": "f16", "hq": 40, "hkv": 40, "d": 128, "b": 16, "seqs": 16,
         "new_lo": 150, "new_hi": 450, "kind": "uniform", "lo": 1, "hi": 1500, "causal": False},
        # one to eight drafted tokens a sequence, checked against long contexts
        {"name": "few_bf16", "op": "attend", "dtype": "bf16", "hq": 64, "hkv": 8, "d": 128, "b": 16, "seqs": 64,
         "new_lo": 1, "new_hi": 8, "kind": "loguniform", "lo": 500, "hi": 8192, "causal": True},
        # whole prompts
        {"name": "prompts_bf16", "op": "attend", "dtype": "bf16", "hq": 32, "hkv": 8, "d": 128, "b": 32, "seqs": 2,
         "new_lo": 7500, "new_hi": 8192, "kind": "own", "lo": 0, "hi": 0, "causal": True},
        # a chunk of a prompt behind a long context (the largest)
        {"name": "chunk_bf16", "op": "attend", "dtype": "bf16", "hq": 32, "hkv": 8, "d": 128, "b": 32, "seqs": 1,
         "new_lo": 1000, "new_hi": 1024, "kind": "own", "lo": 90000, "hi": 100000, "causal": True},
        # ragged chunks with empty rows and sequences, an odd head group, small heads, fp32
        {"name": "ragged_f32", "op": "attend", "dtype": "f32", "hq": 39, "hkv": 3, "d": 64, "b": 32, "seqs": 7,
         "new_lo": 0, "new_hi": 700, "kind": "ragged", "lo": 0, "hi": 1003, "causal": True},
        # sixteen prompts go on as eight samples each
        {"name": "fork_samples", "op": "fork", "b": 16, "rows": 16, "children": 128, "lo": 100, "hi": 2048,
         "pool": 4000, "ends": 0.0, "stays": 0.0, "short": False},
        # a step of 256 beams: some go on twice, some end
        {"name": "fork_beams", "op": "fork", "b": 16, "rows": 256, "children": 256, "lo": 50, "hi": 4000, "pool": 80000,
         "ends": 0.0, "stays": 0.5, "short": False},
        # a large batch: a tenth finishes, the others stay, a few fork, the pool runs short
        {"name": "fork_mixed", "op": "fork", "b": 32, "rows": 1001, "children": 1100, "lo": 0, "hi": 9000,
         "pool": 200000, "ends": 0.1, "stays": 0.8, "short": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "attend", "attend", "fork"])
    if op == "rope":
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 3, 4, 5, 8, 12, 16, 40])
        hq = hkv * min(rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 13]), max(1, 128 // hkv))
        return {"op": op, "dtype": rng.choice(["f32", "f16", "bf16"]), "hq": hq, "hkv": hkv, "d": d,
                "b": rng.choice([16, 32]), "rot": rng.choice([d, d, d // 2, d // 4, 16, 48]),
                "interleaved": rng.choice([False, True]),
                "scaling": rng.choice(["none", "linear", "ntk", "yarn", "bands"]),
                "tokens": _log(rng, 1, max(1, min(32768, (32768 * 48 * 128) // ((hq + 2 * hkv) * d * 2)))),
                "far": _log(rng, 100, 1000000), "fused": rng.choice([False, True])}
    if op == "attend":
        dtype = rng.choice(["f32", "f16", "bf16", "f16", "bf16"])
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 3, 4, 5, 8, 16, 40])
        hq = hkv * min(rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 16, 20]), max(1, 64 // hkv))
        new = rng.choice([_log(rng, 1, 8), _log(rng, 8, 300), _log(rng, 300, 4000)])
        hi = _log(rng, 16, 65536)
        causal = rng.choice([False, True, True])
        longest = hi + (new if causal else 0)
        # seqs * queries * heads * longest is what a padded batch of scores takes
        new = max(1, min(new, (1 << (30 if dtype == "f32" else 31)) // (hq * longest)))
        room = max(1, min((1 << 30) // (hq * new * longest), (1 << 29) // (hkv * d * longest)))
        return {"op": op, "dtype": dtype, "hq": hq, "hkv": hkv, "d": d, "b": rng.choice([16, 32]),
                "seqs": _log(rng, 1, min(200, room)), "new_lo": rng.choice([0, 1, new]), "new_hi": new,
                "kind": rng.choice(["ragged", "own", "loguniform"] if causal else ["ragged", "uniform", "loguniform"]),
                "lo": rng.choice([0, 1, hi // 2]), "hi": hi, "causal": causal}
    b = rng.choice([16, 32])
    hi = _log(rng, 10, 20000)
    rows = _log(rng, 1, max(1, min(2000, 1000000 // (1 + hi // b))))
    children = max(1, min(2000, int(rows * rng.choice([0.5, 1, 1, 1.3, 4, 8]))))
    return {"op": op, "b": b, "rows": rows, "children": children, "lo": rng.choice([0, 1, hi // 2]), "hi": hi,
            "pool": rows * (hi // b + 2) + rng.choice([0, 100, 2500, 100000]), "ends": rng.choice([0.0, 0.1, 0.5]),
            "stays": rng.choice([0.0, 0.5, 0.9]), "short": rng.choice([False, False, True])}


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------
def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _tables(nbs, pool, width, g):
    """int32 [S, width] of distinct random blocks of the pool, -1 padded, and the others."""
    order = g.permutation(pool).astype(np.int32)
    bt = np.full((len(nbs), width), -1, dtype=np.int32)
    at = 0
    for s, n in enumerate(nbs):
        bt[s, :n] = order[at:at + n]
        at += n
    return bt, order[at:]


def _frequencies(rot, scaling):
    """(angles per position, float64 [rot / 2]; amplitude) of the scalings, each a factor 8
    over 4096 positions: linear; ntk, a larger base; yarn and bands, a ramp between scaled and
    unscaled angles over a pair's turns within the 4096 positions."""
    base, factor, length = 10000.0, 8.0, 4096.0
    if scaling == "ntk":
        base *= factor ** (rot / max(rot - 2, 1))
    f = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "bands":                       # linear in the turns, from 1 to 4
        keep = np.clip((length * f / (2 * math.pi) - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        return f / factor * (1 - keep) + f * keep, 1.0
    if scaling == "yarn":                        # linear in the pair's index, from 32 turns to 1
        at = [rot * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _turns(f):
    """Angles per position as int64: turns of 2 pi in units of 2^-64."""
    t = f / (2 * math.pi)
    t = np.rint((t - np.floor(t)) * 2.0 ** 64)
    return np.array([int(x) % (1 << 64) for x in t], dtype=np.uint64).view(np.int64)


def _prepare_rope(case, g, gen):
    st = dict(case)
    n, hq, hkv, d, b = case["tokens"], case["hq"], case["hkv"], case["d"], case["b"]
    dt = DTYPES[case["dtype"]]
    if case["fused"]:                            # one projection's rows: queries, keys, values
        rows = torch.randn(n, (hq + 2 * hkv) * d, device="cuda", generator=gen).to(dt)
        q, k, v = rows.split([hq * d, hkv * d, hkv * d], dim=1)
        st["q"], st["k"], st["v"] = q.unflatten(1, (hq, d)), k.unflatten(1, (hkv, d)), v.unflatten(1, (hkv, d))
    else:
        st["q"], st["k"], st["v"] = (torch.randn(n, h, d, device="cuda", generator=gen).to(dt) for h in (hq, hkv, hkv))
    # runs of tokens at consecutive positions, as chunks of prompts and decode steps have
    start = g.integers(0, 2, size=n) if n < 300 else g.random(n) < 1 / 300
    run_id = np.cumsum(start)
    first = g.integers(0, max(1, case["far"] - n), size=int(run_id[-1]) + 1)
    at = np.arange(n)
    begin = np.maximum.accumulate(np.where(start.astype(bool), at, 0))
    st["pos"] = _dev((first[run_id] + at - begin).astype(np.int32))
    nb = -(-n // b) + 3
    slots = g.permutation(nb).astype(np.int64)[np.arange(n) // b] * b + np.arange(n) % b
    slots[g.random(n) < 0.02] = -1               # padding
    st["slots"] = _dev(slots)
    f, st["amplitude"] = _frequencies(case["rot"], case["scaling"])
    st["f"], st["freqs"] = _dev(f), _dev(_turns(f))
    st["caches"] = torch.zeros(2, nb, b, hkv, d, dtype=dt, device="cuda")
    st["q_out"] = torch.zeros(n, hq, d, dtype=dt, device="cuda")
    return st


def _lens(case, g):
    """(query tokens, context lengths) of an attend case."""
    s = case["seqs"]
    new = g.integers(case["new_lo"], case["new_hi"] + 1, size=s)
    lo, hi = case["lo"], case["hi"]
    if case["kind"] == "loguniform":
        t = np.rint(np.exp(g.uniform(math.log(max(lo, 1)), math.log(max(hi, 1)), size=s))).astype(np.int64)
    else:
        t = g.integers(lo, hi + 1, size=s)
    if case["causal"] and case["kind"] != "ragged":
        t = t + new                              # the query tokens are the last of the context
    if case["kind"] == "ragged":                 # empty sequences, sequences without queries
        t[g.random(s) < 0.15] = 0
        new[g.random(s) < 0.15] = 0
    if new.sum() == 0:
        new[0] = 1
    return new.astype(np.int64), t.astype(np.int64)


def _prepare_attend(case, g, gen):
    st = dict(case)
    hq, hkv, d, b = case["hq"], case["hkv"], case["d"], case["b"]
    new, lens = _lens(case, g)
    nbs = (lens + b - 1) // b
    pool = int(1.1 * int(nbs.sum())) + 1
    bt, _ = _tables(nbs, pool, max(1, int(nbs.max())), g)
    dt = DTYPES[case["dtype"]]
    rows = case["seqs"] * case["new_hi"] + 3     # the rows of a program that planned for the most; the last are padding
    st["caches"] = torch.randn(2, pool, b, hkv, d, device="cuda", generator=gen, dtype=torch.float32).to(dt)
    st["q"] = torch.randn(rows, hq, d, device="cuda", generator=gen).to(dt)
    st["bt"], st["cl"] = _dev(bt), _dev(lens.astype(np.int32))
    st["qs"] = _dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))
    st["longest"], st["most"], st["rows"] = max(1, int(lens.max())), int(new.max()), int(new.sum())
    st["out"] = torch.zeros_like(st["q"])
    st["lse"] = torch.zeros(rows, hq, dtype=torch.float32, device="cuda")
    return st


def _prepare_fork(case, g, gen):
    st = dict(case)
    b, rows, children, pool = case["b"], case["rows"], case["children"], case["pool"]
    lens = g.integers(case["lo"], case["hi"] + 1, size=rows)
    width = -(-case["hi"] // b) + 2
    nbs = -(-lens // b)
    bt, rest = _tables(nbs, max(pool, int(nbs.sum()) + 1), width, g)
    # pairs of rows share their leading full blocks, as samples of one prompt do
    extra = np.zeros(max(pool, int(nbs.sum()) + 1), dtype=np.int32)
    spare = [rest]
    for s in range(1, rows, 2):
        n = min(lens[s - 1] // b, lens[s] // b) // 2
        spare.append(bt[s, :n].copy())
        bt[s, :n] = bt[s - 1, :n]
        extra[bt[s, :n]] += 1
    rest = np.concatenate(spare)
    parents = np.where(g.random(children) < case["stays"], np.arange(children), g.integers(0, rows, size=children))
    if case["stays"] == 0.0 and children % rows == 0:
        parents = np.arange(children) // (children // rows)        # samples of each prompt
    parents[g.random(children) < case["ends"]] = -1
    parents[parents >= rows] = -1
    kids = np.bincount(parents[parents >= 0], minlength=rows)
    need = int(np.maximum(kids - 1, 0)[lens % b > 0].sum())
    spare = min(len(rest), need // 3 if case["short"] else need + 16)
    free = np.zeros(len(extra), dtype=np.int32)
    free[:spare] = rest[:spare]
    st["bt"], st["cl"], st["parents"] = _dev(bt), _dev(lens.astype(np.int32)), _dev(parents.astype(np.int32))
    st["extra"], st["free"], st["nfree"] = _dev(extra), _dev(free), _dev(np.array([spare], dtype=np.int32))
    i32 = dict(dtype=torch.int32, device="cuda")
    st["bt2"], st["cl2"] = torch.full((children, width), -1, **i32), torch.zeros(children, **i32)
    st["nfree2"], st["pairs"] = torch.zeros(1, **i32), torch.zeros(children, 2, **i32)
    st["granted"] = torch.zeros(children, **i32)
    return st


def prepare(case, seed):
    g = np.random.default_rng([seed, 11])
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"rope": _prepare_rope, "attend": _prepare_attend, "fork": _prepare_fork}[case["op"]](case, g, gen)


# ----------------------------------------------------------------------------
# Plain forms
# ----------------------------------------------------------------------------
def _rotate(x, cos, sin, rot, interleaved):
    """x [N, H, d] with its first `rot` elements rotated; cos, sin [N, 1, rot / 2]."""
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _rope_plain(st):
    angle = (st["pos"].double()[:, None] * st["f"])[:, None, :]
    cos, sin = (torch.cos(angle) * st["amplitude"]).float(), (torch.sin(angle) * st["amplitude"]).float()
    q, k = (_rotate(st[n].float(), cos, sin, st["rot"], st["interleaved"]) for n in ("q", "k"))
    dt = st["q"].dtype
    st["q_out"].copy_(q.to(dt))
    kept = st["slots"] >= 0
    rows = st["caches"].flatten(1, 2)
    rows[0, st["slots"][kept]] = k.to(dt)[kept]
    rows[1, st["slots"][kept]] = st["v"][kept]
    return {"q": st["q_out"], "caches": st["caches"]}


def _attend_plain(st):
    hq, hkv, b, d = st["hq"], st["hkv"], st["b"], st["d"]
    bt, cl, qs = st["bt"], st["cl"].long(), st["qs"].long()
    s, w = bt.shape
    m, t = st["most"], st["longest"]
    dev = bt.device
    new = qs[1:] - qs[:-1]
    seq = torch.repeat_interleave(torch.arange(s, device=dev), new, output_size=st["rows"])
    row = torch.arange(st["rows"], device=dev) - qs[seq]
    ids = bt.clamp(min=0).long()
    k, v = (c[ids].float().permute(0, 3, 1, 2, 4).reshape(s, hkv, w * b, d)[:, :, :t] for c in st["caches"])
    q = torch.zeros(s, m, hq, d, device=dev)
    q[seq, row] = st["q"][:st["rows"]].float()
    q = q.view(s, m, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(s, hkv, -1, d)
    sc = torch.matmul(q, k.transpose(-1, -2)).view(s, hkv, hq // hkv, m, t)      # [S, Hkv, G, M, T]
    sc *= d ** -0.5
    last = (cl - new)[:, None] + torch.arange(m, device=dev) if st["causal"] else cl[:, None].expand(s, m) - 1
    key = torch.arange(t, device=dev)
    seen = (key <= last[:, :, None]) & (key < cl[:, None, None])                 # [S, M, T]
    sc.masked_fill_(~seen[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = sc.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(s, hkv, -1, t), v).view(s, hkv, hq // hkv, m, d)
    o = o / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total))[..., 0]
    out, lse_out = st["out"], st["lse"]
    out[:st["rows"]] = o.permute(0, 3, 1, 2, 4).reshape(s, m, hq, d)[seq, row].to(out.dtype)
    lse_out[:st["rows"]] = lse.permute(0, 3, 1, 2).reshape(s, m, hq)[seq, row]
    return {"out": out, "lse": lse_out}


def _fork_plain(st):
    b = st["b"]
    bt, cl, parents = st["bt"], st["cl"].long(), st["parents"].long()
    rows, w = bt.shape
    c = len(parents)
    dev = bt.device
    pool = len(st["extra"])
    j = torch.arange(w, device=dev)
    nb = (cl + b - 1) // b
    half = cl % b > 0                                                            # the last block is not full
    real = parents >= 0
    p = parents.clamp(min=0)
    kids = torch.zeros(rows, dtype=torch.long, device=dev).scatter_add(0, p, real.long())
    i = torch.arange(c, device=dev)
    first = torch.full((rows,), c, device=dev).scatter_reduce(0, p, torch.where(real, i, c), "amin")
    copies = real & half[p] & (i != first[p])
    # references: each old row drops its own, each new row takes one; a half-filled last
    # block stays with the first new row
    delta = (kids - 1)[:, None].expand(rows, w)
    last = half[:, None] & (j == nb[:, None] - 1)
    delta = torch.where(last, delta.clamp(max=0), delta)
    used = j < nb[:, None]
    extra = st["extra"].long().index_add(0, bt[used].long(), delta[used])
    ids = torch.nonzero(extra < 0)[:, 0]
    extra = extra.clamp(min=0)
    nfree = st["nfree"].long()
    free = torch.cat([st["free"].long(), st["free"].new_zeros(1).long()])
    at = nfree + torch.arange(len(ids), device=dev)
    free = free.index_put((at.clamp(max=pool),), ids)[:pool]
    have = nfree + len(ids)
    rank = torch.cumsum(copies.long(), 0) - 1
    refused = copies & (rank >= have)
    got = copies & ~refused
    popped = free[(have - 1 - rank).clamp(0, pool - 1)]
    # a refused row takes no references
    undo = (j < (nb[p] - 1)[:, None]) & refused[:, None]
    extra = extra.index_add(0, bt[p][undo].long(), -torch.ones(1, dtype=torch.long, device=dev).expand(int(undo.sum())))
    alive = real & ~refused
    filled = (j < nb[p][:, None]) & alive[:, None]
    table = torch.where(filled, bt[p], torch.full_like(bt[p], -1))
    table = torch.where(got[:, None] & (j == nb[p][:, None] - 1), popped[:, None].int(), table)
    source = bt[p, (nb[p] - 1).clamp(min=0)].long()
    none = torch.full_like(source, -1)
    pairs = torch.stack([torch.where(got, source, none), torch.where(got, popped, none)], dim=1)
    st["extra"].copy_(extra)
    st["free"].copy_(free)
    return {"tables": table, "lens": torch.where(alive, cl[p], torch.zeros_like(p)).int(), "extra": st["extra"],
            "free": st["free"], "num_free": (have - got.sum()).int(), "pairs": pairs.int(),
            "granted": torch.where(refused, -1, real.long()).int()}


def run(st):
    if own:
        import paged_kv_cache_79_gb300 as P
        if st["op"] == "rope":
            P.pa_rope_append(st["q_out"], st["q"], st["k"], st["v"], st["caches"][0], st["caches"][1], st["pos"],
                             st["slots"], st["freqs"], interleaved=st["interleaved"], amplitude=st["amplitude"])
            return {"q": st["q_out"], "caches": st["caches"]}
        if st["op"] == "attend":
            P.pa_attend(st["out"], st["q"], st["caches"][0], st["caches"][1], st["bt"], st["cl"], st["qs"],
                        st["d"] ** -0.5, st["hq"], st["hkv"], st["d"], st["b"], causal=st["causal"], lse=st["lse"])
            return {"out": st["out"], "lse": st["lse"]}
        P.pa_fork_tables(st["bt2"], st["cl2"], st["bt"], st["cl"], st["parents"], st["extra"], st["free"], st["nfree"],
                         st["b"], st["pairs"], st["granted"], num_free_out=st["nfree2"])
        return {"tables": st["bt2"], "lens": st["cl2"], "extra": st["extra"], "free": st["free"],
                "num_free": st["nfree2"], "pairs": st["pairs"], "granted": st["granted"]}
    if st["op"] == "rope":
        return _rope_plain(st)
    if st["op"] == "attend":
        return _attend_plain(st)
    return _fork_plain(st)


# ----------------------------------------------------------------------------
# Work: each input read once, each output written once
# ----------------------------------------------------------------------------
def work(case):
    g = np.random.default_rng([0, 11])
    if case["op"] == "rope":
        n, e = case["tokens"], DTYPE_BYTES[case["dtype"]]
        return {"bytes": n * (case["hq"] + 2 * case["hkv"]) * case["d"] * 2 * e + n * 12 + case["rot"] * 4,
                "flops": n * (case["hq"] + case["hkv"]) * case["rot"] * 3}
    if case["op"] == "attend":
        new, lens = _lens(case, g)
        hq, hkv, d, e = case["hq"], case["hkv"], case["d"], DTYPE_BYTES[case["dtype"]]
        pairs = 0
        for n, t in zip(new.tolist(), lens.tolist()):
            if not case["causal"]:
                pairs += n * t
            else:                                # query i of n sees t - n + i + 1 keys, none where that is negative
                first = max(0, n - t)
                pairs += (n - first) * (max(t - n, 0) + 1 + t) // 2 if n > first else 0
        rows, keys = int(new.sum()), int(lens[new > 0].sum())
        return {"bytes": keys * hkv * d * 2 * e + rows * hq * (2 * d * e + 4) + (keys // case["b"] + 3 * len(new)) * 4,
                "flops": 4 * pairs * hq * d}
    b, rows, children = case["b"], case["rows"], case["children"]
    width = -(-case["hi"] // b) + 2
    lens = g.integers(case["lo"], case["hi"] + 1, size=rows)
    entries = int((-(-lens // b)).sum())
    # old tables read, new ones written whole, references of the blocks that change
    return {"bytes": 4 * (entries + children * width + int(entries * (1 - case["stays"])) * 2 + rows + 6 * children),
            "flops": entries}


# ----------------------------------------------------------------------------
# The definitions in 64 bits, one sequence or row at a time
# ----------------------------------------------------------------------------
def _exact_rope(case, st):
    rot, d = case["rot"], case["d"]
    angle = st["pos"].double()[:, None] * st["f"]
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    i = torch.arange(rot // 2, device="cuda")
    one, two = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)

    def turned(x):
        x = x.double()
        y = x.clone()
        y[..., one] = (x[..., one] * c - x[..., two] * s) * st["amplitude"]
        y[..., two] = (x[..., one] * s + x[..., two] * c) * st["amplitude"]
        return y

    caches = torch.zeros(2, st["caches"].shape[1] * case["b"], case["hkv"], d, dtype=torch.float64, device="cuda")
    k = turned(st["k"])
    at = torch.nonzero(st["slots"] >= 0)[:, 0]
    caches[0].index_copy_(0, st["slots"][at], k[at])
    caches[1].index_copy_(0, st["slots"][at], st["v"][at].double())
    return {"q": turned(st["q"]), "caches": caches.view(st["caches"].shape)}


def _exact_attend(case, st):
    hq, hkv, b, d = case["hq"], case["hkv"], case["b"], case["d"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device="cuda")
    qs, lens = st["qs"].tolist(), st["cl"].tolist()
    for s, t in enumerate(lens):
        lo, hi = qs[s], qs[s + 1]
        if hi == lo:
            continue
        if t == 0:
            lse[lo:hi] = -math.inf
            continue
        ids = st["bt"][s, :-(-t // b)].long()
        i, j = torch.arange(hi - lo, device="cuda")[:, None], torch.arange(t, device="cuda")
        hidden = j > t - (hi - lo) + i if case["causal"] else None
        for h in range(hkv):
            k, v = (c[ids, :, h].reshape(-1, d)[:t].double() for c in st["caches"])
            for a in range(h * hq // hkv, (h + 1) * hq // hkv):
                sc = st["q"][lo:hi, a].double() @ k.T / math.sqrt(d)
                if hidden is not None:
                    sc[hidden] = -math.inf
                z = torch.logsumexp(sc, -1)
                lse[lo:hi, a] = z
                sc -= torch.where(z == -math.inf, torch.zeros_like(z), z)[:, None]
                out[lo:hi, a] = sc.exp_() @ v
    return {"out": out, "lse": lse}


def _exact_fork(case, st):
    b = case["b"]
    bt, lens, parents, extra, free = (st[k].cpu().numpy().copy() for k in ("bt", "cl", "parents", "extra", "free"))
    have = int(st["nfree"][0])
    rows, width = bt.shape
    table = np.full((len(parents), width), -1, dtype=np.int32)
    pairs = np.full((len(parents), 2), -1, dtype=np.int32)
    lens2, granted = np.zeros(len(parents), dtype=np.int32), np.zeros(len(parents), dtype=np.int32)
    copies, seen = [], set()
    for i, p in enumerate(parents.tolist()):     # every new row takes its references
        if p < 0:
            continue
        n = -(-int(lens[p]) // b)
        table[i, :n], lens2[i], granted[i] = bt[p, :n], lens[p], 1
        full = n - (lens[p] % b > 0)
        extra[bt[p, :full]] += 1
        if full < n and p in seen:
            copies.append(i)
        elif full < n:
            extra[bt[p, full]] += 1
        seen.add(p)
    for p in range(rows):                        # and every old one drops its own
        extra[bt[p, :-(-int(lens[p]) // b)]] -= 1
    for block in np.nonzero(extra < 0)[0]:
        free[have], extra[block] = block, 0
        have += 1
    for i in copies:
        p = int(parents[i])
        n = -(-int(lens[p]) // b)
        if have == 0:
            extra[bt[p, :n - 1]] -= 1
            table[i], lens2[i], granted[i] = -1, 0, -1
            continue
        have -= 1
        pairs[i] = bt[p, n - 1], free[have]
        table[i, n - 1] = free[have]
    out = {"tables": table, "lens": lens2, "extra": extra, "free": free, "num_free": np.array([have], dtype=np.int32),
           "pairs": pairs, "granted": granted}
    return {k: torch.from_numpy(v) for k, v in out.items()}


def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "attend": _exact_attend, "fork": _exact_fork}[case["op"]](case, st)
