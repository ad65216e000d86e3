"""pa_build_tables on the GPU against the one-request-at-a-time model, and the serving
step it opens: tables, append, decode, on the 8-bit and the 16-bit cache."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_79_gb300 as P
from tests import q8_model as M
from tests.test_gpu_q8 import check_decode, dev

pytestmark = pytest.mark.gpu
DEV = "cuda"


def batch(seed, reqs, b, width, pool, max_len, spare=None):
    """Tables, lengths and a free list of a running batch."""
    rng = np.random.default_rng(seed)
    cl = rng.integers(0, max_len + 1, size=reqs).astype(np.int32)
    order = rng.permutation(pool).astype(np.int32)
    bt = np.full((reqs, width), -1, dtype=np.int32)
    at = 0
    for s in range(reqs):
        n = -(-int(cl[s]) // b)
        bt[s, :n] = order[at:at + n]
        at += n
    assert at <= pool
    free = np.full(pool, -77, dtype=np.int32)
    left = pool - at if spare is None else min(spare, pool - at)
    free[:left] = order[at:at + left]
    return rng, bt, cl, free, left


def run(bt, cl, new, free, nfree, b, num_slots, in_place=False):
    d = [dev(bt), dev(cl), dev(new.astype(np.int32)), dev(free), dev(np.array([nfree], dtype=np.int32))]
    slots = torch.full((num_slots,), 12345, dtype=torch.int64, device=DEV)
    qs = torch.full((len(cl) + 1,), 99, dtype=torch.int32, device=DEV)
    granted = torch.full((len(cl),), 99, dtype=torch.int32, device=DEV)
    kw = {}
    if not in_place:
        kw = dict(context_lens_out=torch.full_like(d[1], 99), num_free_out=torch.full_like(d[4], 99))
    P.pa_build_tables(d[0], d[1], d[2], d[3], d[4], b, slots, qs, granted, **kw)
    torch.cuda.synchronize()
    if not in_place:
        assert np.array_equal(d[1].cpu().numpy(), cl) and int(d[4]) == nfree
    return (d[0].cpu().numpy(), (d[1] if in_place else kw["context_lens_out"]).cpu().numpy(), d[3].cpu().numpy(),
            int(d[4] if in_place else kw["num_free_out"]), granted.cpu().numpy(), qs.cpu().numpy(),
            slots.cpu().numpy())


NAMES = ("tables", "lens", "free", "num_free", "granted", "query_start", "slots")


def check(bt, cl, new, free, nfree, b, num_slots, in_place=False):
    got = run(bt, cl, new, free, nfree, b, num_slots, in_place)
    want = M.build_tables(bt, cl, new, free, nfree, b, num_slots)
    for name, g, w in zip(NAMES, got, want):
        assert np.array_equal(g, w), name
    return want


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("reqs,b,max_len,max_new", [
    (1, 16, 0, 1), (1, 32, 100, 5000), (3, 16, 40, 33), (31, 16, 64, 1), (256, 32, 700, 1), (64, 16, 0, 800),
    (1024, 16, 50, 3), (1025, 16, 50, 3), (2600, 32, 90, 20), (5, 1, 9, 4), (9, 48, 100, 200)])
def test_growing_and_releasing(reqs, b, max_len, max_new, in_place):
    width = (max_len + max_new) // b + 2
    rng, bt, cl, free, nfree = batch(reqs + b, reqs, b, width, reqs * width + 3, max_len)
    new = rng.integers(0, max_new + 1, size=reqs)
    check(bt, cl, new, free, nfree, b, int(new.sum()), in_place)          # a slot map that just fits
    new[rng.random(reqs) < 0.3] = -1
    check(bt, cl, new, free, nfree, b, int(np.maximum(new, 0).sum()) + 77, in_place)
    check(bt, cl, np.full(reqs, -5), free, nfree, b, 4, in_place)         # everything goes
    check(bt, cl, np.zeros(reqs, dtype=int), free, nfree, b, 0, in_place)  # nothing happens


@pytest.mark.parametrize("reqs", [7, 300, 1500])
def test_refusals(reqs):
    b, width = 16, 8
    rng, bt, cl, free, nfree = batch(reqs, reqs, b, width, reqs * width, 60, spare=reqs // 2)
    new = rng.integers(0, 40, size=reqs)
    want = check(bt, cl, new, free, nfree, b, int(new.sum()))              # the pool runs short
    assert (want[4] == -1).any() and (want[4] > 0).any()
    new[rng.random(reqs) < 0.2] = -1                                       # released blocks are granted again
    want = check(bt, cl, new, free, nfree, b, 20 * reqs)
    want = check(bt, cl, np.maximum(new, 0), free, nfree, b, 2 * reqs)     # the slot map runs short
    assert (want[4] == -1).any()
    new = rng.integers(0, 200, size=reqs)                                  # table rows run short
    want = check(bt, cl, new, np.concatenate([free, free]), nfree, b, 1000 * reqs)
    assert (want[4] == -1).any()
    check(bt, cl, new, free, 0, b, 100 * reqs)                             # an empty pool
    new = np.full(reqs, 2 ** 31 - 1)
    check(bt, cl, new, free, nfree, b, 5)


def test_out_of_range_inputs_stay_inside():
    b, width, reqs = 16, 4, 6
    rng, bt, cl, free, nfree = batch(3, reqs, b, width, 30, 40)
    cl[0], cl[1] = -9, 10 ** 9                        # a length below 0, one past its row
    new = np.array([5, 1, -1, 3, 30, 2])
    check(bt, cl, new, free, nfree, b, 100)
    check(bt, cl, np.array([-1, -1, 3, 0, 4, 1]), free, nfree, b, 100)
    check(bt, cl, new, free, 10 ** 9, b, 100)         # a count past the list
    check(bt, cl, new, free, -3, b, 100)
    cl[:] = 40
    check(bt, cl, np.full(reqs, -1), free, 28, b, 3)  # more blocks released than the list holds


@pytest.mark.parametrize("slots", [4095, 4096, 4097, 9000])
def test_slot_maps_around_the_second_kernel(slots):
    """Up to 4096 slots one kernel writes the map, above a second one: exact fits and
    padding on both sides, few requests and many."""
    b = 16
    for reqs, each in ((1, slots), (1, slots - 1), (3, slots // 3), (700, 5), (2050, 1)):
        width = (each + 40) // b + 2
        rng, bt, cl, free, nfree = batch(slots + reqs, reqs, b, width, reqs * width, 40)
        check(bt, cl, np.full(reqs, each), free, nfree, b, slots)


def test_two_at_once_on_side_streams():
    jobs = []
    for i, n in enumerate((30, 5000)):                  # one kernel, two kernels
        rng, bt, cl, free, nfree = batch(40 + i, 20, 16, 300, 6000, 60)
        new = rng.integers(0, n // 20 + 1, size=20)
        new[3] = -1
        t = [dev(x) for x in (bt, cl, new.astype(np.int32), free, np.array([nfree], dtype=np.int32))]
        out = [torch.zeros(n, dtype=torch.int64, device=DEV), torch.zeros(21, dtype=torch.int32, device=DEV),
               torch.zeros(20, dtype=torch.int32, device=DEV)]
        jobs.append((t, out, M.build_tables(bt, cl, new, free, nfree, 16, n), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for t, out, _, st in jobs:
        P.pa_build_tables(*t, 16, *out, stream=st)
    torch.cuda.synchronize()
    for t, out, want, _ in jobs:
        got = (t[0], t[1], t[3], t[4], out[2], out[1], out[0])
        for name, g, w in zip(NAMES, got, want):
            assert np.array_equal(np.asarray(g.cpu()).reshape(np.shape(w)), w), name


def test_no_requests():
    slots, qs = torch.full((5,), 7, dtype=torch.int64, device=DEV), torch.full((1,), 7, dtype=torch.int32, device=DEV)
    e = torch.zeros(0, dtype=torch.int32, device=DEV)
    nf = torch.tensor([3], dtype=torch.int32, device=DEV)
    P.pa_build_tables(torch.zeros(0, 4, dtype=torch.int32, device=DEV), e, e, torch.arange(8, dtype=torch.int32, device=DEV),
                      nf, 16, slots, qs, e)
    assert (slots == -1).all() and qs.item() == 0 and nf.item() == 3


def test_a_long_run_in_a_graph_follows_the_host_allocator():
    """50 steps of continuous batching replayed from one graph, in place."""
    b, width, reqs, pool, slots_n = 16, 20, 40, 500, 800
    rng = np.random.default_rng(11)
    order = rng.permutation(pool).astype(np.int32)
    bt, cl = np.full((reqs, width), -1, dtype=np.int32), np.zeros(reqs, dtype=np.int32)
    free, nfree = order.copy(), pool
    d_bt, d_cl, d_new, d_free, d_nf = (dev(bt), dev(cl), dev(np.zeros(reqs, dtype=np.int32)), dev(free),
                                       dev(np.array([nfree], dtype=np.int32)))
    slots = torch.zeros(slots_n, dtype=torch.int64, device=DEV)
    qs, granted = torch.zeros(reqs + 1, dtype=torch.int32, device=DEV), torch.zeros(reqs, dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        P.pa_build_tables(d_bt, d_cl, d_new, d_free, d_nf, b, slots, qs, granted)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        P.pa_build_tables(d_bt, d_cl, d_new, d_free, d_nf, b, slots, qs, granted)
    refused = 0
    for _ in range(50):
        new = np.where(rng.random(reqs) < 0.3, rng.integers(1, 90, size=reqs), 1)
        new[rng.random(reqs) < 0.1] = -1
        d_new.copy_(torch.from_numpy(new.astype(np.int32)))
        g.replay()
        torch.cuda.synchronize()
        bt, cl, free, nfree, gr, q, sl = M.build_tables(bt, cl, new, free, nfree, b, slots_n)
        refused += int((gr < 0).sum())
        for t, w in ((d_bt, bt), (d_cl, cl), (d_free, free), (granted, gr), (qs, q), (slots, sl)):
            assert np.array_equal(t.cpu().numpy(), w)
        assert d_nf.item() == nfree
    assert refused > 0


@pytest.mark.parametrize("dtype,hq,hkv,d,b", [("bf16", 16, 4, 128, 16), ("f32", 6, 3, 64, 32), ("f16", 20, 1, 128, 32)])
def test_a_serving_run(dtype, hq, hkv, d, b):
    """Prompts, single tokens, releases and admissions: tables, append and decode one
    after the other on one stream, against the models at every step; and the same slot
    maps drive the 16-bit cache."""
    td = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    reqs, width, pool = 6, 9, 40
    rng = np.random.default_rng(12)
    bt, cl = np.full((reqs, width), -1, dtype=np.int32), np.zeros(reqs, dtype=np.int32)
    free, nfree = rng.permutation(pool).astype(np.int32), pool
    model = M.Cache(np.zeros((pool, M.block_bytes(hkv, b, d)), dtype=np.uint8), hkv, b, d)
    cache = P.alloc_q8_cache(pool, hkv, d, b)
    kc, vc = (torch.zeros(pool, b, hkv, d, dtype=td, device=DEV) for _ in range(2))
    d_bt, d_cl, d_free, d_nf = dev(bt), dev(cl), dev(free), dev(np.array([nfree], dtype=np.int32))
    scale = 1.0 / math.sqrt(d)
    for step in range(12):
        new = rng.integers(0, 3 * b, size=reqs) if step % 4 == 0 else np.ones(reqs, dtype=int)
        if step % 4 == 3:
            new[rng.integers(0, reqs)] = -1
        n = 4 * b * reqs
        slots = torch.zeros(n, dtype=torch.int64, device=DEV)
        qs, granted = torch.zeros(reqs + 1, dtype=torch.int32, device=DEV), torch.zeros(reqs, dtype=torch.int32, device=DEV)
        k, v = (torch.from_numpy(rng.standard_normal((n, hkv, d))).to(td) for _ in range(2))   # padded rows
        q = torch.from_numpy(rng.standard_normal((reqs, hq, d))).to(td)
        out = torch.empty_like(q, device=DEV)
        P.pa_build_tables(d_bt, d_cl, dev(new.astype(np.int32)), d_free, d_nf, b, slots, qs, granted)
        P.pa_q8_append(k.to(DEV), v.to(DEV), cache, d_bt, d_cl, b, query_start=qs)
        P.pa_q8_decode(out, q.to(DEV), cache, d_bt, d_cl, scale, hq, hkv, d, b)
        P.pa_reshape_and_cache(k.to(DEV), v.to(DEV), kc, vc, slots)
        torch.cuda.synchronize()
        bt, cl, free, nfree, gr, wqs, _ = M.build_tables(bt, cl, new, free, nfree, b, n)
        assert np.array_equal(d_cl.cpu().numpy(), cl) and np.array_equal(d_bt.cpu().numpy(), bt)
        M.append(model, k.double().numpy(), v.double().numpy(), bt, cl, wqs)
        assert np.array_equal(cache.cpu().numpy(), model.raw)
        check_decode(out, model, q, bt, cl, scale, dtype)
        # the rows of the 16-bit cache are the ones the codes stand for, to e4m3's half
        # step (2^-4 of the value, or of the smallest normal number), rounded twice at most
        for s in range(reqs):
            t = int(cl[s])
            if t:
                ids = bt[s, :-(-t // b)]
                codes = model.values(ids).transpose(2, 0, 3, 1, 4).reshape(2, -1, hkv, d)[:, :t]
                rows = torch.stack([kc, vc])[:, torch.from_numpy(ids).long().to(DEV)].double().cpu().numpy()
                rows = rows.reshape(2, -1, hkv, d)[:, :t]
                sc = np.repeat(model.scales[ids].astype(np.float64), b, axis=0)[:t].transpose(2, 0, 1)[..., None]
                assert (np.abs(codes - rows) <= 2 * 2.0 ** -4 * np.maximum(np.abs(rows), 2.0 ** -6 * sc)).all()
    assert P.pa_device_errors() == 0
