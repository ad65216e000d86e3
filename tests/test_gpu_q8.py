"""The 8-bit cache on the GPU against the 64-bit models of tests/q8_model.py: the
quantising append byte for byte, the decode within the rounding of its terms.

Tolerance of the decode, elementwise, with u_T = finfo(T).eps / 2 the output's rounding,
A = sum p |v| / sum p and S = max_t |scale| * sum |q k| (both from the model):
    u_T max(|out|, N_T) + A (r + 2 ds + (n / 16 + 8) 2^-23)
N_T the type's smallest normal number: below it the steps no longer shrink with the
    value, so the output's rounding stays half the smallest step, u_T N_T (fp16: 2^-25)
r   rounding of p: 2^-11 (fp16) for 16-bit types, 2^-21 (two fp16 terms) for fp32; p
    also takes exp2's error, 2^-22, and two products, 2^-23
ds  error of a score, in the exponent (it moves the term and the sum: twice): each of
    the d / 16 (fp32: d / 8) tensor-pipe steps may truncate at 2^-23 of the partial sums,
    at most S; the scale's products add 3 * 2^-24 S; fp32 queries lose 2^-22 each
n   accumulation: a truncation at 2^-23 of the running sum for each 16 tokens
"""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_79_gb300 as P
import workloads as W
from tests import q8_model as M

pytestmark = pytest.mark.gpu
DEV = "cuda"
TD = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def tolerance(dtype, d, out, size, smax, cl):
    u = torch.finfo(TD[dtype]).eps / 2
    f32 = dtype == "f32"
    n = np.maximum(np.asarray(cl), 0)[:, None, None]
    ds = smax[..., None] * ((d / (8 if f32 else 16)) * 2.0 ** -23 + 3 * 2.0 ** -24 + (2.0 ** -22 if f32 else 0))
    r = (2.0 ** -21 if f32 else 2.0 ** -11) + 2.0 ** -22 + 2.0 ** -23
    return u * np.maximum(np.abs(out), torch.finfo(TD[dtype]).smallest_normal) + size * (r + 2 * ds + (n / 16 + 8) * 2.0 ** -23) + 1e-30


def random_cache(rng, nb, hkv, b, d, exps=(-8, -5), spread=110.0):
    """uint8 cache with N(0, spread^2) codes and power-of-two scales."""
    raw = np.zeros((nb, M.block_bytes(hkv, b, d)), dtype=np.uint8)
    c = M.Cache(raw, hkv, b, d)
    c.codes[...] = M.encode(np.clip(rng.standard_normal(c.codes.shape) * spread, -448, 448))
    c.scales[...] = 2.0 ** rng.integers(exps[0], exps[1] + 1, size=c.scales.shape)
    return c


def decode_case(seed, dtype, d, b, hq, hkv, lens, stale=True, **kw):
    rng = np.random.default_rng(seed)
    nbs = [(max(t, 0) + b - 1) // b for t in lens]
    nb = sum(nbs) + 5
    bt, _ = W.random_tables(rng, [max(t, 0) for t in lens], b, nb, pad=1)
    c = random_cache(rng, nb, hkv, b, d, **kw)
    if stale:  # rows past each context and unreferenced blocks: NaN codes, and NaN scales
        used = np.zeros((nb, b), dtype=bool)
        for s, t in enumerate(lens):
            for tok in range(t):
                used[bt[s, tok // b], tok % b] = True
        c.codes.transpose(0, 3, 1, 2, 4)[~used] = 0x7F
        c.scales[~used.any(1)] = np.nan
    q = torch.from_numpy(rng.standard_normal((len(lens), hq, d))).to(TD[dtype])
    return c, q, bt, np.asarray(lens, dtype=np.int32)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def run_decode(c, q, bt, cl, scale, hq, **kw):
    out = torch.full_like(q, float("nan"), device=DEV)
    P.pa_q8_decode(out, q.to(DEV), dev(c.raw), dev(bt), dev(cl), scale, hq, c.hkv, c.d, c.b, **kw)
    torch.cuda.synchronize()
    return out


def check_decode(out, c, q, bt, cl, scale, dtype):
    want, size, smax = M.decode(c, q.double().numpy(), bt, cl, scale)
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    tol = tolerance(dtype, c.d, want, size, smax, cl)
    bad = np.abs(got - want) > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.max(np.abs(got - want) / tol):.2f} x tolerance"


LENS = [[1, 16, 17, 300], [0, 5, 67, 1000], [777, 2, 15, 0, 0, 31, 32, 33, 63, 64, 65]]
SHAPES = []
for dtype in ("f32", "f16", "bf16"):
    for d in (64, 128):
        for b in (16, 32):
            SHAPES.append((dtype, d, b, 8, 8, LENS[0]))
            SHAPES.append((dtype, d, b, 8, 2, LENS[1]))
            SHAPES.append((dtype, d, b, 16, 1, LENS[2]))
            SHAPES.append((dtype, d, b, 33, 3, [129, 64 * b + 7]))
SHAPES += [("bf16", 128, 16, 12, 3, [3000, 1, 17, 4096, 2222, 16]), ("f16", 128, 16, 5, 5, [1]),
           ("bf16", 128, 32, 64, 8, [2049, 513]), ("f32", 128, 32, 40, 1, [700, 40]),
           ("bf16", 128, 32, 32, 8, [1, 31, 32, 33, 5000, 40000]),        # cut over many CTAs
           ("bf16", 128, 16, 8, 1, [60000]), ("f32", 64, 16, 4, 2, [0, 3000, 0, 1, 0]),
           ("bf16", 128, 16, 40, 2, [1 + (i * 7) % 20 for i in range(500)]),   # many tiny sequences, G = 20
           ("f16", 128, 32, 8, 8, [0, 0, 0]),
           # few rows and many parts: the ways in which a unit's parts are merged
           ("f32", 128, 16, 1, 1, [6000]), ("bf16", 64, 32, 2, 1, [20000, 3]), ("f16", 128, 32, 5, 1, [30000, 7]),
           ("f16", 64, 16, 3, 1, [60000]), ("bf16", 128, 16, 3, 1, [9001, 9000]), ("f16", 64, 32, 16, 1, [40000]),
           ("bf16", 64, 16, 32, 2, [4077, 4077]), ("f16", 128, 32, 32, 8, [4096]), ("f32", 64, 16, 16, 2, [9000, 8000]),
           ("f16", 64, 32, 247, 19, [1664, 40, 1664, 1600]), ("bf16", 128, 16, 26, 2, [3000, 5000, 2990])]


@pytest.mark.parametrize("dtype,d,b,hq,hkv,lens", SHAPES, ids=lambda v: str(v).replace(" ", "")[:40])
def test_decode_matches_the_definition(dtype, d, b, hq, hkv, lens):
    c, q, bt, cl = decode_case(d + b + hq + sum(lens) % 89, dtype, d, b, hq, hkv, lens)
    scale = 1.0 / math.sqrt(d)
    out = run_decode(c, q, bt, cl, scale, hq)
    check_decode(out, c, q, bt, cl, scale, dtype)
    for s, t in enumerate(lens):
        if t == 0:
            assert not out[s].any()
    assert P.pa_device_errors() == 0


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_one_token_returns_its_value(dtype):
    c, q, bt, cl = decode_case(5, dtype, 128, 16, 8, 2, [1, 1, 1])
    out = run_decode(c, q, bt, cl, 0.3, 8).float().cpu().numpy()
    for s in range(3):
        v = c.values([bt[s, 0]])[0, :, 1, 0]             # [Hkv, d]
        for h in range(8):
            # p = 1 of a sum of 1: V8 * vs exactly, but for the output's rounding
            want = torch.from_numpy(v[h // 4]).to(TD[dtype]).float().numpy()
            assert np.array_equal(out[s, h], want)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_scales_of_any_value(dtype, d):
    """Scales that are no powers of two, and that differ by 2^24 between blocks: the
    block with the small values carries the weight, or the large ones do."""
    hq, hkv, b = 6, 2, 16
    c, q, bt, cl = decode_case(11, dtype, d, b, hq, hkv, [400, 39, 16], stale=False)
    rng = np.random.default_rng(1)
    c.scales[...] = rng.uniform(0.001, 0.02, size=c.scales.shape)
    check_decode(run_decode(c, q, bt, cl, 0.1, hq), c, q, bt, cl, 0.1, dtype)
    c.scales[..., 1] *= 2.0 ** rng.integers(-24, 1, size=c.scales.shape[:2])
    check_decode(run_decode(c, q, bt, cl, 0.1, hq), c, q, bt, cl, 0.1, dtype)
    c.scales[bt[0, 3]] = 0.0                              # a block that stands for zeros
    c.scales[bt[1, 0]] = 0.0
    check_decode(run_decode(c, q, bt, cl, 0.1, hq), c, q, bt, cl, 0.1, dtype)
    c.scales[..., 1] = 2.0 ** -126                        # the smallest scale
    out = run_decode(c, q, bt, cl, 0.1, hq)
    if dtype == "bf16":
        check_decode(out, c, q, bt, cl, 0.1, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_scores_that_grow_and_fall(dtype):
    """One token far above the rest early, late or in the middle; scores of +-500."""
    hq, hkv, b, d = 4, 2, 16, 128
    c, q, bt, cl = decode_case(12, dtype, d, b, hq, hkv, [900, 900, 900, 20], stale=False)
    for s, at in enumerate((0, 899, 430)):
        ids, row = bt[s, at // b], at % b
        for h in range(hkv):
            qd = q[s, h * 2].double().numpy()
            c.codes[ids, h, 0, row] = M.encode(np.clip(np.sign(qd) * 448.0, -448, 448))
    check_decode(run_decode(c, q, bt, cl, 1.0, hq), c, q, bt, cl, 1.0, dtype)
    # every score falls, or grows, from token to token
    for sign in (1.0, -1.0):
        c, q, bt, cl = decode_case(13, dtype, d, b, hq, hkv, [448, 100], stale=False)
        q[:] = 0.25
        c.scales[...] = 2.0 ** -4
        for s, t in enumerate((448, 100)):
            for tok in range(t):
                c.codes[bt[s, tok // b], :, 0, tok % b] = M.encode(np.full((hkv, d), sign * (tok - 200.0)))
        check_decode(run_decode(c, q, bt, cl, 0.05, hq), c, q, bt, cl, 0.05, dtype)


@pytest.mark.parametrize("mag", [2.0 ** -20, 2.0 ** 9, 2.0 ** 14])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_queries_of_any_magnitude(dtype, mag):
    c, q, bt, cl = decode_case(14, dtype, 64, 32, 4, 2, [200, 33, 64], stale=False)
    q = (q.double() * mag).clamp(-6e4, 6e4).to(TD[dtype])
    q[0, 1] = 0                                          # a zero row: the mean of V
    scale = 0.125 / mag
    check_decode(run_decode(c, q, bt, cl, scale, 4), c, q, bt, cl, scale, dtype)


def test_nan_codes_make_only_their_outputs_nan():
    hq, hkv, b, d = 8, 2, 16, 128
    c, q, bt, cl = decode_case(15, "bf16", d, b, hq, hkv, [100, 100, 100], stale=False)
    c.codes[bt[1, 2], 0, 0, 5, 7] = 0x7F                  # a key of sequence 1, kv head 0
    c.codes[bt[2, 3], 1, 1, 9, 33] = 0xFF                 # a value of sequence 2, kv head 1
    out = run_decode(c, q, bt, cl, 0.1, hq)
    nan = torch.isnan(out).cpu().numpy()
    want = np.zeros((3, hq, d), dtype=bool)
    want[1, :4] = True
    want[2, 4:, 33] = True
    assert np.array_equal(nan, want)


def test_entries_outside_the_pool_read_zeros():
    hq, hkv, b, d = 8, 4, 16, 128
    c, q, bt, cl = decode_case(16, "f16", d, b, hq, hkv, [200, 50, 90], stale=False)
    bt[0, 3], bt[1, 0], bt[2, 5], bt[2, 1] = -1, len(c.raw), 2 ** 31 - 1, -2 ** 31
    check_decode(run_decode(c, q, bt, cl, 0.1, hq), c, q, bt, cl, 0.1, "f16")
    assert P.pa_device_errors() == 0


def test_lengths_outside_the_table_are_clamped():
    c, q, bt, cl = decode_case(17, "bf16", 64, 16, 4, 4, [64, 48, 20], stale=False)
    bt = bt[:, :3].copy()
    cl = np.array([64, 10 ** 9, -7], dtype=np.int32)
    check_decode(run_decode(c, q, bt, cl, 0.1, 4), c, q, bt, np.array([48, 48, 0]), 0.1, "bf16")


def test_workspace_contents_do_not_matter_and_results_repeat():
    hq, hkv, b, d = 16, 4, 16, 128
    c, q, bt, cl = decode_case(18, "bf16", d, b, hq, hkv, [9000, 3, 700, 12000])
    n = P.pa_q8_decode_workspace_size(4, hq, hkv, d, b, bt.shape[1])
    first = run_decode(c, q, bt, cl, 0.09, hq)
    for fill in (0, 0xFF, 0x7F):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        assert torch.equal(run_decode(c, q, bt, cl, 0.09, hq, workspace=ws), first)
        assert torch.equal(run_decode(c, q, bt, cl, 0.09, hq, workspace=ws), first)
    with pytest.raises(P.PagedKVError):
        run_decode(c, q, bt, cl, 0.09, hq, workspace=torch.empty(n - 16, dtype=torch.uint8, device=DEV))


def test_block_permutation_is_bitwise_invariant():
    hq, hkv, b, d = 16, 4, 32, 64
    c, q, bt, cl = decode_case(19, "f16", d, b, hq, hkv, [900, 33, 400])
    a = run_decode(c, q, bt, cl, 0.08, hq)
    perm = np.random.default_rng(1).permutation(len(c.raw))
    raw = np.empty_like(c.raw)
    raw[perm] = c.raw
    bt2 = np.where(bt >= 0, perm[np.maximum(bt, 0)], bt).astype(np.int32)
    assert torch.equal(run_decode(M.Cache(raw, hkv, b, d), q, bt2, cl, 0.08, hq), a)


def test_decode_in_graphs_that_share_a_workspace_and_on_a_side_stream():
    hq, hkv, b, d = 32, 4, 16, 128
    c, q, bt, cl = decode_case(20, "bf16", d, b, hq, hkv, [5000, 20000, 1, 700], stale=False)
    q, cache, bt_d, cl_d = q.to(DEV), dev(c.raw), dev(bt), dev(cl)
    ws = torch.empty(P.pa_q8_decode_workspace_size(4, hq, hkv, d, b, bt.shape[1]), dtype=torch.uint8, device=DEV)
    outs = [torch.empty_like(q) for _ in range(2)]
    s = torch.cuda.Stream()

    def call(out, scale, stream=None):
        P.pa_q8_decode(out, q, cache, bt_d, cl_d, scale, hq, hkv, d, b, workspace=ws, stream=stream)

    with torch.cuda.stream(s):
        call(outs[0], 0.1)
    torch.cuda.synchronize()
    graphs = []
    for out, scale in zip(outs, (0.1, 0.05)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call(out, scale)
        graphs.append(g)
    gen = torch.Generator(device=DEV).manual_seed(2)
    for _ in range(4):
        q.copy_(torch.randn(q.shape, device=DEV, generator=gen).to(q.dtype))
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for out, scale in zip(outs, (0.1, 0.05)):
            want = torch.empty_like(q)
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            # on another stream, with a workspace of the binding's own
            P.pa_q8_decode(want, q, cache, bt_d, cl_d, scale, hq, hkv, d, b, stream=side)
            torch.cuda.synchronize()
            assert torch.equal(out, want)
    assert P.pa_device_errors() == 0


def test_two_decodes_at_once():
    hq, hkv, b, d = 8, 8, 16, 128
    cases = [decode_case(30 + i, "f16", d, b, hq, hkv, [2000 + i, 300, 1500]) for i in range(2)]
    want = [run_decode(*x, 0.1, hq) for x in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    ins = [(x[1].to(DEV), dev(x[0].raw), dev(x[2]), dev(x[3])) for x in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = [torch.empty_like(w) for w in want]
        torch.cuda.synchronize()
        for o, (q, cache, bt, cl), st in zip(outs, ins, streams):
            P.pa_q8_decode(o, q, cache, bt, cl, 0.1, hq, hkv, d, b, stream=st)
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_a_short_wait_limit_returns_and_the_next_call_is_right():
    hq, hkv, b, d = 64, 8, 16, 128
    # empty sequences behind the real ones: a long walk before any work item, so the
    # consumers' first wait surely outlasts 1 ns
    c, q, bt, cl = decode_case(21, "bf16", d, b, hq, hkv, [30000, 5000, 17], stale=False)
    q = torch.cat([q, torch.zeros(16384, hq, d, dtype=q.dtype)])
    bt = np.concatenate([bt, np.full((16384, bt.shape[1]), -1, dtype=np.int32)])
    cl = np.concatenate([cl, np.zeros(16384, dtype=np.int32)])
    P.pa_set_wait_limit_ns(1)
    try:
        run_decode(c, q, bt, cl, 0.1, hq)
        flags = P.pa_device_errors()
    finally:
        P.pa_set_wait_limit_ns(0)
    assert flags and flags & ~(P.PA_DEVERR_TIMEOUT_FULL | P.PA_DEVERR_TIMEOUT_EMPTY) == 0
    out = run_decode(c, q, bt, cl, 0.1, hq)
    assert P.pa_device_errors() == 0
    check_decode(out[:3], c, q[:3], bt[:3], cl[:3], 0.1, "bf16")


def test_a_cache_past_four_gigabytes():
    """Offsets past 32 bits: the sequence's blocks lie at the end of a 5 GB pool."""
    hq, hkv, b, d = 8, 8, 32, 128
    n = 5 * 2 ** 30 // M.block_bytes(hkv, b, d)
    cache = P.alloc_q8_cache(n, hkv, d, b)
    c, q, bt, cl = decode_case(22, "bf16", d, b, hq, hkv, [300, 33], stale=False)
    m = len(c.raw)
    cache[n - m:] = dev(c.raw)
    out = torch.empty_like(q, device=DEV)
    big = np.where(bt >= 0, bt + (n - m), bt).astype(np.int32)
    P.pa_q8_decode(out, q.to(DEV), cache, dev(big), dev(cl), 0.1, hq, hkv, d, b)
    check_decode(out, c, q, bt, cl, 0.1, "bf16")
    k, v = torch.randn(3, hkv, d, device=DEV), torch.randn(3, hkv, d, device=DEV)
    cl2, qs = np.array([302, 34], dtype=np.int32), np.array([0, 2, 3], dtype=np.int32)
    bt2 = np.concatenate([bt, np.full((2, 1), -1, dtype=np.int32)], axis=1)
    bt2[0, 9], bt2[1, 1] = bt[0, 9], bt[1, 1]
    M.append(c, k.double().cpu().numpy(), v.double().cpu().numpy(), bt2, cl2, qs)
    P.pa_q8_append(k, v, cache, dev(np.where(bt2 >= 0, bt2 + (n - m), bt2).astype(np.int32)), dev(cl2), b,
                   query_start=dev(qs))
    assert torch.equal(cache[n - m:].cpu(), torch.from_numpy(c.raw))
    assert not cache[:n - m].any()


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_softmax_scales_of_any_sign(dtype, scale):
    c, q, bt, cl = decode_case(23, dtype, 64, 16, 6, 2, [700, 1, 33, 0], spread=20.0, exps=(-6, -4))
    check_decode(run_decode(c, q, bt, cl, scale, 6), c, q, bt, cl, scale, dtype)


@pytest.mark.parametrize("dtype,hq,hkv", [("f16", 13, 1), ("f32", 30, 2), ("bf16", 17, 1)])
def test_many_short_sequences_of_wide_groups(dtype, hq, hkv):
    """Units of one stage with more than 8 rows, empty ones between them."""
    lens = [(i * 11) % 37 for i in range(350)] + [1200]
    c, q, bt, cl = decode_case(24, dtype, 128, 16, hq, hkv, lens)
    check_decode(run_decode(c, q, bt, cl, 0.1, hq), c, q, bt, cl, 0.1, dtype)


def test_infinite_and_nan_queries_stay_in_their_rows():
    c, q, bt, cl = decode_case(25, "f16", 128, 16, 8, 2, [900, 20], stale=False)
    bad = q.clone()
    bad[0, 3, 5], bad[1, 6, 0] = float("nan"), float("inf")
    got = run_decode(c, bad, bt, cl, 0.1, 8)
    assert got[0, 3].isnan().all() and got[1, 6].isnan().all()
    got[0, 3] = got[1, 6] = 0                             # the other rows: as without them
    want, size, smax = M.decode(c, q.double().numpy(), bt, cl, 0.1)
    want[0, 3] = want[1, 6] = 0
    assert (np.abs(got.double().cpu().numpy() - want) <= tolerance("f16", 128, want, size, smax, cl)).all()


def test_views_at_an_offset_and_refused_tensors():
    """Slices of larger buffers: rows of q and out, blocks of a cache; nothing around them
    changes.  Strided and misaligned ones are refused."""
    hq, hkv, b, d = 4, 2, 16, 64
    c, q, bt, cl = decode_case(26, "f16", d, b, hq, hkv, [70, 9, 33], stale=False)
    want = run_decode(c, q, bt, cl, 0.1, hq)
    pool = torch.full((len(c.raw) + 4, c.raw.shape[1]), 0x5A, dtype=torch.uint8, device=DEV)
    cache = pool[2:-2]
    cache.copy_(dev(c.raw))
    codes, scales = P.q8_views(cache, hkv, d, b)
    assert torch.equal(scales.cpu(), torch.from_numpy(c.scales.copy()))
    assert torch.equal(codes.view(torch.uint8).cpu(), torch.from_numpy(c.codes.copy()))
    qq = torch.zeros(5, hq, d, dtype=torch.float16, device=DEV)
    qq[1:4] = q.to(DEV)
    outs = torch.full((5, hq, d), 7.0, dtype=torch.float16, device=DEV)
    tables, lens = torch.cat([dev(bt)[:1], dev(bt)]), torch.cat([dev(cl)[:1], dev(cl)])
    P.pa_q8_decode(outs[1:4], qq[1:4], cache, tables[1:], lens[1:], 0.1, hq, hkv, d, b)
    assert torch.equal(outs[1:4], want) and (outs[0] == 7).all() and (outs[4] == 7).all()
    k = torch.randn(5, hkv, d, device=DEV, dtype=torch.float16)
    cl2 = cl + 1
    bt2 = np.concatenate([bt, np.full((3, 1), -1, dtype=np.int32)], axis=1)
    P.pa_q8_append(k[1:4], k[2:], cache, dev(bt2), dev(cl2), b)
    M.append(c, k[1:4].double().cpu().numpy(), k[2:].double().cpu().numpy(), bt2, cl2)
    assert np.array_equal(cache.cpu().numpy(), c.raw)
    assert (pool[:2] == 0x5A).all() and (pool[-2:] == 0x5A).all()
    with pytest.raises(ValueError, match="contiguous"):
        P.pa_q8_decode(outs[::2], qq[::2], cache, dev(bt), dev(cl), 0.1, hq, hkv, d, b)
    with pytest.raises(ValueError, match="contiguous"):
        P.pa_q8_append(k[:3], k[:3], cache, torch.cat([dev(bt2)] * 2, 1)[:, ::2][:, :bt2.shape[1]], dev(cl2), b)
    flat = torch.zeros(3 * hq * d + 8, dtype=torch.float16, device=DEV)
    with pytest.raises(P.PagedKVError):                   # 2 bytes off a 16-byte boundary
        P.pa_q8_decode(want, flat[1:1 + 3 * hq * d].view(3, hq, d), cache, dev(bt), dev(cl), 0.1, hq, hkv, d, b)
    with pytest.raises(ValueError, match="CUDA"):
        P.pa_q8_decode(want, q.to(DEV), cache, torch.from_numpy(bt), dev(cl), 0.1, hq, hkv, d, b)


def test_empty_batches():
    cache = P.alloc_q8_cache(3, 2, 64, 16)
    e = torch.zeros(0, 4, 64, device=DEV)
    bt, cl = torch.zeros(0, 2, dtype=torch.int32, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV)
    P.pa_q8_decode(e, e, cache, bt, cl, 0.1, 4, 2, 64, 16)
    P.pa_q8_append(e[:, :2].contiguous(), e[:, :2].contiguous(), cache, bt, cl, 16)
    one = torch.zeros(1, 2, dtype=torch.int32, device=DEV)
    P.pa_q8_append(e[:, :2].contiguous(), e[:, :2].contiguous(), cache, one, one[0, :1].contiguous(), 16,
                   query_start=torch.zeros(2, dtype=torch.int32, device=DEV))
    assert not cache.any()


# ---- append ------------------------------------------------------------------
def append_case(seed, dtype, d, b, hkv, old, new, spread=0.7, extra=3):
    """A cache whose sequences hold `old` rows, and rows for `new` more."""
    rng = np.random.default_rng(seed)
    total = [o + n for o, n in zip(old, new)]
    nb = sum((t + b - 1) // b for t in total) + extra
    bt, _ = W.random_tables(rng, total, b, nb, pad=1)
    c = random_cache(rng, nb, hkv, b, d)
    c.raw[:, hkv * 2 * b * d + hkv * 8:] = 0xA5           # the padding stays as it is
    n = sum(new)
    x = rng.standard_normal((2, n, hkv, d)) * np.exp(spread * rng.standard_normal((2, n, hkv, 1)))
    k, v = (torch.from_numpy(a).to(TD[dtype]) for a in x)
    qs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return c, k, v, bt, np.array(total, dtype=np.int32), qs


def run_append(c, k, v, bt, cl, qs):
    cache = dev(c.raw)
    P.pa_q8_append(k.to(DEV), v.to(DEV), cache, dev(bt), dev(cl), c.b, query_start=None if qs is None else dev(qs))
    torch.cuda.synchronize()
    return cache.cpu().numpy()


def check_append(c, k, v, bt, cl, qs):
    got = run_append(c, k, v, bt, cl, qs)
    M.append(c, k.double().numpy(), v.double().numpy(), bt, cl, qs)
    bad = got != c.raw
    assert not bad.any(), f"{bad.sum()} bytes differ, blocks {np.nonzero(bad.any(1))[0][:8]}"


RUNS = [([0, 0, 0], [50, 1, 33]), ([5, 31, 32, 0, 16, 15, 47, 100], [1, 2, 3, 0, 16, 1, 40, 17]),
        ([0] * 7, [0, 0, 3, 0, 0, 0, 0]), ([7], [1]), ([13], [300])]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("b", [16, 32])
@pytest.mark.parametrize("hkv", [1, 3])
@pytest.mark.parametrize("run", range(len(RUNS)))
def test_append_matches_the_definition(dtype, d, b, hkv, run):
    old, new = RUNS[run]
    check_append(*append_case(40 + run, dtype, d, b, hkv, old, new))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_append_one_token_for_each_sequence(dtype):
    rng = np.random.default_rng(6)
    old = rng.integers(0, 70, size=301)
    c, k, v, bt, cl, qs = append_case(60, dtype, 128, 32, 2, old.tolist(), [1] * 301)
    a = run_append(c, k, v, bt, cl, qs)
    check_append(c, k, v, bt, cl, None)
    assert np.array_equal(a, c.raw)


def test_append_many_sequences_some_without_rows():
    rng = np.random.default_rng(7)
    old, new = rng.integers(0, 40, size=1500), rng.integers(0, 4, size=1500) * (rng.random(1500) < 0.3)
    new[100:400] = 0                                      # a long stretch without rows
    check_append(*append_case(61, "bf16", 64, 16, 1, old.tolist(), new.tolist()))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_append_extreme_values(dtype):
    """The type's largest and smallest values, zeros, infinities and NaN."""
    c, k, v, bt, cl, qs = append_case(62, dtype, 64, 16, 2, [3, 0, 18, 0, 30], [10, 40, 20, 16, 1])
    big, tiny = torch.finfo(TD[dtype]).max, torch.finfo(TD[dtype]).smallest_normal
    k[0, 0, 3], k[12, 1, 5], v[20, 0, 0], v[21, 1, 1] = big, -big, tiny, -tiny / 8
    k[30:50] = 0
    v[30:70, 0] = tiny
    v[30:70, 1] = tiny / 4
    k[5, 0, 1], k[5, 0, 2], v[6, 1, 7], v[75, 0, 9] = float("inf"), float("nan"), float("-inf"), float("nan")
    k[60:76, 0] = float("inf")                            # a whole tile without a finite value
    v[86] = 1e-3
    check_append(c, k, v, bt, cl, qs)


def test_append_grows_scales_again_and_again():
    """Row by row, each larger than the one before: every row rounds the others again."""
    hkv, b, d = 2, 16, 64
    rng = np.random.default_rng(8)
    c = random_cache(rng, 4, hkv, b, d)
    cache = dev(c.raw)
    bt = np.array([[2, 1, 3]], dtype=np.int32)
    for t in range(40):
        k = torch.from_numpy(rng.standard_normal((1, hkv, d)) * 2.0 ** (t - 20)).to(torch.bfloat16)
        v = torch.from_numpy(rng.standard_normal((1, hkv, d)) * 2.0 ** (20 - t)).to(torch.bfloat16)
        cl = np.array([t + 1], dtype=np.int32)
        P.pa_q8_append(k.to(DEV), v.to(DEV), cache, dev(bt), dev(cl), b)
        M.append(c, k.double().numpy(), v.double().numpy(), bt, cl)
    assert np.array_equal(cache.cpu().numpy(), c.raw)


def test_append_to_scales_that_are_no_powers_of_two():
    """A caller's own scale stays where it is large enough (x / s is then a division)."""
    c, k, v, bt, cl, qs = append_case(63, "f32", 128, 16, 2, [5, 9, 3], [4, 2, 6])
    c.scales[...] = np.float32(0.37)                      # above what the rows need
    raw = c.raw.copy()
    got = M.Cache(run_append(c, k, v, bt, cl, qs), 2, 16, 128)
    assert (got.scales == np.float32(0.37)).all()
    # the quotient is rounded to fp32 before the code's rounding: equal but where a value
    # lies within 2^-24 of a border between two codes
    M.append(c, k.double().numpy(), v.double().numpy(), bt, cl, qs)
    near = np.abs(M.CODES[got.codes] - M.CODES[c.codes]) <= 2.0 ** -3 * np.abs(M.CODES[c.codes])
    assert near.all() and (got.codes != c.codes).mean() < 1e-5
    assert (got.raw != raw).any()


def test_append_skips_padding_and_bad_places():
    c, k, v, bt, cl, qs = append_case(64, "bf16", 128, 16, 2, [5, 9, 30, 8], [4, 20, 6, 3])
    k, v = torch.cat([k, k[:9]]), torch.cat([v, v[:9]])   # rows behind the last sequence
    bt[1, 1] = -1                                         # blocks outside the pool
    bt[2, 2] = len(c.raw)
    cl[3] = 2                                             # shorter than its new rows: position -1
    check_append(c, k, v, bt, cl, qs)
    c, k, v, bt, cl, qs = append_case(65, "f16", 64, 16, 2, [40, 3], [30, 5])
    bt = bt[:, :3].copy()                                 # a table that ends before the rows do
    check_append(c, k, v, bt, cl, qs)
    c, k, v, bt, cl, qs = append_case(66, "f16", 64, 16, 2, [1, 3], [30, 5])
    check_append(c, k, v, bt, np.array([0, -4], dtype=np.int32), np.array([0, 1, 2], dtype=np.int32))


def test_append_in_a_graph():
    hkv, b, d, S = 4, 32, 128, 5
    rng = np.random.default_rng(9)
    c = random_cache(rng, 30, hkv, b, d)
    bt = rng.permutation(30).reshape(S, 6).astype(np.int32)
    cl = np.array([40, 0, 64, 31, 7], dtype=np.int32)
    cache, bt_d, cl_d = dev(c.raw), dev(bt), dev(cl)
    k, v = torch.zeros(S, hkv, d, device=DEV, dtype=torch.float16), torch.zeros(S, hkv, d, device=DEV, dtype=torch.float16)
    scratch = cache.clone()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        P.pa_q8_append(k, v, scratch, bt_d, cl_d, b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        P.pa_q8_append(k, v, cache, bt_d, cl_d, b)
    for _ in range(40):
        cl += 1
        x = rng.standard_normal((2, S, hkv, d)) * np.exp(rng.standard_normal((2, S, 1, 1)))
        k.copy_(torch.from_numpy(x[0]))
        v.copy_(torch.from_numpy(x[1]))
        cl_d.copy_(torch.from_numpy(cl))
        g.replay()
        torch.cuda.synchronize()
        M.append(c, k.double().cpu().numpy(), v.double().cpu().numpy(), bt, cl)
    assert np.array_equal(cache.cpu().numpy(), c.raw)


def test_appends_on_two_streams_at_once():
    hkv, b, d = 3, 16, 128
    jobs = []
    for i, st in enumerate([torch.cuda.Stream(), torch.cuda.Stream()]):
        c, k, v, bt, cl, qs = append_case(70 + i, "bf16", d, b, hkv, [5, 40, 0], [100, 3, 17 + i])
        jobs.append((c, k, v, bt, cl, qs, dev(c.raw), [x.to(DEV) for x in (k, v)] + [dev(x) for x in (bt, cl, qs)], st))
    torch.cuda.synchronize()
    for c, k, v, bt, cl, qs, cache, (kd, vd, btd, cld, qsd), st in jobs:
        P.pa_q8_append(kd, vd, cache, btd, cld, b, query_start=qsd, stream=st)
    torch.cuda.synchronize()
    for c, k, v, bt, cl, qs, cache, _, _ in jobs:
        M.append(c, k.double().numpy(), v.double().numpy(), bt, cl, qs)
        assert np.array_equal(cache.cpu().numpy(), c.raw)


# ---- block moves ---------------------------------------------------------------
def test_copy_and_swap_move_codes_and_scales():
    rng = np.random.default_rng(10)
    c = random_cache(rng, 9, 3, 16, 64)
    cache = dev(c.raw)
    pairs = np.array([[2, 7], [0, 8], [-1, 3], [1, 9], [9, 1]], dtype=np.int32)   # three out of range
    P.pa_q8_copy_blocks(cache, dev(pairs))
    want = c.raw.copy()
    want[7], want[8] = c.raw[2], c.raw[0]
    assert np.array_equal(cache.cpu().numpy(), want)
    host = P.alloc_q8_cache(4, 3, 64, 16, device="cpu", pin_memory=True)
    P.pa_q8_swap_blocks(cache, host, dev(np.array([[7, 0], [3, 2]], dtype=np.int32)))
    torch.cuda.synchronize()
    assert np.array_equal(host.numpy()[[0, 2]], want[[7, 3]]) and not host.numpy()[[1, 3]].any()
    P.pa_q8_swap_blocks(host, cache, dev(np.array([[2, 0]], dtype=np.int32)))
    torch.cuda.synchronize()
    want[0] = want[3]
    assert np.array_equal(cache.cpu().numpy(), want)
