"""The 8-bit decode with V scales that differ by many binades from block to block: what a
block adds is its probability times its scale, and neither alone may set the precision.

Tolerance, elementwise, as in tests/test_gpu_q8.py with the score's error for these inputs:
    u_T max(|out|, N_T) + A (r + 2 ds + (n / 16 + 8) 2^-23 + 14 n 2^-31) + 8 * 2^-150
ds   queries are +-a and keys +-c, small dyadic numbers: their products and sums are exact,
     so a score is off by the roundings of the softmax scale, of log2(e), of two products
     and of the difference to the reference, 2^-24 each; a change of references adds two
     more, and there are at most four: 13 * 2^-24 S
14 n 2^-31  a product p vs enters to within 2^-39 of the reference, which is less than 2^8
     times the row's largest product (scales within 6 binades of each other, a mantissa
     above 1/2, and one divided out); values of n tokens differ by at most 14 (codes of 32
     to 448)
8 * 2^-150  below fp32's normal range each of four warps' sums, their merge, the quotient
     and the last products is rounded to a multiple of 2^-149"""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_79_gb300 as P
import workloads as W
from tests import q8_model as M
from tests.test_gpu_q8 import TD, dev, run_decode

pytestmark = pytest.mark.gpu


def check(out, c, q, bt, cl, scale, dtype):
    want, size, smax = M.decode(c, q.double().numpy(), bt, cl, scale)
    got = out.double().cpu().numpy()
    f32, t = dtype == "f32", torch.finfo(TD[dtype])
    n = np.asarray(cl)[:, None, None]
    r = (2.0 ** -21 if f32 else 2.0 ** -11) + 2.0 ** -22 + 2.0 ** -23
    ds = 13 * 2.0 ** -24 * smax[..., None]
    tol = t.eps / 2 * np.maximum(np.abs(want), t.smallest_normal) + 8 * 2.0 ** -150 + \
        size * (r + 2 * ds + (n / 16 + 8) * 2.0 ** -23 + 14 * n * 2.0 ** -31)
    big = np.abs(want) - tol >= t.max * (1 + t.eps / 4)       # rounds to infinity
    assert (np.isposinf(got[big]) == (want[big] > 0)).all() and np.isinf(got[big]).all()
    ok = np.abs(want) + tol < t.max
    bad = np.abs(got[ok] - want[ok]) > tol[ok]
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got[ok] - want[ok]) / tol[ok]):.3g} x"
    return got, want


def two_level_case(seed, dtype, d, b, group, ratio, mantissas, hkv=2):
    """Blocks whose V scales lie `ratio` binades above the others', and whose scores lie so
    far below them that both add the same to the first head of each group, a fraction to
    some heads and nearly all to others."""
    rng = np.random.default_rng(seed)
    lens = [2 * b, 2 * b, 700, 700, 701, 1300, 64, 5 * b]
    nbs = [-(-t // b) for t in lens]
    bt, _ = W.random_tables(rng, lens, b, sum(nbs) + 3, pad=1)
    c = M.Cache(np.zeros((sum(nbs) + 3, M.block_bytes(hkv, b, d)), dtype=np.uint8), hkv, b, d)
    code = rng.uniform(32, 448, size=c.codes.shape) * rng.choice([-1.0, 1.0], size=c.codes.shape)
    c.codes[...] = M.encode(code)
    signs = rng.choice([-1.0, 1.0], size=(len(lens), hkv, d))
    a = np.array([1.0, 1.25, 0.5, 2.0, 1.125, 0.75, 1.5, 1.0, 0.875, 1.0, 1.25, 3.0])[:group]
    q = (signs[:, :, None] * a[None, None, :, None]).reshape(len(lens), hkv * group, d)
    ks = 2.0 ** -5
    c.scales[..., 0] = ks
    for s, nb in enumerate(nbs):
        where = [[0], [nb - 1], [0], [nb - 1], [nb // 2], list(range(0, nb, 2)), [1], [0, 2]][s]
        for j in range(nb):
            large = j in where
            c.codes[bt[s, j], :, 0] = M.encode(signs[s] * (0.0 if large else 8.0))[:, None]
            m = rng.uniform(1, 2, size=hkv) if mantissas else 1.0
            c.scales[bt[s, j], :, 1] = m * 2.0 ** (ratio - 6 if large else -6)
    scale = float(np.float32(ratio * math.log(2) / (8 * d * ks)))
    return c, torch.from_numpy(q).to(TD[dtype]), bt, np.array(lens, dtype=np.int32), scale


@pytest.mark.parametrize("mantissas", [False, True], ids=["powers", "any"])
@pytest.mark.parametrize("ratio", [10, 17, 20, 24, 32, 40, 80])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d,b,group", [(128, 16, 3), (64, 16, 4), (128, 32, 12), (64, 32, 12)])
def test_blocks_with_small_scales_carry_the_weight(d, b, group, dtype, ratio, mantissas):
    c, q, bt, cl, scale = two_level_case(ratio + d, dtype, d, b, group, ratio, mantissas)
    got, want = check(run_decode(c, q, bt, cl, scale, 2 * group), c, q, bt, cl, scale, dtype)
    # head 1: the blocks with the large scales count for nearly nothing, the others are there
    if ratio >= 40:
        assert np.median(np.abs(want[:, 1])) < 8.0 and (np.abs(got[:, 1]) > 2.0 ** -10).mean() > 0.9
    assert P.pa_device_errors() == 0


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_a_dead_block_with_the_largest_scale_in_one_stage(dtype):
    """32 tokens, one stage: a block of scale 2^20 and scores 60 lower, one of 2^-20."""
    for large_first in (True, False):
        c, q, bt, cl, _ = two_level_case(7, dtype, 128, 16, 1, 40, False)
        bt, cl, q = bt[:1], cl[:1], q[:1]
        low, high = bt[0, :2] if large_first else bt[0, 1::-1]
        k = np.sign(q[0].double().numpy())[:, None]
        c.codes[low, :, 0], c.codes[high, :, 0] = M.encode(0.0 * k), M.encode(8.0 * k)
        c.scales[low, :, 1], c.scales[high, :, 1] = 2.0 ** 20, 2.0 ** -20
        scale = float(np.float32(60.0 / (8 * 128 * 2.0 ** -5)))
        got, want = check(run_decode(c, q, bt, cl, scale, 2), c, q, bt, cl, scale, dtype)
        assert (np.abs(want) > 0).all() and np.median(np.abs(got)) > 2.0 ** -17


@pytest.mark.parametrize("exponent", [-126, -120, -140])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_the_smallest_scales(dtype, exponent):
    c, q, bt, cl, scale = two_level_case(9, dtype, 128, 16, 3, 10, False)
    c.scales[..., 1] = 2.0 ** exponent
    got, want = check(run_decode(c, q, bt, cl, scale, 6), c, q, bt, cl, scale, dtype)
    if dtype == "f16":
        assert not got.any()                                  # all below its smallest number
    else:                                                     # a step above 0 or more: not lost
        seen = np.abs(want) > 1.5 * torch.finfo(TD[dtype]).smallest_normal * torch.finfo(TD[dtype]).eps
        assert seen.any() or (dtype, exponent) == ("bf16", -140)   # there all lie near or below one step, 2^-133
        assert got[seen].all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_scales_of_zero_among_others(dtype):
    """Blocks that stand for zeros carry most of the weight, or none, or all of it."""
    for group in (3, 12):
        c, q, bt, cl, scale = two_level_case(10, dtype, 128, 16, group, 24, True)
        c.scales[bt[2, 1:20], :, 1] = 0.0
        c.scales[bt[3, 43], :, 1] = 0.0
        c.scales[bt[5, ::2], :, 1] = 0.0
        c.scales[bt[6, :4], :, 1] = 0.0
        out = run_decode(c, q, bt, cl, scale, 2 * group)
        check(out, c, q, bt, cl, scale, dtype)
        assert not out[6].any()


@pytest.mark.parametrize("above", [1, 20, 60, 100])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d,group,outside", [(128, 3, False), (64, 12, False), (128, 3, True)])
def test_blocks_of_zeros_that_score_highest(d, group, outside, dtype, above):
    """Scales of 0, or table entries outside the pool, `above` binades over scales that are all
    alike: what the others add is small, and all there is."""
    c, q, bt, cl, _ = two_level_case(13, dtype, d, 16, group, 10, False)
    c.scales[..., 1] = 2.0 ** -6
    for s, js in enumerate([[0], [1], [0, 43], list(range(0, 44, 3)), [20], [81], [0, 1, 2], [4]]):
        sign = np.sign(q[s].double().numpy())[::group, None]
        c.codes[bt[s], :, 0] = M.encode((-8.0 if outside else 0.0) * sign)
        c.codes[bt[s, js], :, 0] = M.encode((0.0 if outside else 8.0) * sign)
        c.scales[bt[s, js], :, 1] = 0.0
        if outside:
            bt[s, js] = len(c.raw) + 5
    scale = float(np.float32(above * math.log(2) / (8 * d * 2.0 ** -5)))
    check(run_decode(c, q, bt, cl, scale, 2 * group), c, q, bt, cl, scale, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [3, 12])
def test_scores_that_overflow_before_others_that_do_not(dtype, group):
    """Blocks whose scores are -inf (no weight), of large V scales, before and behind the
    rest: the others are as they are without them."""
    c, q, bt, cl, scale = two_level_case(12, dtype, 128, 16, group, 10, True)
    c.scales[..., 1] = 2.0 ** -6
    over = M.Cache(c.raw.copy(), c.hkv, c.b, c.d)
    dead = [[0], [1], list(range(40)), list(range(4, 44)), [0, 43], list(range(0, 82, 2)), [0, 1, 2], [4]]
    for s, js in enumerate(dead):
        sign = np.sign(q[s].double().numpy())[::group, None]
        c.codes[bt[s, js], :, 0], over.codes[bt[s, js], :, 0] = M.encode(-64.0 * sign), M.encode(-8.0 * sign)
        over.scales[bt[s, js], :, 0] = 2.0 ** 127        # the model: e^-27 of the rest at most
        over.scales[bt[s, js], :, 1] = 2.0 ** 20
    out = run_decode(over, q, bt, cl, scale, 2 * group)
    check(out, c, q, bt, cl, scale, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_scales_over_the_whole_range(dtype):
    """Every block its own scale, 2^-100 to 2^100, its scores so that all add alike; and
    scores in any order against the scales'."""
    hkv, b, d = 2, 16, 128
    for seed in range(4):
        c, q, bt, cl, _ = two_level_case(20 + seed, dtype, d, b, 2, 10, True)
        rng = np.random.default_rng(seed)
        signs = np.sign(q.double().numpy())[:, ::2]
        for s in range(len(cl)):
            for j in range(-(-int(cl[s]) // b)):
                e = int(rng.integers(-12, 13))                # scale 2^8e, score -8 e ln 2 + ...
                k = -e if seed < 2 else int(rng.integers(-12, 13))
                c.codes[bt[s, j], :, 0] = M.encode(signs[s] * k)[:, None]
                c.scales[bt[s, j], :, 1] = rng.uniform(1, 2, size=hkv) * 2.0 ** (8 * e)
        scale = float(np.float32(8 * math.log(2) / (d * 2.0 ** -5)))
        check(run_decode(c, q, bt, cl, scale, 4), c, q, bt, cl, scale, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,group,lens", [(64, 1, [30000, 40]), (128, 4, [20000]), (64, 12, [9000, 12000]),
                                          (128, 12, [30001])])
def test_far_scales_in_units_of_many_parts(dtype, d, group, lens):
    """As above in units that are merged from up to 38 parts and more: all blocks add alike
    (first head), so no part's weight may be lost."""
    hkv, b = 1, 16
    rng = np.random.default_rng(30 + d + group)
    nbs = [-(-t // b) for t in lens]
    bt, _ = W.random_tables(rng, lens, b, sum(nbs), pad=1)
    c = M.Cache(np.zeros((sum(nbs), M.block_bytes(hkv, b, d)), dtype=np.uint8), hkv, b, d)
    c.codes[...] = M.encode(rng.uniform(32, 448, size=c.codes.shape) * rng.choice([-1.0, 1.0], size=c.codes.shape))
    signs = rng.choice([-1.0, 1.0], size=(len(lens), d))
    a = np.array([1.0, 1.25, 0.5, 2.0, 1.125, 0.75, 1.5, 1.0, 0.875, 1.0, 1.25, 3.0])[:group]
    q = torch.from_numpy(signs[:, None] * a[None, :, None]).to(TD[dtype])
    c.scales[..., 0] = 2.0 ** -5
    for s, nb in enumerate(nbs):
        e = np.sort(rng.integers(-12, 13, size=nb))           # parts far apart from each other
        for j in range(nb):
            c.codes[bt[s, j], 0, 0] = M.encode(signs[s] * float(-e[j]))
            c.scales[bt[s, j], 0, 1] = rng.uniform(1, 2) * 2.0 ** (8 * int(e[j]))
    scale = float(np.float32(8 * math.log(2) / (d * 2.0 ** -5)))
    cl = np.array(lens, dtype=np.int32)
    check(run_decode(c, q, bt, cl, scale, group), c, q, bt, cl, scale, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("scale", [0.37, 1.9999998, 3.1e-3, 1.1754944e-38])
def test_one_token_of_any_scale_returns_its_value(dtype, scale):
    """p = 1 of a sum of 1.  The scale's mantissa leaves the product and comes back: its
    inverse, two products and the last one round, 2^-24 each; then the output."""
    c, q, bt, cl, _ = two_level_case(11, dtype, 128, 16, 3, 10, False)
    c.scales[..., 1] = np.float32(scale)
    cl[:] = 1
    got = run_decode(c, q, bt, cl, 0.1, 6).double().cpu().numpy()
    t = torch.finfo(TD[dtype])
    for s in range(len(cl)):
        v = c.values([bt[s, 0]])[0, :, 1, 0]                  # [Hkv, d]
        for h in range(6):
            want = v[h // 3]
            tol = t.eps / 2 * np.maximum(np.abs(want), t.smallest_normal) + 4 * 2.0 ** -24 * np.abs(want) + 2.0 ** -150
            assert (np.abs(got[s, h] - want) <= tol).all()
