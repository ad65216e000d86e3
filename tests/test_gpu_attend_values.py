"""pa_attend with values at the ends of their types, against the definition in 64 bits."""
import math

import pytest
import torch

import paged_kv_cache_79_gb300 as P
from tests.test_gpu_attend import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"


def rows_of(c, s):
    """Slots of sequence s's keys, in their order."""
    t = c.lens[s]
    ids = c.bt[s, :-(-t // c.B)].long()
    return (ids[:, None] * c.B + torch.arange(c.B, device=DEV)).reshape(-1)[:t]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("at", [0, 30000, 59999])
@pytest.mark.parametrize("below", [10.0, 17.75, 20.0])
@pytest.mark.parametrize("new", [1, 40])
def test_many_small_weights_under_a_dominant_one(dtype, at, below, new):
    """One key holds nearly all of the weight and a value of 0; the output is the 60,000 others',
    each e^-below of it.  (160 sequences over the same blocks, so that a CTA goes through most of
    one's keys: a part with small weights alone would take its base from them.)

    Tolerance: a weight is off by 2 delta + 2^-20 of itself (delta: the score, exact here but for
    the scale's rounding and one of the exponent's, 2^-22 of it each), half a step of the type for
    the weight, and in fp16, whose smallest step is 2^-24, by 2^-25 where the largest weight is at
    least 2^11: by 2^-36 of the largest.  T 2^-24 for the sums in fp32 (tensor cores may cut: as
    much again), half a step of the output, 2^-25 in fp16 for one below its normal range."""
    t = 60000
    c = Case([new], [t], 1, 1, 64, 16, dtype, seed=at + int(below), pad=0)
    slots = rows_of(c, 0)
    k, v = c.k.view(-1, 64), c.v.view(-1, 64)
    k[slots] = 0.0
    k[slots[at]] = below / 8                     # 64 of them times the scale, 1/8: `below`
    v[slots] = (v[slots].abs() + 0.5).to(c.dt)   # of one sign: errors that lean one way add up
    v[slots[at]] = 0.0
    c.bt = c.bt.expand(160, -1).contiguous()
    c.cl = c.cl.expand(160).contiguous()
    c.qs = torch.arange(161, dtype=torch.int32, device=DEV) * new
    c.n = 160 * new
    c.q = torch.ones(c.n, 1, 64, device=DEV, dtype=c.dt)
    out, lse = c.run(False)
    assert P.pa_device_errors() == 0
    score = float(k[slots[at], 0].double() * 8)
    total = 1.0 + (t - 1) * math.exp(-score)
    p = math.exp(-score) / total
    size = p * v[slots].double().sum(0)          # want: all of one sign
    half = torch.finfo(c.dt).eps / 2
    tol = size * (4 * score * 2.0 ** -22 + 2.0 ** -20 + t * 2.0 ** -23 + half) + size * half
    if dtype == "f16":
        tol = tol + 2.0 ** -36 / total * v[slots].double().sum(0) + 2.0 ** -25
    err = (out[:, 0].double() - size).abs()
    assert (err <= tol).all(), (float((err / tol).max()), float((err / size).max()))
    z = score + math.log(total)
    assert ((lse.double() - z).abs() <= t * 2.0 ** -24 + 2.0 ** -20 + z * 2.0 ** -21).all()


def definition(c, causal):
    """(out, lse) in 64 bits of a case with values that are not finite: hidden keys are left out."""
    out = torch.zeros(c.n, c.hq, c.d, device=DEV, dtype=torch.float64)
    lse = torch.full((c.n, c.hq), -math.inf, device=DEV, dtype=torch.float64)
    at = 0
    for s, (n, t) in enumerate(zip(c.new, c.lens)):
        slots = rows_of(c, s)
        for i in range(n):
            seen = t - n + i + 1 if causal else t
            for h in range(c.hq):
                kv = h * c.hkv // c.hq
                k, v = (x.view(-1, c.hkv, c.d)[slots[:seen], kv].double() for x in (c.k, c.v))
                sc = (k * c.q[at + i, h].double()).sum(-1) * c.scale
                z = torch.logsumexp(sc, 0)
                p = torch.exp(sc - z)
                out[at + i, h] = (torch.where(p[:, None] == 0, 0.0, p[:, None] * v)).sum(0)
                lse[at + i, h] = z
        at += n
    return out, lse


NANS = [0x7fffffff, -1, 0x7f800001, 0x7fc00000, -0x400000]     # bit patterns of fp32 NaN


def same_kind(got, want, tol):
    """NaN and infinities where the definition has them, the others within tol."""
    assert torch.equal(got.isnan(), want.isnan())
    inf = want.isinf()
    assert torch.equal(got[inf].double(), want[inf])
    fin = want.isfinite()
    assert (got.double() - want)[fin].abs().le((tol * torch.ones_like(want))[fin]).all()


def nan_of(bits):
    return torch.tensor(bits, dtype=torch.int32, device=DEV).view(torch.float32)


@pytest.mark.parametrize("bits", NANS)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("where", ["q", "k", "v"])
def test_nan_of_any_bits_fp32(bits, causal, d, where):
    """One NaN in a query, a key or a value: it reaches the rows that see it, and no other.

    Tolerance: scale * sum |q k| <= 12 in two tf32 terms (2^-21) and 132 roundings of 2^-24, twice
    that for a weight, times |v| <= 5: below 2^-9."""
    c = Case([33, 5], [70, 40], 4, 2, d, 16, "f32", seed=3, pad=0)
    flat = (c.q if where == "q" else c.k if where == "k" else c.v).view(-1, c.hq if where == "q" else c.hkv, d)
    row = 20 if where == "q" else int(rows_of(c, 0)[55])
    flat.view(torch.int32)[row, 1, 7] = bits
    want, want_lse = definition(c, causal)
    assert want.isnan().any() and not want.isnan().all()
    out, lse = c.run(causal)
    same_kind(out, want, 2.0 ** -9)
    assert torch.equal(lse.isnan(), want_lse.isnan())


@pytest.mark.parametrize("value", [math.inf, -math.inf])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("where", ["k", "v"])
def test_infinities_fp32(value, causal, where):
    """An infinite value makes its column infinite for the rows that see it; an infinite key gives a
    weight of 0 where its score is -inf, NaN where it is +inf."""
    c = Case([33, 5], [70, 40], 4, 2, 64, 16, "f32", seed=4, pad=0)
    (c.k if where == "k" else c.v).view(-1, 2, 64)[int(rows_of(c, 0)[55]), 1, 7] = value
    want, _ = definition(c, causal)
    out, _ = c.run(causal)
    same_kind(out, want, 2.0 ** -9)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_values_that_every_row_sees(dtype, value):
    """Without a mask every row of the sequence sees the value, and no other column changes.
    Tolerance: as above, and half a step of the type twice for a weight, once for the output."""
    c = Case([33, 5], [70, 40], 4, 2, 128, 16, dtype, seed=5, pad=0)
    c.v.view(-1, 2, 128)[int(rows_of(c, 0)[55]), 1, 7] = value
    want, _ = definition(c, False)
    out, _ = c.run(False)
    same_kind(out, want, {"f32": 2.0 ** -9, "f16": 2.0 ** -6, "bf16": 2.0 ** -3}[dtype])


@pytest.mark.parametrize("big", [3.4028234663852886e38, 3.4024e38, 3.3e38, -3.4028234663852886e38])
def test_values_next_to_the_largest_fp32(big):
    """A key and a value next to the largest number: score and output stay finite, to 2^-20."""
    c = Case([3], [40], 1, 1, 64, 16, "f32", seed=6, pad=0)
    slots = rows_of(c, 0)
    k, v = c.k.view(-1, 64), c.v.view(-1, 64)
    c.scale = 2.0 ** -117
    k[slots] = 0.0
    k[slots[11], 5] = big
    c.q[...] = 0.0
    c.q[..., 5] = math.copysign(0.25, big)       # score: 2^-119 of |big|, about 512; the others 0
    v[slots[11], 9] = big
    v[slots[12], 9] = 1.0
    v[slots[11], 10] = 2.5
    out, lse = c.run(False)
    score = abs(float(k[slots[11], 5].double())) * 2.0 ** -119
    assert ((lse.double() - score).abs() <= score * 2.0 ** -20).all()
    assert (out[:, 0, 9].double() - float(v[slots[11], 9])).abs().le(abs(big) * 2.0 ** -20).all()
    assert (out[:, 0, 10].double() - 2.5).abs().le(2.0 ** -19).all()
