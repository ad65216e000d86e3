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
