"""pa_attend: a row's bits depend on its own sequence's queries and keys alone (and on the lengths).

Groups that do not divide a row tile leave rows of it that no query fills; runs shorter than a
tile leave rows that hold the next sequence's queries or the padding of q.  None of them may
decide how the real rows are rounded."""
import math

import pytest
import torch

import paged_kv_cache_79_gb300 as P
from tests.test_gpu_attend import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"


def filled_before(d, dtype, value):
    """A call over the whole GPU that leaves `value`-sized queries in every SM's shared memory."""
    c = Case([2000], [4000], 8, 2, d, 16, dtype, seed=21, pad=0)
    c.q.copy_((torch.randn(c.q.shape, device=DEV, generator=torch.Generator(DEV).manual_seed(5)) * value).to(c.dt))
    c.run(False)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [3, 5, 7, 13])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_rows_that_no_query_fills(dtype, group, d, causal):
    """The same call after calls that left small and large queries in shared memory."""
    c = Case([9, 40, 130, 400], [700, 3000, 1000, 5000], 2 * group, 2, d, 16, dtype, seed=group)
    got = []
    for value in (0.0, 300.0, 0.0, 30.0):
        filled_before(d, dtype, value)
        got.append(c.run(causal))
    c.check(*got[0], causal)
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (10, 2), (13, 1), (2, 2)])
@pytest.mark.parametrize("causal", [False, True])
def test_other_rows_queries(dtype, hq, hkv, causal):
    """Other queries of the next sequence, and of the rows behind the last one."""
    c = Case([9, 77, 21], [900, 3000, 2500], hq, hkv, 128, 32, dtype, seed=hq, pad=300)
    own = torch.cat([torch.arange(0, 9), torch.arange(86, 107)]).to(DEV)       # the first and the last sequence's
    want, want_lse = c.run(causal)
    for value in (0.0, 200.0, 60000.0, math.inf, math.nan):
        x = torch.full((), value, device=DEV) if not math.isfinite(value) else torch.randn(
            c.q[9:86].shape, device=DEV, generator=torch.Generator(DEV).manual_seed(3)).clamp(-1, 1) * value
        c.q[9:86] = x.to(c.dt)
        c.q[107:] = value
        out, lse = c.run(causal)
        assert torch.equal(out[own], want[own]) and torch.equal(lse[own], want_lse[own]), value
    assert P.pa_device_errors() == 0


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_the_same_bits_every_time(dtype):
    """Cut items, one-tile items, rows of nobody: ten calls, other work in between."""
    c = Case([1, 300, 7, 0, 64], [9000, 5000, 100, 40, 20000], 15, 3, 128, 16, dtype, seed=31)
    want, want_lse = c.run(True)
    for i in range(10):
        torch.randn(1 << 20, device=DEV)
        if dtype != "f32":
            filled_before(128, dtype, 10.0 * i)
        out, lse = c.run(True)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
