"""pa_attend at its limits: waits that run out."""
import pytest
import torch

import paged_kv_cache_79_gb300 as P
from tests.test_gpu_attend import Case

pytestmark = pytest.mark.gpu
TIMEOUTS = P.PA_DEVERR_TIMEOUT_FULL | P.PA_DEVERR_TIMEOUT_EMPTY
EMPTY = [0] * 16384      # behind a CTA's last item: a walk of milliseconds before the next is handed on


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,lens", [
    ([5], [100]),                    # one CTA, one tile of keys: all copies issued before any wait runs out
    ([200, 3], [128, 40]),           # two row tiles, whole tiles
    ([7, 300], [3000, 900]),         # several CTAs, cut items
])
def test_waits_that_surely_run_out(dtype, d, new, lens):
    """With a limit of 1 ns the warps that wait for the next item give up while another walks over
    thousands of empty sequences.  The launch lets its copies land, returns and says so, and a call
    enqueued right behind it is right."""
    c = Case(new + EMPTY + [2], lens + EMPTY + [50], 4, 2, d, 16, dtype, seed=sum(lens))
    assert P.pa_device_errors() == 0
    for causal in (True, False):
        P.pa_set_wait_limit_ns(1)
        try:
            c.run(causal)
        finally:
            P.pa_set_wait_limit_ns(0)
        out, lse = c.run(causal)
        flags = P.pa_device_errors()
        assert flags & TIMEOUTS and not flags & ~TIMEOUTS, hex(flags)
        c.check(out, lse, causal)


def test_fp32_has_no_wait_to_run_out():
    """The fp32 kernel's copies are waited for by the threads that issued them."""
    c = Case([5] + EMPTY + [2], [100] + EMPTY + [50], 4, 2, 64, 16, "f32", seed=1)
    P.pa_set_wait_limit_ns(1)
    try:
        out, lse = c.run(True)
        assert P.pa_device_errors() == 0
    finally:
        P.pa_set_wait_limit_ns(0)
    c.check(out, lse, True)
