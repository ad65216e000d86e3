"""pa_attend at its limits: waits that run out, contexts next to 2^31 keys."""
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


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B", [16, 32])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("short", [0, 5])
def test_a_context_next_to_two_to_the_31(dtype, B, causal, short):
    """The widest table whose slots are below 2^31, all but its last entry one block of score 0; the
    last block's keys hold all of the weight, but for the `short` ones past the context, which would
    outweigh them.  The others' weights are e^-100, 2^31 of them: nothing in fp32."""
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    width = (1 << 31) // B - 1
    T = width * B - short
    bt = torch.zeros(1, width, dtype=torch.int32, device="cuda")
    bt[0, -1] = 1
    k, v = torch.zeros(2, B, 1, 64, device="cuda", dtype=dt), torch.randn(2, B, 1, 64, device="cuda").to(dt)
    k[1] = 100.0 / 8
    if short:
        k[1, B - short:], v[1, B - short:] = 200.0 / 8, float("nan")
    n = 3 if causal else 2
    q = torch.ones(n, 2, 64, device="cuda", dtype=dt)
    out, lse = torch.empty_like(q), torch.empty(n, 2, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    P.pa_attend(out, q, k, v, bt, torch.tensor([T], **i32), torch.tensor([0, n], **i32), 0.125, 2, 1, 64, B,
                causal=causal, lse=lse)
    assert P.pa_device_errors() == 0
    for i in range(n):
        keys = B - short - (n - 1 - i if causal else 0)
        want = v[1, :keys, 0].double().mean(0)
        # weights 1/keys, half a step of the type off each; sums of at most 32; half a step of the output
        half = torch.finfo(dt).eps / 2
        tol = v[1, :keys, 0].double().abs().mean(0) * (2 * half + 2.0 ** -18)
        assert ((out[i].double() - want).abs() <= tol).all(), i
        z = 100.0 + torch.tensor(float(keys)).log().item()
        assert ((lse[i].double() - z).abs() <= z * 2.0 ** -20).all()
