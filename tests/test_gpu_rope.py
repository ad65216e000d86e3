"""pa_rope and pa_rope_append against the formula in 64 bits.

Tolerances.  An output is amplitude * (a cos - b sin) in fp32, rounded once to its type.  The
angle is held to 2^-33 of a turn and its fp32 value to 2^-25 of half a turn, together at most
1e-7 + 1e-9 radians; cosine and sine are off by at most 2 ulp (2^-23 each), times the amplitude
(one rounding, 2^-24); products, sum: three roundings of 2^-24.  Relative to |a| + |b| times the
amplitude: 1e-7 + 2^-23 + 4 * 2^-24 < 5e-7.  Then half a step of the type (2^-24, 2^-11, 2^-8)
relative to the value.
"""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_79_gb300 as P

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def angles(rot, scaling="none", base=10000.0):
    f, a = P.rope_frequencies(rot, base, scaling, factor=8.0, original_len=4096, low=1.0,
                              high=4.0 if scaling == "bands" else 32.0)
    return f.to(DEV), a


def turned(x, pos, freqs, interleaved, amplitude):
    """(values in 64 bits, |a| + |b| of each element's pair)."""
    x = x.double().cpu()
    half = freqs.numel()
    # the fraction of a turn in exact integers
    f = [int(v) % (1 << 64) for v in freqs.cpu().tolist()]
    turn = np.array([[(int(p) * v) % (1 << 64) / 2.0 ** 64 for v in f] for p in pos.cpu().tolist()]).reshape(-1, half)
    w = torch.from_numpy(turn) * (2 * math.pi)
    c, s = torch.cos(w)[:, None], torch.sin(w)[:, None]
    i = torch.arange(half)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y, size = x.clone(), torch.zeros_like(x)
    y[..., one] = (x[..., one] * c - x[..., two] * s) * amplitude
    y[..., two] = (x[..., two] * c + x[..., one] * s) * amplitude
    size[..., one] = size[..., two] = (x[..., one].abs() + x[..., two].abs()) * abs(amplitude)
    return y, size


def check(got, x, pos, freqs, interleaved, amplitude, rot):
    y, size = turned(x, pos, freqs, interleaved, amplitude)
    g = got.double().cpu()
    tol = y.abs() * (torch.finfo(got.dtype).eps / 2) + size * 5e-7
    if got.dtype == torch.float16:
        tol = tol + 2.0 ** -25                    # half a step below fp16's normal range
    assert ((g - y).abs() <= tol).all(), float(((g - y).abs() - tol).max())
    assert torch.equal(got[..., rot:].cpu(), x[..., rot:].cpu())     # copied bit for bit


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot,hq,hkv,n", [(64, 64, 1, 1, 1), (64, 16, 3, 1, 33), (128, 128, 8, 2, 100),
                                            (128, 48, 5, 5, 257), (64, 48, 39, 3, 70), (128, 96, 64, 8, 3)])
def test_rope(dtype, interleaved, d, rot, hq, hkv, n):
    gen = torch.Generator(DEV).manual_seed(n)
    q, k = (torch.randn(n, h, d, device=DEV, generator=gen).to(DT[dtype]) for h in (hq, hkv))
    pos = torch.randint(-1000, 200000, (n,), device=DEV, generator=gen, dtype=torch.int32)
    freqs, _ = angles(rot)
    qo, ko = torch.full_like(q, 9.0), torch.full_like(k, 9.0)
    P.pa_rope(qo, q, ko, k, pos, freqs, interleaved=interleaved, amplitude=1.25)
    check(qo, q, pos, freqs, interleaved, 1.25, rot)
    check(ko, k, pos, freqs, interleaved, 1.25, rot)
    before = (q.clone(), k.clone())
    P.pa_rope(q, q, k, k, pos, freqs, interleaved=interleaved, amplitude=1.25)        # in place
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert not torch.equal(before[0], qo) or n == 0


@pytest.mark.parametrize("pos", [0, 1, -1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31])
def test_far_positions(pos):
    """Angles stay exact at the ends of 32 bits; position 0 copies."""
    q = torch.randn(2, 2, 128, device=DEV)
    p = torch.full((2,), pos, dtype=torch.int32, device=DEV)
    freqs, _ = angles(128, base=500000.0)
    qo, ko = torch.empty_like(q), torch.empty_like(q)
    P.pa_rope(qo, q, ko, q, p, freqs)
    check(qo, q, p, freqs, False, 1.0, 128)
    if pos == 0:
        assert torch.equal(qo, q)


@pytest.mark.parametrize("dtype,d,hq,hkv,B,n", [("bf16", 128, 64, 8, 16, 64), ("f32", 64, 39, 3, 32, 517),
                                                ("f16", 64, 4, 4, 16, 3000), ("bf16", 128, 2, 1, 32, 9001)])
@pytest.mark.parametrize("fused", [False, True])
def test_rope_append(dtype, d, hq, hkv, B, n, fused):
    """Rows of a fused projection or apart, shuffled slots with padding and slots past the pool."""
    gen = torch.Generator(DEV).manual_seed(n)
    if fused:
        x = torch.randn(n, (hq + 2 * hkv) * d + 8, device=DEV, generator=gen).to(DT[dtype])
        q, k, v = (x[:, a:b].unflatten(1, (-1, d)) for a, b in
                   ((0, hq * d), (hq * d, (hq + hkv) * d), ((hq + hkv) * d, (hq + 2 * hkv) * d)))
    else:
        q, k, v = (torch.randn(n, h, d, device=DEV, generator=gen).to(DT[dtype]) for h in (hq, hkv, hkv))
    rot = 32
    NB = n // B + 4
    pos = torch.randint(0, 40000, (n,), device=DEV, generator=gen, dtype=torch.int32)
    slots = torch.randperm(NB * B, device=DEV, generator=gen)[:n].contiguous()
    slots[::7] = -1
    slots[3::11] = NB * B
    freqs, amp = angles(rot, "yarn")
    kc, vc = (torch.full((NB, B, hkv, d), 3.0, device=DEV, dtype=DT[dtype]) for _ in range(2))
    out = torch.empty(n, hq, d, device=DEV, dtype=DT[dtype])
    P.pa_rope_append(out, q, k, v, kc, vc, pos, slots, freqs, amplitude=amp)
    check(out, q, pos, freqs, False, amp, rot)
    at = torch.nonzero((slots >= 0) & (slots < NB * B))[:, 0]
    rows = slots[at]
    check(kc.view(-1, hkv, d)[rows], k[at], pos[at], freqs, False, amp, rot)
    assert torch.equal(vc.view(-1, hkv, d)[rows], v[at])
    rest = torch.ones(NB * B, dtype=torch.bool, device=DEV)
    rest[rows] = False
    assert (kc.view(-1, hkv, d)[rest] == 3.0).all() and (vc.view(-1, hkv, d)[rest] == 3.0).all()


def test_in_place_in_a_fused_buffer():
    n, hq, hkv, d = 40, 6, 2, 64
    x = torch.randn(n, (hq + 2 * hkv) * d, device=DEV)
    want = x.clone()
    q, k = x[:, :hq * d].unflatten(1, (hq, d)), x[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    freqs, _ = angles(64)
    qo, ko = torch.empty(n, hq, d, device=DEV), torch.empty(n, hkv, d, device=DEV)
    P.pa_rope(qo, q, ko, k, pos, freqs)
    P.pa_rope(q, q, k, k, pos, freqs)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(x[:, (hq + hkv) * d:], want[:, (hq + hkv) * d:])


def test_nan_stays_in_its_pair():
    q = torch.ones(1, 1, 64, device=DEV)
    q[0, 0, 3] = math.nan
    q[0, 0, 7] = math.inf
    freqs, _ = angles(32)
    out, k = torch.empty_like(q), torch.ones_like(q)
    P.pa_rope(out, q, torch.empty_like(q), k, torch.tensor([5], dtype=torch.int32, device=DEV), freqs)
    bad = {i for i in range(64) if not math.isfinite(out[0, 0, i])}
    assert bad == {3, 19, 7, 23}


def test_no_tokens_and_another_stream():
    freqs, _ = angles(32)
    e = torch.empty(0, 2, 64, device=DEV)
    P.pa_rope(e, e, e, e, torch.empty(0, dtype=torch.int32, device=DEV), freqs)
    q = torch.randn(300, 2, 64, device=DEV)
    pos = torch.arange(300, dtype=torch.int32, device=DEV)
    a, b, c, d = (torch.empty_like(q) for _ in range(4))
    P.pa_rope(a, q, b, q, pos, freqs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    P.pa_rope(c, q, d, q, pos, freqs, stream=s)
    s.synchronize()
    assert torch.equal(a, c) and torch.equal(b, d)
