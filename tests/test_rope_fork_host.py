"""Rotary frequencies, and what the rotary and fork entry points refuse (no GPU needed)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_79_gb300 as P
from paged_kv_cache_79_gb300 import _lib

FAKE = 1 << 20   # a 16-byte aligned non-null value; never dereferenced: validation fails first


def turns(f):
    """Exact distance is judged in turns: int64 entries as fractions of a turn."""
    return np.array([int(v) % (1 << 64) for v in f.tolist()], dtype=object)


@pytest.mark.parametrize("rot", [2, 16, 48, 64, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
@pytest.mark.parametrize("scaling", sorted(P.ROPE_SCALINGS))
def test_frequencies(rot, base, scaling):
    """Against the formulas with Python floats: to 2^-50 of the angle (a few roundings of
    2^-53 in pow, log and the ramp) and half a unit of 2^-64."""
    factor, length, low, high = 8.0, 4096.0, 1.0, 32.0
    f, amp = P.rope_frequencies(rot, base, scaling, factor, length, low, high)
    assert f.dtype == torch.int64 and f.shape == (rot // 2,)
    assert amp == pytest.approx(0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0, rel=1e-7)
    b = base * factor ** (rot / (rot - 2) if rot > 2 else 1.0) if scaling == "ntk" else base
    lo = max(math.floor(rot * math.log(length / (high * 2 * math.pi)) / (2 * math.log(base))), 0)
    hi = min(math.ceil(rot * math.log(length / (low * 2 * math.pi)) / (2 * math.log(base))), rot - 1)
    for i, got in enumerate(turns(f)):
        t = b ** (-2 * i / rot)
        keep = {"none": 1.0, "ntk": 1.0, "linear": 0.0, "bands": (length * t / (2 * math.pi) - low) / (high - low),
                "yarn": 1 - (i - lo) / max(hi - lo, 0.001)}[scaling]
        keep = min(max(keep, 0.0), 1.0)
        want = (t / factor * (1 - keep) + t * keep) / (2 * math.pi) * 2.0 ** 64
        assert abs(got - want) <= want * 2.0 ** -47 + 1


def test_frequency_refusals():
    for kw in (dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=16, base=1.0), dict(rotary_dim=16, scaling="x"),
               dict(rotary_dim=16, base=math.inf), dict(rotary_dim=16, scaling="linear", factor=0.5),
               dict(rotary_dim=16, scaling="yarn", factor=2.0, original_len=0),
               dict(rotary_dim=16, scaling="bands", factor=2.0, original_len=10, low=4.0, high=4.0),
               dict(rotary_dim=16, scaling="ntk", factor=math.nan)):
        with pytest.raises((ValueError, P.PagedKVError)):
            P.rope_frequencies(**kw)
    amp = ctypes.c_float()
    lib = _lib.load()
    assert lib.pa_rope_frequencies(None, ctypes.byref(amp), 16, 1e4, 0, 1, 0, 0, 0) == P.PA_ERR_INVALID
    buf = (ctypes.c_int64 * 8)()
    assert lib.pa_rope_frequencies(buf, ctypes.byref(amp), 16, 1e4, 9, 1, 0, 0, 0) == P.PA_ERR_UNSUPPORTED


def _append(**kw):
    a = dict(qo=FAKE, qos=256, q=FAKE, qs=256, k=FAKE, ks=128, v=FAKE, vs=128, kc=FAKE, vc=FAKE, pos=FAKE, slots=FAKE,
             f=FAKE, n=4, hq=4, hkv=2, d=64, rot=64, il=0, amp=1.0, B=16, NB=8, dt=2)
    a.update(kw)
    return _lib.load().pa_rope_append(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=0), P.PA_OK), (dict(q=None), P.PA_ERR_INVALID), (dict(qo=None), P.PA_ERR_INVALID),
    (dict(k=None), P.PA_ERR_INVALID), (dict(v=None), P.PA_ERR_INVALID), (dict(kc=None), P.PA_ERR_INVALID),
    (dict(vc=None), P.PA_ERR_INVALID), (dict(pos=None), P.PA_ERR_INVALID), (dict(slots=None), P.PA_ERR_INVALID),
    (dict(f=None), P.PA_ERR_INVALID), (dict(q=FAKE + 8), P.PA_ERR_INVALID), (dict(v=FAKE + 4), P.PA_ERR_INVALID),
    (dict(vc=FAKE + 2), P.PA_ERR_INVALID), (dict(pos=FAKE + 2), P.PA_ERR_INVALID),
    (dict(slots=FAKE + 4), P.PA_ERR_INVALID), (dict(f=FAKE + 4), P.PA_ERR_INVALID), (dict(n=-1), P.PA_ERR_INVALID),
    (dict(hq=0), P.PA_ERR_INVALID), (dict(hkv=-1), P.PA_ERR_INVALID), (dict(rot=0), P.PA_ERR_INVALID),
    (dict(rot=-16), P.PA_ERR_INVALID), (dict(rot=17), P.PA_ERR_INVALID), (dict(rot=80), P.PA_ERR_INVALID),
    (dict(rot=24), P.PA_ERR_UNSUPPORTED), (dict(d=96), P.PA_ERR_UNSUPPORTED), (dict(dt=3), P.PA_ERR_UNSUPPORTED),
    (dict(qs=252), P.PA_ERR_INVALID), (dict(qs=248), P.PA_ERR_INVALID), (dict(ks=0), P.PA_ERR_INVALID),
    (dict(vs=-128), P.PA_ERR_INVALID), (dict(qos=8), P.PA_ERR_INVALID), (dict(amp=math.inf), P.PA_ERR_INVALID),
    (dict(B=0), P.PA_ERR_INVALID), (dict(NB=0), P.PA_ERR_INVALID), (dict(NB=1 << 27), P.PA_ERR_INVALID),
    (dict(hq=1 << 20, qs=1 << 26, qos=1 << 26), P.PA_ERR_UNSUPPORTED),
])
def test_rope_append_validation(kw, want):
    assert _append(**kw) == want


def _fork(**kw):
    a = dict(bo=FAKE, bi=FAKE + 64, W=4, lo=FAKE, li=FAKE + 64, rows=2, par=FAKE, kids=3, ex=FAKE, fl=FAKE, NB=8,
             nfo=FAKE, nf=FAKE, B=16, pairs=FAKE, gr=FAKE)
    a.update(kw)
    return _lib.load().pa_fork_tables(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(bo=None), P.PA_ERR_INVALID), (dict(bi=None), P.PA_ERR_INVALID), (dict(lo=None), P.PA_ERR_INVALID),
    (dict(li=None), P.PA_ERR_INVALID), (dict(par=None), P.PA_ERR_INVALID), (dict(ex=None), P.PA_ERR_INVALID),
    (dict(fl=None), P.PA_ERR_INVALID), (dict(nfo=None), P.PA_ERR_INVALID), (dict(nf=None), P.PA_ERR_INVALID),
    (dict(pairs=None), P.PA_ERR_INVALID), (dict(gr=None), P.PA_ERR_INVALID), (dict(rows=-1), P.PA_ERR_INVALID),
    (dict(kids=-1), P.PA_ERR_INVALID), (dict(W=0), P.PA_ERR_INVALID), (dict(NB=0), P.PA_ERR_INVALID),
    (dict(B=0), P.PA_ERR_INVALID), (dict(bi=FAKE), P.PA_ERR_INVALID), (dict(li=FAKE), P.PA_ERR_INVALID),
    (dict(pairs=FAKE + 2), P.PA_ERR_INVALID), (dict(ex=FAKE + 1), P.PA_ERR_INVALID),
    (dict(NB=1 << 27), P.PA_ERR_INVALID), (dict(W=1 << 27), P.PA_ERR_INVALID),
    (dict(rows=65537), P.PA_ERR_UNSUPPORTED), (dict(kids=65537), P.PA_ERR_UNSUPPORTED),
    (dict(W=65535 * 1024 + 1, B=1), P.PA_ERR_UNSUPPORTED), (dict(NB=0x7fffffff - 1000, B=1), P.PA_ERR_UNSUPPORTED),
])
def test_fork_validation(kw, want):
    assert _fork(**kw) == want


def test_binding_refuses_cpu_tensors_and_types():
    q = torch.zeros(2, 2, 64)
    pos, f = torch.zeros(2, dtype=torch.int32), torch.zeros(16, dtype=torch.int64)
    with pytest.raises(ValueError):
        P.pa_rope(q, q, q, q, pos, f)
    with pytest.raises(TypeError):
        P.pa_rope(q, q, q, q, pos.long(), f)
    with pytest.raises(TypeError):
        P.pa_rope(q, q, q.half(), q, pos, f)
    with pytest.raises(ValueError):
        P.pa_rope(q, q.transpose(1, 2), q, q, pos, f)
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError):
        P.pa_fork_tables(t, i, t, i, i, torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int32), i[:1], 16,
                         torch.zeros(2, 2, dtype=torch.int32), i)
    with pytest.raises(TypeError):
        P.pa_fork_tables(t, i, t, i, i.long(), t, t, i[:1], 16, t, i)
