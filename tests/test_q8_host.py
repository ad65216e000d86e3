"""The 8-bit cache and the table step on the host: layout, refusals, and the pins of the
models that the GPU tests compare with (no GPU needed)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_79_gb300 as P
from paged_kv_cache_79_gb300 import _lib
from tests import q8_model as M

FAKE = 1 << 20   # a 16-byte aligned non-null value; never dereferenced: validation fails first


def lib():
    return _lib.load()


# ---- layout -------------------------------------------------------------------
@pytest.mark.parametrize("hkv", [1, 2, 5, 8, 40, 63])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("b", [16, 32])
def test_block_layout(hkv, d, b):
    assert P.pa_q8_block_bytes(hkv, d, b) == M.block_bytes(hkv, b, d)
    assert lib().pa_q8_scales_offset(hkv, d, b) == hkv * 2 * b * d
    cache = torch.zeros(3, M.block_bytes(hkv, b, d), dtype=torch.uint8)
    codes, scales = P.q8_views(cache, hkv, d, b)
    assert codes.shape == (3, hkv, 2, b, d) and scales.shape == (3, hkv, 2)
    m = M.Cache(cache.numpy(), hkv, b, d)
    m.scales[2, hkv - 1, 1] = 0.25
    m.codes[1, hkv - 1, 0, b - 1, d - 1] = 0x38
    assert scales[2, hkv - 1, 1] == 0.25 and scales.sum() == 0.25
    assert codes.float()[1, hkv - 1, 0, b - 1, d - 1] == 1.0 and codes.float().sum() == 1.0


def test_layout_of_sizes_that_are_not_built():
    for hkv, d, b in ((0, 128, 16), (4, 96, 16), (4, 256, 16), (4, 128, 8), (4, 128, 64), (-1, 64, 32),
                      (65536, 64, 16)):
        with pytest.raises(P.PagedKVError):
            P.pa_q8_block_bytes(hkv, d, b)
    with pytest.raises(ValueError):
        P.q8_views(torch.zeros(2, 100, dtype=torch.uint8), 2, 64, 16)


# ---- refusals (C ABI) -----------------------------------------------------------
def _append(**kw):
    a = dict(k=FAKE, v=FAKE, c=FAKE, bt=FAKE, W=4, cl=FAKE, qs=FAKE, S=2, N=5, NB=8, Hkv=2, D=128, B=16, dt=2)
    a.update(kw)
    return lib().pa_q8_append(a["k"], a["v"], a["c"], a["bt"], a["W"], a["cl"], a["qs"], a["S"], a["N"], a["NB"],
                              a["Hkv"], a["D"], a["B"], a["dt"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), P.PA_ERR_INVALID), (dict(v=None), P.PA_ERR_INVALID), (dict(c=None), P.PA_ERR_INVALID),
    (dict(bt=None), P.PA_ERR_INVALID), (dict(cl=None), P.PA_ERR_INVALID),
    (dict(k=FAKE + 8), P.PA_ERR_INVALID), (dict(v=FAKE + 2), P.PA_ERR_INVALID), (dict(c=FAKE + 8), P.PA_ERR_INVALID),
    (dict(bt=FAKE + 2), P.PA_ERR_INVALID), (dict(cl=FAKE + 1), P.PA_ERR_INVALID), (dict(qs=FAKE + 2), P.PA_ERR_INVALID),
    (dict(qs=None), P.PA_ERR_INVALID),                     # 5 rows, 2 sequences, no query_start
    (dict(S=-1), P.PA_ERR_INVALID), (dict(N=-1), P.PA_ERR_INVALID), (dict(W=0), P.PA_ERR_INVALID),
    (dict(NB=0), P.PA_ERR_INVALID), (dict(Hkv=0), P.PA_ERR_INVALID), (dict(NB=1 << 28), P.PA_ERR_INVALID),
    (dict(W=1 << 28), P.PA_ERR_INVALID),
    (dict(D=96), P.PA_ERR_UNSUPPORTED), (dict(B=8), P.PA_ERR_UNSUPPORTED), (dict(dt=5), P.PA_ERR_UNSUPPORTED),
    (dict(Hkv=1 << 16), P.PA_ERR_UNSUPPORTED),
    (dict(S=0), P.PA_OK), (dict(N=0), P.PA_OK),
])
def test_append_refusals(kw, want):
    assert _append(**kw) == want


def _decode(**kw):
    a = dict(out=FAKE, q=FAKE, c=FAKE, bt=FAKE, W=4, cl=FAKE, S=2, NB=8, Hq=4, Hkv=2, D=128, B=16, dt=2, ws=FAKE,
             wsb=1 << 30)
    a.update(kw)
    return lib().pa_q8_decode(a["out"], a["q"], a["c"], a["bt"], a["W"], a["cl"], a["S"], a["NB"], 0.1, a["Hq"],
                              a["Hkv"], a["D"], a["B"], a["dt"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(out=None), P.PA_ERR_INVALID), (dict(q=None), P.PA_ERR_INVALID), (dict(c=None), P.PA_ERR_INVALID),
    (dict(bt=None), P.PA_ERR_INVALID), (dict(cl=None), P.PA_ERR_INVALID), (dict(out=FAKE + 4), P.PA_ERR_INVALID),
    (dict(q=FAKE + 8), P.PA_ERR_INVALID), (dict(c=FAKE + 4), P.PA_ERR_INVALID), (dict(S=-2), P.PA_ERR_INVALID),
    (dict(Hq=5), P.PA_ERR_INVALID), (dict(Hq=0), P.PA_ERR_INVALID), (dict(Hkv=0), P.PA_ERR_INVALID),
    (dict(NB=0), P.PA_ERR_INVALID), (dict(W=0), P.PA_ERR_INVALID), (dict(NB=1 << 27), P.PA_ERR_INVALID),
    (dict(D=32), P.PA_ERR_UNSUPPORTED), (dict(B=64), P.PA_ERR_UNSUPPORTED), (dict(dt=3), P.PA_ERR_UNSUPPORTED),
    (dict(Hq=1 << 17, Hkv=1 << 16), P.PA_ERR_UNSUPPORTED),
    (dict(S=0), P.PA_OK),
])
def test_decode_refusals(kw, want):
    assert _decode(**kw) == want


def _tables(**kw):
    a = dict(bt=FAKE, W=4, clo=FAKE, cl=FAKE, nt=FAKE, S=2, fl=FAKE, NB=8, nfo=FAKE, nf=FAKE, B=16, gr=FAKE, qs=FAKE,
             sl=FAKE, ns=4)
    a.update(kw)
    return lib().pa_build_tables(a["bt"], a["W"], a["clo"], a["cl"], a["nt"], a["S"], a["fl"], a["NB"], a["nfo"],
                                 a["nf"], a["B"], a["gr"], a["qs"], a["sl"], a["ns"], None)


@pytest.mark.parametrize("kw", [dict(bt=None), dict(clo=None), dict(cl=None), dict(nt=None), dict(fl=None),
                                dict(nfo=None), dict(nf=None), dict(gr=None), dict(qs=None), dict(sl=None),
                                dict(bt=FAKE + 2), dict(sl=FAKE + 4), dict(qs=FAKE + 1), dict(S=-1), dict(ns=-1),
                                dict(W=0), dict(NB=0), dict(B=0), dict(NB=1 << 27), dict(W=1 << 27)], ids=str)
def test_tables_refusals(kw):
    assert _tables(**kw) == P.PA_ERR_INVALID


def test_block_move_refusals():
    f = lib().pa_q8_copy_blocks
    assert f(None, FAKE, 1, 4, 256, None) == P.PA_ERR_INVALID
    assert f(FAKE, None, 1, 4, 256, None) == P.PA_ERR_INVALID
    assert f(FAKE, FAKE, 1, 4, 100, None) == P.PA_ERR_INVALID
    assert f(FAKE, FAKE, -1, 4, 256, None) == P.PA_ERR_INVALID
    assert f(FAKE, FAKE, 1, 0, 256, None) == P.PA_ERR_INVALID
    assert f(None, None, 0, 4, 256, None) == P.PA_OK
    g = lib().pa_q8_swap_blocks
    assert g(None, FAKE, FAKE, 1, 4, 4, 256, None) == P.PA_ERR_INVALID
    assert g(FAKE, FAKE + 8, FAKE, 1, 4, 4, 256, None) == P.PA_ERR_INVALID
    assert g(FAKE, FAKE, FAKE, 1, 4, 4, 0, None) == P.PA_ERR_INVALID
    assert g(None, None, None, 0, 4, 4, 256, None) == P.PA_OK


# ---- refusals (binding) ---------------------------------------------------------
def test_binding_refuses_wrong_tensors():
    cache = torch.zeros(4, P.pa_q8_block_bytes(2, 64, 16), dtype=torch.uint8)
    k = torch.zeros(3, 2, 64)
    bt, cl = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    qs = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        P.pa_q8_append(k, k, cache, bt, cl, 16)
    with pytest.raises(ValueError, match="alike"):
        P.pa_q8_append(k, k[:2], cache, bt, cl, 16)
    with pytest.raises(TypeError):
        P.pa_q8_append(k, k.half(), cache, bt, cl, 16)
    with pytest.raises(ValueError, match="kv_cache"):
        P.pa_q8_append(k, k, cache, bt, cl, 32)
    with pytest.raises(TypeError):
        P.pa_q8_append(k, k, cache, bt.long(), cl, 16)
    with pytest.raises(ValueError, match="query_start"):
        P.pa_q8_append(k, k, cache, bt, cl, 16, query_start=qs[:3])
    with pytest.raises(ValueError, match="context_lens"):
        P.pa_q8_append(k, k, cache, bt, cl[:2], 16)
    q = torch.zeros(3, 4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        P.pa_q8_decode(q, q, cache, bt, cl, 0.1, 4, 2, 64, 16)
    with pytest.raises(ValueError, match="q and out"):
        P.pa_q8_decode(q, q[:2], cache, bt, cl, 0.1, 4, 2, 64, 16)
    with pytest.raises(TypeError):
        P.pa_q8_decode(q.half(), q, cache, bt, cl, 0.1, 4, 2, 64, 16)
    with pytest.raises(TypeError):
        P.pa_q8_decode(q, q, cache.float(), bt, cl, 0.1, 4, 2, 64, 16)
    one, slots = torch.zeros(1, dtype=torch.int32), torch.zeros(5, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        P.pa_build_tables(bt, cl, cl, qs, one, 16, slots, qs, cl)
    with pytest.raises(TypeError):
        P.pa_build_tables(bt, cl, cl, qs, one, 16, slots.int(), qs, cl)
    with pytest.raises(ValueError, match="query_start"):
        P.pa_build_tables(bt, cl, cl, qs, one, 16, slots, cl, cl)
    with pytest.raises(ValueError, match="num_free"):
        P.pa_build_tables(bt, cl, cl, qs, cl, 16, slots, qs, cl)


def test_binding_refuses_wrong_moves():
    cache = torch.zeros(4, P.pa_q8_block_bytes(2, 64, 16), dtype=torch.uint8)
    pairs = torch.zeros(3, 2, dtype=torch.int32)
    for wrong in (pairs[0], pairs[:, :1].contiguous(), torch.zeros(3, 3, dtype=torch.int32)):
        with pytest.raises(ValueError, match=r"\[n, 2\]"):
            P.pa_q8_copy_blocks(cache, wrong)
        with pytest.raises(ValueError, match=r"\[n, 2\]"):
            P.pa_q8_swap_blocks(cache, cache, wrong)
    with pytest.raises(TypeError):
        P.pa_q8_copy_blocks(cache, pairs.long())
    with pytest.raises(TypeError):
        P.pa_q8_copy_blocks(cache.view(torch.int32), pairs)
    with pytest.raises(ValueError, match="pools"):
        P.pa_q8_copy_blocks(cache.view(-1), pairs)
    with pytest.raises(ValueError, match="different sizes"):
        P.pa_q8_swap_blocks(cache, torch.zeros(4, 256, dtype=torch.uint8), pairs)
    with pytest.raises(ValueError, match="CUDA"):
        P.pa_q8_copy_blocks(cache, pairs)
    with pytest.raises(ValueError, match="pinned"):
        P.pa_q8_swap_blocks(cache, cache, pairs)
    P.pa_q8_copy_blocks(cache, pairs[:0])
    P.pa_q8_swap_blocks(cache, cache, pairs[:0])


# ---- the models' pins -----------------------------------------------------------
def test_code_values_are_e4m3():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, M.CODES, equal_nan=True)


def test_encode_rounds_to_nearest_even():
    v = M.CODES[:127]
    mid = (v[1:] + v[:-1]) / 2
    for y in (v, mid, mid * (1 + 1e-9), mid * (1 - 1e-9), np.linspace(0, 448, 100001)):
        for sign in (1, -1):
            want = torch.from_numpy(sign * y).float()      # (torch rounds from fp32)
            got = M.encode(want.double().numpy())
            assert np.array_equal(M.CODES[got], want.to(torch.float8_e4m3fn).double().numpy())
    assert (M.encode([np.nan, np.inf, -np.inf]) == 0x7F).all()


@pytest.mark.parametrize("top,want", [(448.0, 1.0), (448.0000001, 2.0), (447.0, 1.0), (224.0, 0.5), (0.0, 2.0 ** -126),
                                      (1.0, 2.0 ** -8), (1.75, 2.0 ** -8), (1.7500001, 2.0 ** -7), (1e-44, 2.0 ** -126),
                                      (3.3e38, 2.0 ** 120)])
def test_need_scale(top, want):
    x = np.array([0.0, -top, np.nan, np.inf, top / 2])
    assert M.need_scale(x) == want


def test_rows_one_at_a_time_hold_what_one_write_holds():
    # values that stay in e4m3's normal range at every scale met: the same codes
    rng = np.random.default_rng(3)
    hkv, b, d, n = 2, 16, 64, 41
    x = np.exp2(rng.uniform(-3, 3, size=(2, n, hkv, d))) * rng.choice([-1, 1], size=(2, n, hkv, d))
    bt = np.array([[2, 0, 3]], dtype=np.int32)
    one = M.Cache(np.full((4, M.block_bytes(hkv, b, d)), 0xA5, dtype=np.uint8), hkv, b, d)
    all_ = M.Cache(one.raw.copy(), hkv, b, d)
    M.append(all_, x[0], x[1], bt, np.array([n]), np.array([0, n]))
    for t in range(n):
        M.append(one, x[0, t:t + 1], x[1, t:t + 1], bt, np.array([t + 1]))
    for blk in (2, 0, 3):
        assert np.array_equal(one.scales[blk], all_.scales[blk])
    v1 = one.values([2, 0, 3]).transpose(2, 1, 0, 3, 4).reshape(2, hkv, 48, d)[:, :, :n]
    v2 = all_.values([2, 0, 3]).transpose(2, 1, 0, 3, 4).reshape(2, hkv, 48, d)[:, :, :n]
    assert np.array_equal(v1, v2)
    assert np.abs(v1 - x.transpose(0, 2, 1, 3)).max() <= 2.0 ** -4 * 8


def test_table_model_is_the_host_allocator():
    """Random steps of releases and appends: the model's tables, free list and slots are
    those of the library's host allocator, run in the documented order."""
    rng = np.random.default_rng(5)
    b, pool, width, reqs = 16, 60, 12, 7
    order = rng.permutation(pool).astype(np.int32)
    host = P.BlockAllocator(pool, b, order)
    seqs = [host.new_seq() for _ in range(reqs)]
    bt = np.full((reqs, width), -1, dtype=np.int32)
    cl, free, nfree = np.zeros(reqs, dtype=np.int32), order.copy(), pool
    for step in range(40):
        new = rng.integers(0, 40, size=reqs)
        new[rng.random(reqs) < 0.25] = -1
        bt, cl2, free, nfree, granted, qs, slots = M.build_tables(bt, cl, new, free, nfree, b, 400)
        for s in range(reqs):
            if new[s] < 0:
                host.free_seq(seqs[s])
                seqs[s] = host.new_seq()
        at = 0
        for s in range(reqs):
            if granted[s] > 0:
                want, pairs = host.append_n(seqs[s], int(granted[s]))
                assert np.array_equal(slots[at:at + len(want)], want) and len(pairs) == 0
                at += len(want)
            assert host.seq_len(seqs[s]) == cl2[s]
            tab = host.block_table(seqs[s])
            assert tab == bt[s, :len(tab)].tolist()
        assert at == qs[-1] and (slots[at:] == -1).all()
        assert host.free_list() == free[:nfree].tolist()
        cl = cl2
