"""pa_attend against the definition in 64 bits.

Tolerances, per row and element, with p the row's probabilities and d the head dimension:
  a score is off by at most  delta = scale * |q| . |k| * (2^-21 + (d + 4) 2^-24): products in two
  tf32 terms (16-bit operands are exact), d sums in fp32, the scale;
  so a probability is off by 2 delta (the sum's share included) + 2^-20 (the exponentials) of
  itself, and in fp16 and bf16 by half a step of the type more;
  sums over T keys in fp32 add T 2^-23 (tensor cores may cut instead of rounding);
  all of that times sum p |v|, and half a step of the output's type.
lse: delta + 2^-20 + T 2^-24 + 2^-22 |lse|.
"""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_79_gb300 as P

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


class Case:
    def __init__(self, new, lens, hq, hkv, d, B, dtype, seed=0, pad=3, stale=math.nan, amount=1.0, apart=False,
                 q_pad=0):
        g = torch.Generator(DEV).manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.new, self.lens, self.hq, self.hkv, self.d, self.B, self.dt = new, lens, hq, hkv, d, B, DT[dtype]
        nbs = [-(-t // B) for t in lens]
        pool, width = sum(nbs) + 4, max(nbs + [1]) + 1
        order = rng.permutation(pool)
        bt = np.full((len(lens), width), -1, np.int32)
        kv = torch.full((2, pool, B, hkv, d), stale, device=DEV, dtype=self.dt)
        at = 0
        for s, t in enumerate(lens):
            ids = order[at:at + nbs[s]]
            at += nbs[s]
            bt[s, :nbs[s]] = ids
            slots = torch.from_numpy((ids[:, None] * B + np.arange(B)).reshape(-1)[:t].astype(np.int64)).to(DEV)
            kv.view(2, pool * B, hkv, d)[:, slots] = (
                torch.randn(2, t, hkv, d, device=DEV, generator=g) * amount).to(self.dt)
        n = sum(new) + pad
        self.k, self.v = (kv[0], kv[1]) if not apart else (kv[0].clone(), kv[1].clone())
        if apart and self.v.data_ptr() > self.k.data_ptr():
            self.k, self.v = self.v.copy_(kv[0]), self.k.copy_(kv[1])      # V below K
        x = torch.randn(n, hq * d + q_pad, device=DEV, generator=g).to(self.dt)
        self.q = x[:, :hq * d].unflatten(1, (hq, d))
        self.bt = torch.from_numpy(bt).to(DEV)
        self.cl = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.qs = torch.tensor([0] + np.cumsum(new).tolist(), dtype=torch.int32, device=DEV)
        self.n = n
        self.scale = d ** -0.5

    def run(self, causal, with_lse=True, out=None, **kw):
        out = torch.full((self.n, self.hq, self.d), 7.0, device=DEV, dtype=self.dt) if out is None else out
        lse = torch.full((self.n, self.hq), 7.0, device=DEV) if with_lse else None
        P.pa_attend(out, self.q, self.k, self.v, self.bt, self.cl, self.qs, self.scale, self.hq, self.hkv, self.d,
                    self.B, causal=causal, lse=lse, **kw)
        return out, lse

    def check(self, out, lse, causal):
        assert P.pa_device_errors() == 0
        f32 = self.dt == torch.float32
        half = torch.finfo(self.dt).eps / 2
        at = 0
        for s, (n, t) in enumerate(zip(self.new, self.lens)):
            rows = slice(at, at + n)
            at += n
            if n == 0:
                continue
            if t == 0:
                assert (out[rows] == 0).all() and (lse is None or (lse[rows] == -math.inf).all())
                continue
            ids = self.bt[s, :-(-t // self.B)].long()
            k, v = (c[ids].reshape(-1, self.hkv, self.d)[:t].double() for c in (self.k, self.v))
            i, j = torch.arange(n, device=DEV)[:, None], torch.arange(t, device=DEV)
            hidden = j > t - n + i if causal else None
            for h in range(self.hq):
                kh, vh, q = k[:, h * self.hkv // self.hq], v[:, h * self.hkv // self.hq], self.q[rows, h].double()
                sc = q @ kh.T * self.scale
                size = q.abs() @ kh.abs().T * self.scale
                if causal:
                    sc[hidden] = -math.inf
                    size[hidden] = 0
                z = torch.logsumexp(sc, -1)
                none = z == -math.inf
                p = torch.exp(sc - torch.where(none, torch.zeros_like(z), z)[:, None])
                delta = size.amax(-1) * (2.0 ** -21 * f32 + (self.d + 4) * 2.0 ** -24)
                tol = (2 * delta + 2.0 ** -20 + t * 2.0 ** -23 + (0 if f32 else 2 * half))[:, None] * (p @ vh.abs())
                want = p @ vh
                tol = tol + want.abs() * half + (2.0 ** -25 if self.dt == torch.float16 else 0)
                err = (out[rows, h].double() - want).abs()
                assert (err <= tol).all(), (s, h, n, t, float((err - tol).max()), float(err.max()))
                if lse is not None:
                    got = lse[rows, h].double()
                    assert torch.equal(got == -math.inf, none)
                    e = (got - z).abs()[~none]
                    assert (e <= (delta + 2.0 ** -20 + t * 2.0 ** -24 + z.abs() * 2.0 ** -22)[~none]).all(), (s, h)
        assert (out[at:] == 7.0).all() and (lse is None or (lse[at:] == 7.0).all())       # padding


DTYPES = ["f32", "f16", "bf16"]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,B", [(64, 16), (128, 16), (64, 32), (128, 32)])
def test_one_short_sequence(dtype, causal, d, B):
    c = Case([7], [50], 8, 8, d, B, dtype)
    c.check(*c.run(causal), causal)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("new,lens", [
    ([1], [1]), ([1], [0]), ([5], [3]), ([300], [100]), ([129], [129]), ([0, 1, 0], [5, 6, 0]),
    ([128, 1, 257, 0, 33], [128, 700, 300, 40, 0]), ([3, 2, 1, 8], [1000, 15, 16, 4097]), ([64], [4096 + 31]),
    ([260], [127]), ([500], [513]),
])
def test_ragged(dtype, causal, new, lens):
    """Lengths around tiles and blocks, empty sequences, more queries than keys."""
    c = Case(new, lens, 6, 2, 128, 16, dtype, seed=sum(lens))
    c.check(*c.run(causal), causal)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 1), (39, 3), (14, 2), (16, 1), (130, 1), (300, 2), (40, 40)])
@pytest.mark.parametrize("d", [64, 128])
def test_head_groups(dtype, hq, hkv, d):
    """Groups that do not divide a tile's rows, groups wider than a tile."""
    c = Case([9, 40, 1], [70, 200, 333], hq, hkv, d, 32, dtype, seed=hq)
    c.check(*c.run(True), True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("new,t", [(1, 30000), (3, 20011), (40, 9000), (700, 5000)])
def test_items_cut_between_ctas(dtype, causal, new, t):
    """Few rows over long contexts: one item's keys on many CTAs, merged."""
    c = Case([new], [t], 2, 1, 64, 16, dtype, seed=new)
    c.check(*c.run(causal), causal)


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_sequences(dtype):
    """More sequences than a CTA has threads; most of them tiny."""
    rng = np.random.default_rng(3)
    new = rng.integers(0, 4, size=700).tolist()
    lens = [int(x) for x in rng.integers(0, 60, size=700)]
    lens[500], new[500], new[699] = 3000, 200, 5
    c = Case(new, lens, 4, 2, 64, 16, dtype, seed=4)
    c.check(*c.run(True), True)


@pytest.mark.parametrize("dtype", DTYPES)
def test_scores_far_apart(dtype):
    """Scores of several hundred: running maxima that jump, rows whose weight is one key's."""
    c = Case([200], [1500], 4, 2, 64, 16, dtype, seed=5, amount=8.0)
    c.q.mul_(8.0)
    c.check(*c.run(True), True)
    rising = torch.arange(1500, device=DEV) / 30.0               # every tile raises the maximum
    c.q[...] = 1.0
    slots = (c.bt[0, :94].long()[:, None] * 16 + torch.arange(16, device=DEV)).reshape(-1)[:1500]
    c.k.view(-1, 2, 64)[slots] = (rising / 8.0)[:, None, None].to(c.dt)
    c.check(*c.run(False), False)


@pytest.mark.parametrize("dtype", DTYPES)
def test_placements_strides_and_workspace(dtype):
    """Separate caches with V below K, q a part of wider rows, a workspace full of NaN, no lse."""
    c = Case([100, 31], [200, 1000], 6, 3, 128, 16, dtype, seed=6, apart=True, q_pad=64)
    ws = torch.full((P.pa_attend_workspace_size(6, 3, 128),), 255, dtype=torch.uint8, device=DEV)
    out, lse = c.run(True, workspace=ws)
    c.check(out, lse, True)
    alone, _ = c.run(True, with_lse=False)
    assert torch.equal(alone, out)
    again, lse2 = c.run(True)
    assert torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("dtype", DTYPES)
def test_outputs_and_workspace_at_any_16_bytes(dtype):
    """out and workspace 16 bytes past a 32-byte boundary: whole items, cut ones, empty rows."""
    c = Case([300, 5, 9], [900, 6000, 3], 4, 1, 64, 16, dtype, seed=17)
    want, want_lse = c.run(True)
    n = c.n * 4 * 64
    off = 16 // c.q.element_size()
    buf = torch.full((n + 2 * off,), 7.0, device=DEV, dtype=c.dt)
    out = buf[off:off + n].view(c.n, 4, 64)
    ws = torch.empty(P.pa_attend_workspace_size(4, 1, 64) + 16, dtype=torch.uint8, device=DEV)[16:]
    assert out.data_ptr() % 32 == 16 and ws.data_ptr() % 32 == 16
    out, lse = c.run(True, out=out, workspace=ws)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert (buf[:off] == 7.0).all() and (buf[off + n:] == 7.0).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_entries_outside_the_pool_read_zeros(dtype):
    c = Case([20], [100], 2, 2, 64, 16, dtype, seed=7)
    zero = c.bt[0, 3].item()
    c.k[zero], c.v[zero] = 0, 0
    want, want_lse = c.run(False)
    for bad in (-1, c.k.shape[0], 0x7fffffff, -0x80000000):
        c.bt[0, 3] = bad
        out, lse = c.run(False)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("dtype", DTYPES)
def test_stale_infinities_past_the_context(dtype):
    for stale in (math.inf, -math.inf, math.nan):
        c = Case([17, 2], [33, 130], 4, 1, 64, 32, dtype, seed=8, stale=stale)
        c.check(*c.run(True), True)


@pytest.mark.parametrize("dtype", DTYPES)
def test_as_decode_for_one_token_each(dtype):
    """Cross attention of one token a sequence is pa_decode's definition: both to half a step
    of each other's errors, judged by the 64-bit check of both."""
    lens = [1, 0, 400, 77]
    c = Case([1, 1, 1, 1], lens, 8, 2, 128, 16, dtype, seed=9, pad=0)
    out, lse = c.run(False)
    c.check(out, lse, False)
    dec = torch.empty_like(out)
    P.pa_decode(dec, c.q, c.k, c.v, c.bt, c.cl, c.scale, 8, 2, 128, 16)
    c.check(dec, None, False)


@pytest.mark.parametrize("dtype", DTYPES)
def test_captured_with_new_lengths(dtype):
    """A captured call replayed after the lengths, tables and starts changed on the device."""
    a = Case([60, 3, 0], [90, 800, 5], 4, 2, 64, 16, dtype, seed=10, pad=40)
    out = torch.full((a.n, 4, 64), 7.0, device=DEV, dtype=a.dt)
    lse = torch.full((a.n, 4), 7.0, device=DEV)
    ws = torch.empty(P.pa_attend_workspace_size(4, 2, 64), dtype=torch.uint8, device=DEV)
    args = (out, a.q, a.k, a.v, a.bt, a.cl, a.qs, a.scale, 4, 2, 64, 16)
    P.pa_attend(*args, causal=True, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        P.pa_attend(*args, causal=True, lse=lse, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    a.check(out, lse, True)
    a.new, a.lens = [5, 90, 8], [70, 333, 2]
    a.cl.copy_(torch.tensor(a.lens))
    a.qs.copy_(torch.tensor([0, 5, 95, 103]))
    out.fill_(7.0)
    lse.fill_(7.0)
    b = Case([0, 0, 0], [90, 800, 16], 4, 2, 64, 16, dtype, seed=11)
    a.bt[:, :b.bt.shape[1]] = b.bt[:, :a.bt.shape[1]]
    a.k.copy_(b.k[:a.k.shape[0]] if b.k.shape[0] >= a.k.shape[0] else torch.randn_like(a.k))
    a.v.copy_(b.v[:a.v.shape[0]] if b.v.shape[0] >= a.v.shape[0] else torch.randn_like(a.v))
    a.bt.clamp_(max=a.k.shape[0] - 1)
    a.k.nan_to_num_(0.5)
    a.v.nan_to_num_(0.5)
    g.replay()
    torch.cuda.synchronize()
    a.check(out, lse, True)


def test_another_stream_and_two_at_once():
    """Two calls at once on two streams, each with its own workspace."""
    a, b = (Case([100, 7], [300, 5000], 8, 2, 128, 16, "bf16", seed=s) for s in (12, 13))
    want = [a.run(True), b.run(True)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [torch.full_like(want[0][0], 7.0), torch.full_like(want[1][0], 7.0)]
    torch.cuda.synchronize()
    for _ in range(5):
        a.run(True, out=outs[0], stream=s1)
        b.run(True, out=outs[1], stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0][0]) and torch.equal(outs[1], want[1][0])


def test_nothing_to_do():
    c = Case([0, 0], [5, 0], 2, 2, 64, 16, "bf16", seed=14, pad=0)
    c.run(True)
    c = Case([0, 0], [5, 0], 2, 2, 64, 16, "bf16", seed=14, pad=4)
    out, lse = c.run(True)
    assert (out == 7.0).all() and (lse == 7.0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("power", [5, 15])
def test_scores_of_any_size(dtype, sign, power):
    """Scores up to 2^40, far apart: each row is the value of its largest score (the others'
    weights are 0), also where the scale is negative: to half a step of its one weight and half
    a step of the output in fp16 and bf16, in fp32 to the 2^-22 that two tf32 terms leave."""
    if dtype == "f16":
        power = 5                                        # (2^5 * 255 is fp16's, 2^15 * 255 is not)
    t = 250
    c = Case([t], [t], 2, 1, 64, 16, dtype, seed=15)
    c.scale = 0.125 * sign
    c.q[...] = 2.0 ** power
    rank = torch.randperm(t, device=DEV) + 1
    slots = (c.bt[0, :16].long()[:, None] * 16 + torch.arange(16, device=DEV)).reshape(-1)[:t]
    c.k.view(-1, 1, 64)[slots] = (rank * 2.0 ** power * sign)[:, None, None].to(c.dt)
    out, lse = c.run(True)
    best = torch.stack([rank[:i + 1].argmax() for i in range(t)])
    want = c.v.view(-1, 64)[slots[best]]
    for h in range(2):
        assert ((out[:t, h] - want).abs().double() <= want.abs().double() * (2.0 ** -22 if dtype == "f32" else torch.finfo(c.dt).eps)).all()
    top = rank[best].double() * 2.0 ** (2 * power + 3)   # 64 * 2^power * 2^power * rank / 8
    assert ((lse[:t, 0].double() - top).abs() <= top * 2.0 ** -21).all()
    assert P.pa_device_errors() == 0


@pytest.mark.parametrize("dtype,new,lens", [("bf16", [300, 40], [900, 5000]), ("f16", [1], [60000]),
                                            ("bf16", [2000], [9000]), ("f32", [20], [3000])])
def test_waits_that_run_out(dtype, new, lens):
    """With a limit shorter than a copy takes, waits may run out: the launch then gives up with its
    copies in flight, returns and says so, and the next one is right."""
    timeouts = P.PA_DEVERR_TIMEOUT_FULL | P.PA_DEVERR_TIMEOUT_EMPTY
    c = Case(new, lens, 4, 2, 128, 16, dtype, seed=16)
    for _ in range(3):
        P.pa_set_wait_limit_ns(1)
        try:
            c.run(True)
            flags = P.pa_device_errors()
        finally:
            P.pa_set_wait_limit_ns(0)
        print(f"[waits] {dtype} {new} {lens}: flags {flags:#x}")
        assert flags & ~timeouts == 0
        c.check(*c.run(True), True)
