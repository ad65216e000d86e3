"""pa_fork_tables on the GPU against a plain model, equal in every entry."""
import numpy as np
import pytest
import torch

import paged_kv_cache_79_gb300 as P
from tests import fork_model as F

pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).to(DEV)


class Batch:
    """A batch on the device: tables, lengths, references and free list."""

    def __init__(self, lens, block_size, pool, width, rng, share=()):
        self.B = block_size
        lens = np.asarray(lens, dtype=np.int32)
        nbs = -(-lens // block_size)
        order = rng.permutation(pool).astype(np.int32)
        bt = np.full((len(lens), width), -1, np.int32)
        at = 0
        extra = np.zeros(pool, np.int32)
        for s, n in enumerate(nbs):
            bt[s, :n] = order[at:at + n]
            at += n
        spare = []
        for a, b, n in share:                         # row b's first n blocks are row a's
            spare += bt[b, :n].tolist()
            bt[b, :n] = bt[a, :n]
            extra[bt[a, :n]] += 1
        free = np.zeros(pool, np.int32)
        rest = order[at:].tolist() + spare
        free[:len(rest)] = rest
        self.tables, self.lens, self.extra, self.free, self.num_free = bt, lens, extra, free, len(rest)

    def run(self, parents, num_free=None, **kw):
        """(got, want): pa_fork_tables's outputs and the model's."""
        nf = self.num_free if num_free is None else num_free
        parents = np.asarray(parents, np.int32)
        n = len(parents)
        want = F.fork(self.tables, self.lens, parents, self.extra, self.free, nf, self.B)
        t = {k: dev(getattr(self, k)) for k in ("tables", "lens", "extra", "free")}
        num_free = dev([nf])
        i32 = dict(dtype=torch.int32, device=DEV)
        out = torch.full((n, self.tables.shape[1]), 77, **i32)
        lens, pairs, granted = torch.full((n,), 77, **i32), torch.full((n, 2), 77, **i32), torch.full((n,), 77, **i32)
        P.pa_fork_tables(out, lens, t["tables"], t["lens"], dev(parents), t["extra"], t["free"], num_free, self.B,
                         pairs, granted, **kw)
        torch.cuda.synchronize()
        got = {"tables": out, "lens": lens, "pairs": pairs, "granted": granted, "extra": t["extra"],
               "free": t["free"], "num_free": num_free}
        return {k: v.cpu().numpy() for k, v in got.items()}, want


def same(got, want):
    for k in want:
        assert np.array_equal(got[k], want[k]), (k, got[k], want[k])


@pytest.mark.parametrize("block_size", [16, 32, 5])
@pytest.mark.parametrize("parents", [
    [0], [0, 0], [0, 0, 0, 1], [1, 1, 1], [-1], [-1, 2, 9, 0], [2, 1, 0], [], [3, 3, 2, 2, 1, 1, 0, 0],
    [-5, 0x7fffffff, 0],
])
def test_small(block_size, parents):
    """Forks, swaps, releases, parents outside the batch; empty, full and half-filled blocks."""
    rng = np.random.default_rng(1)
    b = Batch([3 * block_size, 0, 2 * block_size + 1, 1], block_size, 40, 6, rng, share=[(0, 2, 2)])
    same(*b.run(parents))


@pytest.mark.parametrize("rows,children,pool,width,hi", [
    (1, 1, 1 << 17, 3, 40), (16, 128, 4000, 130, 2048), (256, 256, 30000, 200, 3000), (1025, 2049, 90000, 90, 1200),
    (3, 1025, 2000, 1100, 17000), (2, 2, 9000, 4100, 65000),
])
@pytest.mark.parametrize("stays", [0.0, 0.7])
def test_random(rows, children, pool, width, hi, stays):
    """Wide tables (several parts of a row), more than a thousand rows, shared prefixes."""
    rng = np.random.default_rng(rows + children)
    lens = rng.integers(0, hi + 1, size=rows)
    lens[rng.random(rows) < 0.2] //= 16
    share = [(s - 1, s, int(min(lens[s - 1], lens[s]) // 16 // 2)) for s in range(1, rows, 2)]
    b = Batch(lens, 16, max(pool, int((-(-lens // 16)).sum()) + 5), width, rng, share)
    parents = np.where(rng.random(children) < stays, np.arange(children), rng.integers(-1, rows, size=children))
    got, want = b.run(parents)
    same(got, want)


@pytest.mark.parametrize("num_free", [0, 1, 2, 5, -3, 1 << 30])
def test_counts_at_any_4_bytes(num_free):
    """extra_refs that does not begin at 16 bytes, as a slice of a larger buffer may."""
    rng = np.random.default_rng(11)
    b = Batch(rng.integers(0, 200, size=50), 16, 1500, 14, rng, share=[(0, 1, 1)])
    parents = rng.integers(-1, 50, size=60)
    want = F.fork(b.tables, b.lens, parents, b.extra, b.free, num_free, 16)
    buf = torch.full((1503,), 9, dtype=torch.int32, device=DEV)
    extra = buf[1:1501]
    extra.copy_(dev(b.extra))
    i32 = dict(dtype=torch.int32, device=DEV)
    out, lens, pairs, granted = torch.empty(60, 14, **i32), torch.empty(60, **i32), torch.empty(60, 2, **i32), torch.empty(60, **i32)
    free, nf = dev(b.free), dev([num_free])
    P.pa_fork_tables(out, lens, dev(b.tables), dev(b.lens), dev(parents), extra, free, nf, 16, pairs, granted)
    got = {"tables": out, "lens": lens, "pairs": pairs, "granted": granted, "extra": extra, "free": free, "num_free": nf}
    same({k: v.cpu().numpy() for k, v in got.items()}, want)
    assert buf[0] == 9 and (buf[1501:] == 9).all()


@pytest.mark.parametrize("num_free", [0, 1, 2, 5, -3, 1 << 30])
def test_short_pool(num_free):
    """Refused rows are empty, hold nothing, and the ones that need no block go on."""
    rng = np.random.default_rng(5)
    b = Batch([33, 48, 7], 16, 64, 5, rng)
    got, want = b.run([0, 0, 1, 1, 0, 2, 2, 0], num_free=num_free)
    same(got, want)
    if num_free <= 0:
        assert got["granted"].tolist() == [1, -1, 1, 1, -1, 1, -1, -1]


def test_released_blocks_serve_the_copies():
    rng = np.random.default_rng(6)
    b = Batch([40, 64], 16, 8, 4, rng)
    got, want = b.run([0, 0, 0], num_free=0)
    same(got, want)
    assert got["granted"].tolist() == [1, 1, 1] and got["num_free"][0] == 2


def test_entries_and_lengths_outside():
    """Lengths past the table are clamped, table entries outside the pool counted nowhere."""
    rng = np.random.default_rng(7)
    b = Batch([40, 64, 20], 16, 16, 4, rng)
    b.lens = np.array([1 << 30, -4, 20], np.int32)
    b.tables[0] = [3, 1 << 30, -7, 5]
    same(*b.run([0, 0, 1, 2, 2, -1]))


def test_in_place_count_and_repeat():
    """num_free_out apart leaves num_free; the same call again from the same inputs gives the same bits."""
    rng = np.random.default_rng(8)
    b = Batch(rng.integers(0, 900, size=300), 16, 20000, 60, rng, share=[(2, 3, 1)])
    parents = rng.integers(-1, 300, size=400)
    nf = dev([0])
    got, want = b.run(parents, num_free_out=nf)
    assert got["num_free"][0] == b.num_free and int(nf) == want["num_free"][0]
    want["num_free"] = got["num_free"]
    same(got, want)
    again, _ = b.run(parents, num_free_out=nf)
    same(again, got)


def test_steps_keep_the_pool_whole():
    """Thirty steps of a beam search: after each, references and free list account for every block."""
    rng = np.random.default_rng(9)
    B, S, W, pool = 16, 24, 12, 400
    b = Batch(rng.integers(1, 60, size=S), B, pool, W, rng)
    for step in range(30):
        parents = np.where(rng.random(S) < 0.5, np.arange(S), rng.integers(-1, S, size=S))
        got, want = b.run(parents)
        same(got, want)
        b.tables, b.lens, b.extra, b.free = got["tables"], got["lens"], got["extra"], got["free"]
        b.num_free = int(got["num_free"][0])
        count = np.zeros(pool, int)
        for s in range(S):
            n = -(-int(b.lens[s]) // B)
            count[b.tables[s, :n]] += 1
            if b.lens[s] % B:
                assert count[b.tables[s, n - 1]] == 1
        free = b.free[:b.num_free]
        assert len(set(free.tolist())) == len(free) and not count[free].any()
        assert np.array_equal(np.maximum(count - 1, 0), b.extra)
        assert (count > 0).sum() + len(free) == pool
        b.lens = np.where(b.lens % B > 0, np.minimum(b.lens + rng.integers(0, 2, size=S), (b.lens + B - 1) // B * B), b.lens).astype(np.int32)


def test_captured_and_on_another_stream():
    """The call captured into a graph and replayed on the state that each replay left."""
    rng = np.random.default_rng(10)
    b = Batch(rng.integers(1, 300, size=20), 16, 2000, 24, rng)
    parents = np.concatenate([np.arange(18), [3, -1]])
    i32 = dict(dtype=torch.int32, device=DEV)
    t = {k: dev(getattr(b, k)) for k in ("tables", "lens", "extra", "free")}
    nf, pd = dev([b.num_free]), dev(parents)
    out, lens, pairs, granted = (torch.zeros(20, 24, **i32), torch.zeros(20, **i32), torch.zeros(20, 2, **i32),
                                 torch.zeros(20, **i32))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        P.pa_fork_tables(out, lens, t["tables"], t["lens"], pd, t["extra"], t["free"], nf, 16, pairs, granted)
        t["tables"].copy_(out)
        t["lens"].copy_(lens)
    state = (b.tables, b.lens, b.extra, b.free, b.num_free)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        w = F.fork(state[0], state[1], parents, state[2], state[3], state[4], 16)
        state = (w["tables"], w["lens"], w["extra"], w["free"], int(w["num_free"][0]))
        for k, v in (("tables", out), ("lens", lens), ("extra", t["extra"]), ("free", t["free"]), ("pairs", pairs)):
            assert np.array_equal(v.cpu().numpy(), w[k]), k
