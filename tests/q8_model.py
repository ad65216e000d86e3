"""The 8-bit cache's operations and the table step from their definitions: numpy, 64
bits, one block, sequence or request at a time.  Shares no code with the library."""
from __future__ import annotations

import numpy as np


def up(x, m):
    return (x + m - 1) // m * m


def block_bytes(hkv, b, d):
    return hkv * 2 * b * d + up(up(hkv, 2) * 8, 128)


# the 256 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN
CODES = np.array([(-1.0 if c & 0x80 else 1.0) *
                  (np.nan if c & 0x7F == 0x7F else
                   (c & 7) * 2.0 ** -9 if (c >> 3) & 15 == 0 else (8 + (c & 7)) * 2.0 ** (((c >> 3) & 15) - 10))
                  for c in range(256)])


def encode(y):
    """Nearest code of each value (ties to the even code); non-finite values give 0x7f."""
    y = np.asarray(y, dtype=np.float64)
    v = CODES[:127]
    a = np.where(np.isfinite(y), np.abs(y), 0.0)
    assert (a <= 448.0).all()
    hi = np.clip(np.searchsorted(v, a), 1, 126)
    lo = hi - 1
    dl, dh = a - v[lo], v[hi] - a
    c = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo).astype(np.uint8)
    c = c | np.where(np.signbit(y), 0x80, 0).astype(np.uint8)
    return np.where(np.isfinite(y), c, 0x7F).astype(np.uint8)


def need_scale(x):
    """Smallest power of two (2^-126 at least) whose 448-fold covers the finite |x|."""
    x = np.abs(x[np.isfinite(x)])
    top = x.max() if x.size else 0.0
    e = -126
    while top > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


class Cache:
    """A uint8 [NB, bytes] cache with views of its codes and scales."""

    def __init__(self, raw, hkv, b, d):
        self.raw, self.hkv, self.b, self.d = raw, hkv, b, d
        n = hkv * 2 * b * d
        assert raw.shape[1] == block_bytes(hkv, b, d)
        self.codes = raw[:, :n].reshape(-1, hkv, 2, b, d) if raw.size == 0 else \
            np.lib.stride_tricks.as_strided(raw, (raw.shape[0], hkv, 2, b, d),
                                            (raw.strides[0], 2 * b * d, b * d, d, 1))
        self.scales = np.lib.stride_tricks.as_strided(raw[:, n:n + 8].view(np.float32), (raw.shape[0], hkv, 2),
                                                      (raw.strides[0], 8, 4))

    def values(self, ids):
        """float64 [n, Hkv, 2, B, d] of the blocks `ids`."""
        return CODES[self.codes[ids]] * self.scales[ids].astype(np.float64)[..., None, None]


def append(cache, k, v, bt, cl, qs=None):
    """k, v: float64 [N, Hkv, d]; updates the cache's bytes in place."""
    hkv, b = cache.hkv, cache.b
    x = np.stack([k, v], axis=2)                      # [N, Hkv, 2, d]
    if qs is None:
        qs = np.arange(len(cl) + 1)
    for s in range(len(cl)):
        n = int(qs[s + 1] - qs[s])
        rows = {}
        for i in range(n):
            p = int(cl[s]) - n + i
            if p < 0 or p >= bt.shape[1] * b or qs[s] + i >= len(x):
                continue
            blk = int(bt[s, p // b])
            if 0 <= blk < len(cache.raw):
                rows.setdefault(blk, []).append((p % b, int(qs[s]) + i))
        for blk, lst in rows.items():
            offs, toks = [o for o, _ in lst], [t for _, t in lst]
            for h in range(hkv):
                for kv in range(2):
                    new = x[toks, h, kv]              # [m, d]
                    scale = need_scale(new)
                    old = float(cache.scales[blk, h, kv])
                    if 0 not in offs:
                        scale = max(scale, old)
                        if scale > old:
                            rest = [r for r in range(b) if r not in offs]
                            val = CODES[cache.codes[blk, h, kv, rest]] * (old / scale)
                            cache.codes[blk, h, kv, rest] = encode(val)
                    cache.codes[blk, h, kv, offs] = encode(new / scale)
                    cache.scales[blk, h, kv] = scale


def decode(cache, q, bt, cl, scale):
    """(out, abs, smax): out [S, Hq, d] float64; abs = sum p |v| / sum p, the size that
    rounding errors of p are relative to; smax [S, Hq] = largest |scale| * sum |q k|."""
    s_, hq, d = q.shape
    g = hq // cache.hkv
    out = np.zeros((s_, hq, d))
    size = np.zeros((s_, hq, d))
    smax = np.zeros((s_, hq))
    for s in range(s_):
        t = min(max(int(cl[s]), 0), bt.shape[1] * cache.b)
        if t == 0:
            continue
        ids = bt[s, :(t + cache.b - 1) // cache.b]
        good = (ids >= 0) & (ids < len(cache.raw))
        kv = cache.values(np.where(good, ids, 0))
        kv[~good] = 0.0
        kv = kv.transpose(2, 1, 0, 3, 4).reshape(2, cache.hkv, -1, d)[:, :, :t]
        for h in range(hq):
            key, val = kv[0, h // g], kv[1, h // g]
            sc = scale * (key @ q[s, h])
            p = np.exp(sc - sc.max())
            out[s, h] = p @ val / p.sum()
            size[s, h] = p @ np.abs(val) / p.sum()
            smax[s, h] = np.max(abs(scale) * (np.abs(key) @ np.abs(q[s, h])))
    return out, size, smax


def build_tables(bt, cl, new, free, nfree, b, num_slots):
    """One request at a time; returns copies: (bt, cl, free, nfree, granted, qs, slots)."""
    bt, cl, free = bt.copy(), [max(int(t), 0) for t in cl], list(free)
    width, pool = bt.shape[1], len(free)
    have = min(max(int(nfree), 0), pool)
    for s, n in enumerate(new):
        if n < 0:
            for j in range(min(-(-cl[s] // b), width)):
                if have < pool:
                    free[have] = int(bt[s, j])
                    have += 1
    granted, qs, slots = [], [0], []
    blocks = rows = 0
    left = have
    for s, n in enumerate(new):
        n = int(n)
        ok = n <= 0
        if n > 0 and cl[s] + n <= width * b:
            nb = -(-cl[s] // b)
            need = -(-(cl[s] + n) // b) - nb
            blocks += need
            rows += n
            ok = (need == 0 or blocks <= have) and rows <= num_slots
            if ok:
                for i in range(need):
                    left -= 1
                    bt[s, nb + i] = free[left]
                for p in range(cl[s], cl[s] + n):
                    blk = int(bt[s, p // b])
                    slots.append(blk * b + p % b if blk >= 0 else -1)
        granted.append((n if n > 0 else 0) if ok else -1)
        cl[s] = 0 if n < 0 else cl[s] + max(granted[-1], 0)
        qs.append(len(slots))
    slots += [-1] * (num_slots - len(slots))
    return (bt, np.array(cl, dtype=np.int32), np.array(free, dtype=np.int32), left,
            np.array(granted, dtype=np.int32), np.array(qs, dtype=np.int32), np.array(slots, dtype=np.int64))
