"""Plain model of pa_fork_tables: one row and one block at a time, in Python integers."""
from __future__ import annotations

import numpy as np


def fork(tables, lens, parents, extra, free, num_free, block_size):
    """The outputs of pa_fork_tables as a dict of numpy arrays; inputs are left as they were."""
    tables, lens, parents = np.asarray(tables), np.asarray(lens), np.asarray(parents)
    rows, width = tables.shape
    pool = len(free)
    refs = [int(x) + 1 for x in extra]               # references of a block, if it has any
    free = list(np.asarray(free))
    have = min(max(int(num_free), 0), pool)
    tokens = [min(max(int(t), 0), width * block_size) for t in lens]
    blocks = [-(-t // block_size) for t in tokens]
    held = [[int(b) for b in tables[r, :blocks[r]]] for r in range(rows)]

    new, first = [], set()
    for p in parents.tolist():
        if not 0 <= p < rows:
            new.append(None)
            continue
        row = list(held[p])
        half = tokens[p] % block_size != 0
        wants = half and p in first
        first.add(p)
        for b in (row[:-1] if wants else row):
            if 0 <= b < pool:
                refs[b] += 1
        new.append([p, row, wants])
    for r in range(rows):
        for b in held[r]:
            if 0 <= b < pool:
                refs[b] -= 1
    for b in range(pool):
        if refs[b] <= 0:
            refs[b] = 1
            if have < pool:
                free[have] = b
                have += 1

    n = len(new)
    out = {"tables": np.full((n, width), -1, np.int32), "lens": np.zeros(n, np.int32),
           "pairs": np.full((n, 2), -1, np.int32), "granted": np.zeros(n, np.int32)}
    for i, x in enumerate(new):
        if x is None:
            continue
        p, row, wants = x
        if wants and have == 0:
            out["granted"][i] = -1
            for b in row[:-1]:
                if 0 <= b < pool:
                    refs[b] -= 1
            continue
        if wants:
            have -= 1
            out["pairs"][i] = row[-1], free[have]
            row[-1] = int(free[have])
        out["tables"][i, :len(row)] = row
        out["lens"][i], out["granted"][i] = tokens[p], 1
    out["extra"] = np.array([r - 1 for r in refs], np.int32)
    out["free"] = np.array(free, np.int32)
    out["num_free"] = np.array([have], np.int32)
    return out
