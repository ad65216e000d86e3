"""pa_build_tables at the ends of its ranges, against the one-request-at-a-time model."""
import numpy as np
import pytest
import torch

import paged_kv_cache_79_gb300 as P
from tests.test_gpu_tables import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("b,width,cl,new", [
    (2 ** 31 - 1, 1, [5], [1]),                       # length + B - 1 passes 2^31
    (2 ** 31 - 1, 1, [2 ** 31 - 9], [3]),
    (10 ** 9, 2, [2 * 10 ** 9 - 7], [7]),
    (10 ** 9, 2, [10 ** 9, 10 ** 9 - 3], [4, 5]),     # a new block, and one that spans two
    (2 ** 30, 1, [2 ** 30 - 4], [4]),
    (7 * 10 ** 8, 3, [7 * 10 ** 8 + 1, 14 * 10 ** 8 + 5], [2, 9]),
])
def test_blocks_of_nearly_all_the_range(b, width, cl, new):
    """A block size near the limit of 2^31 tokens per table row: own blocks are found."""
    blocks = (2 ** 31 - 1) // b
    bt = np.full((len(cl), width), -1, dtype=np.int32)
    for s, t in enumerate(cl):
        bt[s, :-(-t // b)] = 0                        # (the values are not looked into)
    free = np.zeros(blocks, dtype=np.int32)
    for left in {0, min(1, blocks)}:
        want = check(bt, np.array(cl, dtype=np.int32), np.array(new), free, left, b, 40)
        if left:
            assert (want[4] == new).sum() >= 1


def granted(cl, new, left, num_slots, b=16, width=8):
    bt = np.full((len(cl), width), -1, dtype=np.int32)
    at = 20
    for s, t in enumerate(cl):
        for j in range(min(-(-t // b), width)):
            bt[s, j], at = at, at + 1
    free = np.arange(64, dtype=np.int32)
    return check(bt, np.array(cl, dtype=np.int32), np.array(new), free, left, b, num_slots)[4].tolist()


def test_who_is_served_behind_a_refused_request():
    # 40 slots: the prompt of 100 tokens has none, and nobody behind it; those before it have
    assert granted([5, 0, 5, 5], [1, 100, 1, 0], 9, 40) == [1, -1, -1, 0]
    # 2 blocks: the prompt of 50 needs 4; a step within its own block goes on, a new block not
    assert granted([5, 0, 5, 16], [1, 50, 1, 1], 2, 400) == [1, -1, 1, -1]
    # its slots count although it is refused
    assert granted([5, 0, 5, 5], [1, 50, 1, 1], 2, 52) == [1, -1, 1, -1]
    # a row that is too short counts nothing
    assert granted([5, 0, 5, 16], [1, 200, 1, 1], 2, 40) == [1, -1, 1, 1]


def test_no_new_tokens_are_granted_whatever_the_length():
    assert granted([0, 128, 129, 10 ** 9], [0, 0, 0, 0], 0, 0) == [0, 0, 0, 0]


def test_the_longest_slot_map():
    """2^31 - 1024 slots, 17 GB: two requests' own, then padding to the very end."""
    n, b = 2 ** 31 - 1024, 16
    i32 = dict(dtype=torch.int32, device="cuda")
    slots = torch.empty(n, dtype=torch.int64, device="cuda")
    slots[:100], slots[-5000:] = 7, 7
    bt, cl = torch.full((2, 4), -1, **i32), torch.zeros(2, **i32)
    qs, granted, nfree = torch.zeros(3, **i32), torch.zeros(2, **i32), torch.tensor([6], **i32)
    P.pa_build_tables(bt, cl, torch.tensor([20, 33], **i32), torch.arange(6, **i32), nfree, b, slots, qs, granted)
    assert granted.tolist() == [20, 33] and qs.tolist() == [0, 20, 53] and nfree.item() == 1
    own = [5 * b + i for i in range(16)] + [4 * b + i for i in range(4)] + \
        [3 * b + i for i in range(16)] + [2 * b + i for i in range(16)] + [b]
    assert slots[:53].tolist() == own and (slots[53:100] == -1).all() and (slots[-5000:] == -1).all()
    assert (slots[n // 2 - 5:n // 2 + 70000] == -1).all()
