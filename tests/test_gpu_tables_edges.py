"""pa_build_tables at the ends of its ranges, against the one-request-at-a-time model."""
import numpy as np
import pytest

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
