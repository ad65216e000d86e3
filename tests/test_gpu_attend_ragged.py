"""pa_attend over ragged batches with heads of 64 dims and with blocks of 32 tokens."""
import pytest

from tests.test_gpu_attend import DTYPES, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,B", [(64, 16), (64, 32), (128, 32)])
@pytest.mark.parametrize("new,lens", [
    ([300], [100]), ([129], [129]), ([0, 1, 0], [5, 6, 0]), ([128, 1, 257, 0, 33], [128, 700, 300, 40, 0]),
    ([3, 2, 1, 8], [1000, 31, 32, 4097]), ([64], [4096 + 31]), ([260], [127]), ([500], [513]),
])
def test_ragged(dtype, causal, d, B, new, lens):
    c = Case(new, lens, 10, 2, d, B, dtype, seed=sum(lens) + d)
    c.check(*c.run(causal), causal)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,B", [(64, 32), (128, 16)])
def test_one_token_rows_beside_a_long_chunk(dtype, d, B):
    """Decode rows and a chunk of a prompt in one call."""
    c = Case([1] * 20 + [900] + [1] * 20, [50 * i + 1 for i in range(20)] + [6000] + [3000 - 37 * i for i in range(20)],
             8, 2, d, B, dtype, seed=5)
    c.check(*c.run(True), True)


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_short_sequences(dtype):
    """One tile of keys an item, a few rows each."""
    c = Case([1 + i % 8 for i in range(200)], [8 + 2 * i for i in range(200)], 4, 4, 64, 16, dtype, seed=6)
    c.check(*c.run(True), True)
