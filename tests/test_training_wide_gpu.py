"""The training operators at the widest calls that they take, where a tile of 288
rows would pass 31-bit byte offsets: bit for bit where every sum is exact."""
import pytest

import training_exact as exact
from test_training_gpu import tre  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

WIDEST = (1 << 21) - 64
ROWS = [288]     # one expert: a tall tile, were the rows not so wide


@pytest.mark.parametrize("d,I", [(128, WIDEST), (WIDEST, 128)])
def test_forward(tre, d, I):
    exact.check_forward(tre, ROWS, d, I)


@pytest.mark.parametrize("again", [False, True])
@pytest.mark.parametrize("d,I", [(128, WIDEST), (WIDEST, 128)])
def test_backward(tre, d, I, again):
    exact.check_backward(tre, ROWS, d, I, again)
