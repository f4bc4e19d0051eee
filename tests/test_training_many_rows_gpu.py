"""Training calls of more than 65536 rows whose products are cut into ranges of
their k-stages, bit for bit where every sum is exact: deep products of few columns,
whose tiles (one for 256 rows) would leave part of a last round idle."""
import pytest

import training_exact as exact
from test_training_gpu import tre  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


# (rows of each expert, d, I): y in 3, 3 and 2 ranges
@pytest.mark.parametrize("counts,d,I", [([70000], 128, 8192), ([66000], 256, 16000), ([65000, 0, 5100], 64, 8192)])
def test_forward(tre, counts, d, I):
    exact.check_forward(tre, counts, d, I)


# dx in 3, 3 and 2 ranges
@pytest.mark.parametrize("counts,d,I", [([70000], 128, 4096), ([66000], 256, 8000), ([65000, 0, 5100], 64, 4096)])
def test_backward(tre, counts, d, I):
    exact.check_backward(tre, counts, d, I, again=False)


# the most rows that d x I allows, and an expert that has nearly all of them
@pytest.mark.parametrize("counts,d,I", [([9_000_000, 7_777_000], 64, 64), ([100, 5_592_000, 0], 128, 192)])
def test_the_most_rows(tre, counts, d, I):
    assert sum(counts) * 2 * I < 1 << 31 < (sum(counts) + 2000) * 2 * I
    exact.check_forward(tre, counts, d, I)
    exact.check_backward(tre, counts, d, I, again=False)
    exact.check_backward(tre, counts, d, I, again=True)
