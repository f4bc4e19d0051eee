"""The training operators at the widest calls that they take, where a tile of 288
rows would pass 31-bit byte offsets: bit for bit where every sum is exact."""
import numpy as np
import pytest
import torch

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


# few rows and long sums, on both sides of the rule that sends such calls to the kernels of few tiles
LONG = [([1], 64, 16384), ([64], 64, 8192), ([0, 5, 1], 512, 16384), ([2, 0], 16384, 64), ([64], 64, 2880),
        ([1] + [0] * 63, 512, 8192), ([3, 0], 4096, 64)]


@pytest.mark.parametrize("counts,d,I", LONG)
def test_few_rows_and_long_sums(tre, counts, d, I):
    exact.check_forward(tre, counts, d, I)
    exact.check_backward(tre, counts, d, I, again=False)
    exact.check_layer(tre, np.repeat(np.arange(len(counts)), counts)[:, None].astype(np.int32), d, len(counts), I)


@pytest.mark.parametrize("d,I", [(128, WIDEST), (WIDEST, 128)])
def test_float32(tre, d, I):
    exact.check_forward(tre, ROWS, d, I, torch.float32)
    exact.check_backward(tre, ROWS, d, I, False, torch.float32)
