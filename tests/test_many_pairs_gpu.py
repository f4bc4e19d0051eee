"""moe_backward of more given pairs a token than there can be experts, against the
oracle."""
import numpy as np
import pytest

import test_parity_gpu as parity
import workloads
from test_parity_gpu import tre  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k", [(9, 257), (6, 700)])
def test_backward_of_more_pairs_than_experts(tre, T, k, dtype):
    inp = workloads.make_custom(T=T, d=64, E=4, k=1, I=64, dtype=dtype, seed=k, logits=None)
    rng = np.random.default_rng(k)
    inp.k = k
    inp.pair_expert = rng.integers(-1, 4, T * k).astype(np.int32)
    inp.pair_w = rng.random(T * k).astype(np.float32)
    parity.check_backward(tre, inp, seed=T)
