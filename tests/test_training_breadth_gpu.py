"""Calls of the training operators that their documentation allows at its edges:
buffers far larger than their rows, 256 experts, more pairs a token than experts,
float32 steps of some thousand rows; bit for bit where every sum is exact."""
import numpy as np
import pytest
import torch

import training_exact as exact
from test_training_gpu import tre  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# rows of each expert of 256
EVEN = [(7 * e) % 5 for e in range(256)]
LAST = [0] * 255 + [300]
FULL = [128 + (37 * e) % 40 for e in range(256)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("counts,extra,d,I", [([5, 0, 70], 4096, 128, 192), ([5, 0, 70], 4096, 1024, 832),
                                              ([0, 1], 20000, 64, 128), ([3], 700, 2048, 64), ([0, 0], 1000, 128, 832),
                                              ([300, 20] * 4, 3000, 128, 1024)])
def test_buffers_larger_than_their_rows(tre, counts, extra, d, I, dtype):
    exact.check_forward(tre, counts, d, I, TYPES[dtype], extra)
    exact.check_backward(tre, counts, d, I, False, TYPES[dtype], extra)
    if dtype == "bf16":
        exact.check_backward(tre, counts, d, I, True, extra=extra)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("counts", [EVEN, LAST, FULL], ids=["even", "last", "full"])
def test_256_experts(tre, counts, dtype):
    for d, I in ((128, 192), (64, 832)):
        exact.check_forward(tre, counts, d, I, TYPES[dtype])
        exact.check_backward(tre, counts, d, I, False, TYPES[dtype])


def pairs(T_, k, E, drop, seed):
    rng = np.random.default_rng(seed)
    idx = rng.integers(0, E, (T_, k))
    return np.where(rng.random((T_, k)) < drop, -1, idx).astype(np.int32)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T_,k,E,drop,d,I", [(9, 300, 4, 0.1, 64, 64), (40, 256, 256, 0, 64, 128), (2000, 4, 16, 0.95, 128, 832),
                                             (3000, 2, 8, 0.2, 512, 448), (1, 1, 256, 0, 128, 64), (700, 3, 256, 0, 192, 64)])
def test_layers(tre, T_, k, E, drop, d, I, dtype):
    exact.check_layer(tre, pairs(T_, k, E, drop, T_), d, E, I, TYPES[dtype])


@pytest.mark.parametrize("counts,d,I", [([1500, 0, 700, 1, 900], 512, 448), ([4000], 128, 1024), ([130] * 40, 576, 704)])
def test_float32_steps_of_some_thousand_rows(tre, counts, d, I):
    exact.check_forward(tre, counts, d, I, torch.float32)
    exact.check_backward(tre, counts, d, I, False, torch.float32)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T_,k,E,d,I", [(40, 3, 5, 64, 128), (700, 2, 16, 128, 832), (2000, 2, 4, 128, 832)])
def test_dropped_pairs_hide_what_is_theirs(tre, T_, k, E, d, I, dtype):
    """Weights of dropped pairs, and rows of tokens that have no other pair, may hold anything: outputs are those of zeros
    there, bit for bit."""
    idx = pairs(T_, k, E, 0.4, T_)
    idx[::7] = -1
    idx[1::7, 0] = E + 3                    # an id that is no expert's here drops its pair too
    gone = torch.from_numpy((idx < 0) | (idx >= E)).cuda()
    g = exact.gen(T_)
    wgu, wd = exact.weights(E, d, I, g, TYPES[dtype])
    x, dout = exact.rows_of(T_, d, g, TYPES[dtype])
    w = torch.rand((T_, k), generator=g, device="cuda")
    idx = torch.from_numpy(idx).cuda()
    got = []
    for hidden in (0.0, float("nan"), float("inf"), -3e38):
        xs, ds, ws = x.clone(), dout.clone(), w.clone()
        ws[gone] = hidden
        xs[gone.all(1)], ds[gone.all(1)] = hidden, hidden
        out, _, _, kept = tre.moe_forward_train_q8(xs, wgu, wd, k, topk_idx=idx, topk_w=ws)
        r = tre.moe_backward_q8(xs, wgu, wd, k, ds, idx, ws, kept, want_dlogits=True)
        got.append([out, *r.values()])
    torch.cuda.synchronize()
    for other in got[1:]:
        for a, b, name in zip(got[0], other, ("out", "dx", "dw_gate_up", "dw_down", "dtopk_w", "dlogits")):
            assert torch.equal(a, b), name
