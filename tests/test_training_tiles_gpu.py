"""The training operators' bf16 kernels of many tiles, and those whose sums are
cut into ranges: the checks of test_training_gpu at sizes that lead there (the
sizes of that file mostly go to the kernels of few tiles)."""
import numpy as np
import pytest

import test_training_gpu as base
from helpers import to_device
from test_training_gpu import tre  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

# rows of each expert: as base.COUNTS, times as many experts as make the tiles many
MANY = {
    "64-row tiles": base.COUNTS["64-row tiles"] * 14,
    "128-row tiles": base.COUNTS["128-row tiles"] * 14,
    "tall tiles": base.COUNTS["tall tiles"] * 8,
    "tall and not": base.COUNTS["tall and not"] * 5,
    "256-row tiles": base.COUNTS["256-row tiles"] * 2,
}
# (rows of each expert, d, I) where sums are cut
CUT = {
    "k in ranges": ([5, 0, 64, 1, 70], 1024, 832),
    "k in ranges, tiles of 128 rows": ([300, 0, 129], 832, 1024),
    "few rows, wide": ([5, 0, 3], 1024, 832),
    "one row, widest": ([0, 1], 2880, 64),
    "rows in ranges": ([3000], 64, 128),
    "rows in ranges, an expert of few": ([2, 2500, 0], 128, 64),
}


@pytest.fixture
def many(monkeypatch):
    for case, counts in MANY.items():
        monkeypatch.setitem(base.COUNTS, case, counts)


@pytest.fixture
def cut(monkeypatch):
    for case, (counts, _, _) in CUT.items():
        monkeypatch.setitem(base.COUNTS, case, counts)


@pytest.mark.parametrize("d,I", [(64, 64), (128, 192)])
@pytest.mark.parametrize("case", list(MANY))
def test_grouped_backward_exact(tre, many, case, d, I):
    base.test_grouped_backward_exact(tre, case, d, I, "bf16")


@pytest.mark.parametrize("case", list(CUT))
def test_grouped_backward_exact_cut(tre, cut, case):
    base.test_grouped_backward_exact(tre, case, *CUT[case][1:], "bf16")


@pytest.mark.parametrize("again", [False, True])
@pytest.mark.parametrize("case", list(MANY))
def test_grouped_backward(tre, many, case, again):
    base.test_grouped_backward(tre, case, 128, 192, "bf16", again)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("again", [False, True])
@pytest.mark.parametrize("case", list(CUT))
def test_grouped_backward_cut(tre, cut, case, again, dtype):
    base.test_grouped_backward(tre, case, *CUT[case][1:], dtype, again)


@pytest.mark.parametrize("case", list(MANY))
def test_grouped_train(tre, many, case):
    base.test_grouped_train(tre, case, 128, 192, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", list(CUT))
def test_grouped_train_cut(tre, cut, case, dtype):
    base.test_grouped_train(tre, case, *CUT[case][1:], dtype)


@pytest.mark.parametrize("T_,d,E,k,I", [(700, 128, 64, 2, 192), (300, 1024, 6, 2, 832), (4, 1024, 3, 2, 832),
                                        (2000, 64, 2, 2, 128), (1, 64, 4, 3, 2880)])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_step(tre, T_, d, E, k, I, given, dtype):
    base.test_layer_step(tre, T_, d, E, k, I, given, dtype)


@pytest.mark.parametrize("case", ["64-row tiles", "128-row tiles", "tall tiles", "256-row tiles"])
def test_checkpoint_of_extreme_rows(tre, many, case):
    base.test_checkpoint_of_extreme_rows(tre, case, "bf16")


@pytest.mark.parametrize("case", ["64-row tiles", "128-row tiles", "tall tiles", "256-row tiles"])
def test_nan_stays_in_its_row_and_expert(tre, many, case):
    base.test_nan_stays_in_its_row_and_expert(tre, case, "bf16")


@pytest.mark.parametrize("bad", [[0, -5, 300, 20], [-9, 900, 900, 2 ** 31 - 1], [700, 600, 10, 5],
                                 [-2 ** 31, -1, 600, 601], [600, 600, 600, 600]])
@pytest.mark.parametrize("R,d,I", [(600, 1024, 832), (8, 1024, 832), (1300, 64, 128)])
def test_arrays_out_of_range(tre, bad, R, d, I):
    """As base.test_arrays_out_of_range, in the kernels of these sizes."""
    E, dtype = 3, "bf16"
    bad = [b * R // 600 if 0 < b < 2000 else b for b in bad]
    offs = to_device(np.array(bad, dtype=np.int32))
    wgu, wd = base.rand((E, d, 2 * I), dtype, 1)[0], base.rand((E, I, d), dtype, 2)[0]
    guard = 4096
    whole = base.sentinel((R + 2 * guard, d), dtype)
    x, _ = base.rand((R, d), dtype, 3)
    y, q, s = tre.moe_grouped_ffn_train(x, offs, wgu, wd, y_perm=whole[guard:guard + R])
    tre.moe_grouped_ffn_backward(x, offs, wgu, wd, x, gu_q=q, gu_s=s, dx_perm=whole[guard:guard + R])
    tre.moe_grouped_ffn_backward(x, offs, wgu, wd, x, dx_perm=whole[guard:guard + R])
    rng = np.random.default_rng(1)
    wild = to_device(rng.integers(-2 ** 31, 2 ** 31, R).astype(np.int32))
    near = to_device(rng.integers(-3, R + 3, R).astype(np.int32))
    for tok, row in ((wild, near), (near, wild)):
        kept = tre.Checkpoint(offs, tok, row, q, s)
        tre.moe_backward_q8(x[:R // 2], wgu, wd, 2, x[:R // 2], near.view(-1, 2),
                            base.T().ones((R // 2, 2), device="cuda"), kept, want_dlogits=True,
                            dx=whole[guard:guard + R // 2])
    base.sync()
    edge = base.sentinel((1,), dtype)
    assert base.T().all(whole[:guard] == edge) and base.T().all(whole[guard + R:] == edge)


def layer(**sizes):
    return lambda tre, dtype, seed=0: base.layer_step(tre, dtype, seed, **sizes)


def grouped(**sizes):
    return lambda tre, dtype, seed=0: base.grouped_step(tre, dtype, seed, **sizes)


STEPS = {
    "layer, many tiles": layer(T_=700, E=64),
    "layer, k in ranges": layer(T_=300, d=1024, E=6, I=832),
    "layer, few rows, wide": layer(T_=4, d=1024, E=3, I=832),
    "layer, rows in ranges": layer(T_=2000, d=64, E=2, I=128),
    "grouped, many tiles": grouped(counts=MANY["tall tiles"]),
    "grouped, k in ranges": grouped(counts=(70, 0, 300), d=1024, I=832),
    "grouped, few rows, wide": grouped(counts=(5, 0, 3), d=1024, I=832),
    "grouped, rows in ranges": grouped(counts=(2, 2500, 0), d=128, I=64),
}


@pytest.mark.parametrize("step", list(STEPS))
def test_graph_replays(tre, step):
    base.test_graph_replays(tre, STEPS[step], "bf16")


@pytest.mark.parametrize("step", list(STEPS))
def test_two_streams(tre, step):
    base.test_two_streams(tre, STEPS[step], "bf16")


@pytest.mark.parametrize("step", list(STEPS))
def test_device_checked_build_equals_release(tre, step):
    run, _ = STEPS[step](tre, "bf16")
    want = [t.clone() for t in run()]
    base.sync()
    release = tre._lib
    try:
        tre._lib = tre.open_library(tre.DEBUG_LIB_PATH)
        got = run()
        base.sync()
    finally:
        tre._lib = release
    for a, b in zip(got, want):
        assert base.T().equal(a.view(base.T().uint8), b.view(base.T().uint8))
