"""The training operators write inside their outputs and workspaces alone, for
offsets, tokens, pair rows and expert ids of every value.  All outputs of a call and
its workspace lie in one buffer, with bytes of a known value between them."""
import ctypes

import numpy as np
import pytest

import test_training_gpu as base
from helpers import to_device
from test_training_gpu import tre  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

GAP, MARK = 1 << 18, 0xA5
E = 3
BAD = [[0, -5, 300, 20], [-9, 900, 900, 2 ** 31 - 1], [700, 600, 10, 5], [-2 ** 31, -1, 600, 601], [600, 600, 600, 600],
       [0, 100, 350, 600]]     # (of 600 rows; the last is right)
# (rows, d, I): few tiles, ranges, tiles of 128 rows, tall ones and 256-row ones (bf16)
SIZES = [(600, 64, 128), (600, 1024, 832), (8, 1024, 832), (1300, 64, 128), (360, 128, 832), (1000, 128, 832),
         (1300, 128, 832)]


class Arena:
    """Arrays with gaps between them."""

    def __init__(self, **bytes_of):
        t = base.T()
        self.at, n = {}, GAP
        for name, size in bytes_of.items():
            self.at[name] = (n, n + size)
            n += size + (-size) % 256 + GAP
        self.buf = t.full((n,), MARK, dtype=t.uint8, device="cuda")

    def __getitem__(self, name):
        return ctypes.c_void_p(self.buf.data_ptr() + self.at[name][0])

    def check(self):
        edges = [0] + [x for span in self.at.values() for x in span] + [self.buf.numel()]
        for lo, hi in zip(edges[::2], edges[1::2]):
            assert base.T().all(self.buf[lo:hi] == MARK), (lo, hi, self.at)


def ptr(a):
    return ctypes.c_void_p(a.data_ptr())


def scaled(bad, R):
    return to_device(np.array([b * R // 600 if 0 < b < 2000 else b for b in bad], dtype=np.int32))


@pytest.mark.parametrize("R,d,I", SIZES)
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_grouped(tre, bad, R, d, I, dtype):
    lib, size, dt = tre.load(), 4 if dtype == "f32" else 2, 0 if dtype == "f32" else 1
    offs = scaled(bad, R)
    wgu, wd = base.rand((E, d, 2 * I), dtype, 1)[0], base.rand((E, I, d), dtype, 2)[0]
    x = base.rand((R, d), dtype, 3)[0]
    fws, bws = (f(R, E, d, I, dt) for f in (lib.moe_grouped_ffn_train_workspace_size,
                                           lib.moe_grouped_ffn_backward_workspace_size))
    a = Arena(y=R * d * size, q=R * 2 * I, s=R * 8 * (I // 64), ws=fws)
    sizes = (R, E, d, I, ptr(wgu), ptr(wd), dt)
    assert lib.moe_grouped_ffn_train(ptr(x), ptr(offs), *sizes, a["y"], a["q"], a["s"], a["ws"], fws, None) == 0
    base.sync()
    a.check()
    for q, s in ((a["q"], a["s"]), (None, None)):
        b = Arena(dx=R * d * size, dwgu=E * d * 2 * I * size, dwd=E * I * d * size, ws=bws)
        assert lib.moe_grouped_ffn_backward(ptr(x), ptr(offs), *sizes, q, s, ptr(x), b["dx"], b["dwgu"], b["dwd"],
                                            b["ws"], bws, None) == 0
        base.sync()
        b.check()
    a.check()


@pytest.mark.parametrize("R,d,I", SIZES)
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer(tre, bad, R, d, I, dtype):
    """Two pairs a token: a forward on wild expert ids, and backwards whose grouping is wild."""
    lib, size, dt, k = tre.load(), 4 if dtype == "f32" else 2, 0 if dtype == "f32" else 1, 2
    T_ = R // k
    rng = np.random.default_rng(R + d)
    wild = to_device(rng.integers(-2 ** 31, 2 ** 31, R).astype(np.int32))
    near = to_device(rng.integers(-3, R + 3, R).astype(np.int32))
    ids = to_device(np.where(rng.random(R) < 0.5, rng.integers(-2, E + 2, R),
                             rng.integers(-2 ** 31, 2 ** 31, R)).astype(np.int32))
    w = base.T().ones(R, device="cuda")
    wgu, wd = base.rand((E, d, 2 * I), dtype, 1)[0], base.rand((E, I, d), dtype, 2)[0]
    x = base.rand((T_, d), dtype, 3)[0]
    sizes = (T_, d, E, k, I, ptr(wgu), ptr(wd), dt)
    fws, bws = (f(T_, d, E, k, I, dt) for f in (lib.moe_forward_train_q8_workspace_size,
                                               lib.moe_backward_q8_workspace_size))
    a = Arena(offs=4 * (E + 1), tok=4 * R, row=4 * R, q=R * 2 * I, s=R * 8 * (I // 64), out=T_ * d * size, ws=fws)
    assert lib.moe_forward_train_q8(ptr(x), None, *sizes, ptr(ids), ptr(w), a["offs"], a["tok"], a["row"], a["q"],
                                    a["s"], a["out"], a["ws"], fws, None) == 0
    base.sync()
    a.check()
    offs = scaled(bad, R)
    for idx, offsets, tok, row in ((ids, a["offs"], a["tok"], a["row"]), (near, ptr(offs), ptr(wild), ptr(near)),
                                   (wild, ptr(offs), ptr(near), ptr(wild))):
        b = Arena(dx=T_ * d * size, dwgu=E * d * 2 * I * size, dwd=E * I * d * size, dw=4 * R, dlogits=4 * T_ * E,
                  ws=bws)
        assert lib.moe_backward_q8(ptr(x), *sizes, ptr(idx), ptr(w), offsets, tok, row, a["q"], a["s"], ptr(x),
                                   b["dx"], b["dwgu"], b["dwd"], b["dw"], b["dlogits"], b["ws"], bws, None) == 0
        base.sync()
        b.check()
    a.check()


def test_values(tre):
    for dtype, size, dt in (("bf16", 2, 1), ("f32", 4, 0)):
        for rows, I in ((1, 64), (5, 192), (77, 2880)):
            q = base.T().zeros((rows, 2 * I), dtype=base.T().int8, device="cuda")
            s = base.T().ones((rows, 2, I // 64), device="cuda")
            a = Arena(gu=rows * 2 * I * size)
            assert tre.load().moe_checkpoint_values(ptr(q), ptr(s), rows, I, dt, a["gu"], None) == 0
            base.sync()
            a.check()
