"""Pre-activations up to the largest float32: the checkpoint holds them as the
header says, and gradients are the formula's, against the 64-bit forms, in every
kernel that writes or reads codes of 8 or 16 bits."""
import numpy as np
import pytest

import test_training_gpu as base
import test_training_tiles_gpu as tiles
import training_ref as ref
from helpers import as_f64, to_device, to_host
from test_training_gpu import tre  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

FLT_MAX = float(np.finfo(np.float32).max)
BF16_MAX = (2.0 - 2.0 ** -7) * 2.0 ** 127
# the largest up projection of a block of 64 columns, for a token of size 1
SIZES = [2.0 ** 125, 2.0 ** 126, 1.5 * 2.0 ** 126, 1e38, 2.0 ** 127, BF16_MAX, 1.0]
# (rows of each expert, d, I): the kernels of few tiles, products in ranges, and every kind of tile
SHAPES = {
    "few tiles": ([5, 0, 64, 1], 64),
    "few rows, wide": ([5, 0, 3], 1024),
    "k in ranges": ([5, 0, 64, 1, 70], 1024),
    "k in ranges, tiles of 128 rows": ([300, 0, 129], 1024),
} | {case: (counts, 128) for case, counts in tiles.MANY.items()}
I = 64 * len(SIZES)


def inputs(counts, d, dtype, seed):
    """Ups of the sizes above, gates around 1, and gradients that keep every product finite."""
    rng = np.random.default_rng(seed)
    E, R = len(counts), sum(counts)
    x = rng.standard_normal((R, d))
    x[:, 0] = rng.choice([1.0, 0.5, 0.75, -1.0], R)
    wgu = rng.standard_normal((E, d, 2 * I)) * 0.3 * d ** -0.5
    up = rng.uniform(-1, 1, (E, len(SIZES), 64))
    up[:, :, 5] = 1.0
    wgu[:, 1:, I:I + 64 * (len(SIZES) - 1)] = 0.0      # (one product each: no sum overflows)
    wgu[:, 0, I:] = (up * np.array(SIZES)[:, None]).reshape(E, I)
    wd = rng.standard_normal((E, I, d)) * 2.0 ** -60
    dy = rng.standard_normal((R, d)) * 2.0 ** -50
    dev = [base.put(a, dtype) for a in (x, wgu, wd, dy)]
    return dev, [as_f64(to_host(t)) for t in dev]


@pytest.mark.parametrize("case", list(SHAPES))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward(tre, case, dtype):
    counts, d = SHAPES[case]
    (x, wgu, wd, _), (vx, vgu, vd, _) = inputs(counts, d, dtype, 1)
    y, q, s = tre.moe_grouped_ffn_train(x, base.offsets(counts), wgu, wd)
    base.sync()
    for e, lo, hi in base.spans(counts):
        gu, egu, vy, ey = ref.forward(vx[lo:hi], vgu[e], vd[e], dtype)
        ref.check_codes(q[lo:hi].cpu().numpy(), s[lo:hi].cpu().numpy(), gu, egu)
        ref.near(base.host(y[lo:hi]), vy, ey, dtype, f"y of expert {e}")


@pytest.mark.parametrize("again", [False, True])
@pytest.mark.parametrize("case", list(SHAPES))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward(tre, case, dtype, again):
    counts, d = SHAPES[case]
    (x, wgu, wd, dy), (vx, vgu, vd, vdy) = inputs(counts, d, dtype, 2)
    offs, kw = base.offsets(counts), {}
    if not again:
        _, q, s = tre.moe_grouped_ffn_train(x, offs, wgu, wd)
        kw = dict(gu_q=q, gu_s=s)
    dx, dwgu, dwd = tre.moe_grouped_ffn_backward(x, offs, wgu, wd, dy, **kw)
    base.sync()
    for e, lo, hi in base.spans(counts):
        if again:
            gu, egu = ref.product(vx[lo:hi], np.zeros((hi - lo, d)), vgu[e])
            if dtype == "bf16":   # 16-bit codes in between: half a step of amax / 32767, and their float32
                amax = np.abs(gu + egu).reshape(hi - lo, -1, 64).max(-1)
                egu = egu + np.repeat(amax, 64, 1) * (0.5 / 32767 + 4 * ref.SUM)
        else:
            gu = ref.values(q[lo:hi].cpu().numpy(), s[lo:hi].cpu().numpy())
            assert np.all(np.abs(gu).reshape(hi - lo, 2, -1, 64).max(-1) > 0)
            egu = np.zeros_like(gu)
        a, b, c, _ = ref.backward(vx[lo:hi], vdy[lo:hi], np.ones(hi - lo), gu[:, :I], gu[:, I:], vgu[e], vd[e], dtype,
                                  egu[:, :I], egu[:, I:])
        ref.near(base.host(dx[lo:hi]), *a, dtype, f"dx of expert {e}")
        ref.near(base.host(dwgu[e]), *b, dtype, f"dw_gate_up of expert {e}")
        # (h is held in the type: silu(g) reaches 1.3 here, and a row of dw_down whose h passes the type's largest
        # number in 64 bits, 1.3 * 3.39e38 in one, is no finite number)
        held = np.abs(ref.swiglu(gu[:, :I], gu[:, I:], 0, 0)[0]).max(0) < BF16_MAX
        assert held.sum() >= I - 2
        ref.near(base.host(dwd[e])[held], c[0][held], c[1][held], dtype, f"dw_down of expert {e}")


def test_values_of_the_largest(tre):
    """Codes of both signs times scales up to the largest float32 / 127: one rounding, and finite."""
    rng = np.random.default_rng(3)
    q = rng.integers(-127, 128, (8, 128)).astype(np.int8)
    q[:, ::64] = 127
    q[:, 1::64] = -127
    s = (np.array([2.0 ** 126, 2.0 ** 127, 1e38, BF16_MAX, FLT_MAX, FLT_MAX * 127 / 128, 3e38, 1.0])[:, None, None]
         * np.ones((1, 2, 1)) / 127).astype(np.float32)
    s[4] = np.float32(FLT_MAX) * np.float32(1 / 127)
    want = ref.values(q, s).astype(np.float32)
    assert np.all(np.isfinite(want))
    got = tre.moe_checkpoint_values(to_device(q), to_device(s), base.T().float32)
    base.sync()
    assert np.array_equal(base.host(got), want.astype(np.float64))


@pytest.mark.parametrize("rows", [5, 200, 700])
def test_the_largest_float32_is_kept(tre, rows):
    """Float32 rows whose gates and ups are the largest float32 itself: codes of 127 and their scale (silu(g) u is no
    float32 there, and y is not looked at)."""
    d, n = 64, 64
    x, wgu = np.zeros((rows, d)), np.zeros((1, d, 2 * n))
    x[:, 0] = 1.0
    wgu[0, 0] = FLT_MAX * np.resize([1.0, -1.0, 0.5], 2 * n)
    _, q, s = tre.moe_grouped_ffn_train(base.put(x, "f32"), base.offsets([rows]), base.put(wgu, "f32"),
                                        base.put(np.zeros((1, n, d)), "f32"))
    base.sync()
    ref.check_codes(q.cpu().numpy(), s.cpu().numpy(), np.repeat(wgu[0, :1], rows, 0), np.zeros((rows, 2 * n)))


@pytest.mark.parametrize("T_,E,n", [(1400, 64, 192), (800, 8, 832), (2048, 8, 832), (4096, 4, 832)],
                         ids=["64-row tiles", "128-row tiles", "tall tiles", "256-row tiles"])
def test_an_infinite_h_is_infinite_in_its_weight_gradient(tre, T_, E, n):
    """One kept row whose silu(g) u passes float32 in one column: its routing weight's gradient is <dh, h> = infinity (dh
    is positive there), and every other row's is exact.  n is no multiple of a tile's 256 columns, and the column lies
    in the first block of the tile that ends inside."""
    d, k = 128, 1
    at = (n - 1) // 256 * 256
    idx, w = base.route_given(T_, E, k, T_, drop=0)
    x, dout, wgu, wd, _ = base.exact_inputs(T_, E, d, n, T_)
    u = base.sparse_ints((T_, n), 0.7, T_, 2)
    bad = 77                                # the pair; its grouped row:
    offs, tok, row = base.grouping(tre, base.put(x, "bf16"), idx, E)
    r = int(row[bad])
    u[r, at:at + 64] = 0.0
    u[r, at + 5] = 1.0
    dout[bad], wd[idx[bad, 0], at + 5] = np.abs(dout[bad]), 1.0
    dout[bad, 0] = 1.0
    q, s = base.exact_checkpoint(u)
    s[r, :, at // 64] = 1e20
    got = tre.moe_backward_q8(base.put(x, "bf16"), base.put(wgu, "bf16"), base.put(wd, "bf16"), k,
                              base.put(dout, "bf16"), to_device(idx), to_device(w), tre.Checkpoint(offs, tok, row, q, s))
    base.sync()
    dw = base.host(got["dtopk_w"]).reshape(-1)
    want = np.zeros(T_)
    for e, pairs in enumerate(base.group_numpy(idx, E)):
        rows = row[to_device(pairs)].cpu().numpy()
        want[pairs] = (64 * u[rows] * (dout[pairs] @ wd[e].T)).sum(1)
    assert dw[bad] == np.inf
    assert np.array_equal(np.delete(dw, bad), np.delete(want, bad))
