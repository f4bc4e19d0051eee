"""The training operators at the widest calls that they take, where a tile of 288
rows would pass 31-bit byte offsets: bit for bit where every sum is exact.

The gates are 64, so that silu(g) = 64 in float32 and h = 64 u, dg = dh u, du = 64
dh, with small whole numbers everywhere else.  Reference sums are float64, in
pieces of the width."""
import pytest

import test_training_gpu as base
from test_training_gpu import tre  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

WIDEST = (1 << 21) - 64
ROWS, EXTRA = 288, 2     # one expert: a tall tile, were the rows not so wide; rows behind it
PIECE = 1 << 16


def ints(shape, top, density, g):
    """Whole numbers in [-top, top], most of them zero for a small density, as bf16."""
    t = base.T()
    v = t.randint(-top, top + 1, shape, generator=g, device="cuda", dtype=t.int8)
    keep = t.rand(shape, generator=g, device="cuda") < density if density < 1 else None
    return (v if keep is None else v * keep).to(t.bfloat16)


def pieces(n):
    return [slice(a, min(a + PIECE, n)) for a in range(0, n, PIECE)]


def same(got, want, name):
    """want (float64, exact in float32) rounded to bf16 once."""
    t = base.T()
    f = want.float()
    assert t.equal(f.double(), want), name
    assert t.equal(got, f.to(t.bfloat16)), name


def inputs(d, I):
    t = base.T()
    g = t.Generator(device="cuda")
    g.manual_seed(d + I)
    offs = t.tensor([0, ROWS], dtype=t.int32, device="cuda")
    p = min(1.0, (3.0 / d) ** 0.5)       # dh: sums of d products, a few of them not zero
    x, dy = ints((ROWS + EXTRA, d), 1, 1.0, g), ints((ROWS + EXTRA, d), 1, p, g)
    x[:, 0] = 1.0
    wgu = ints((1, d, 2 * I), 1, min(1.0, 128.0 / d), g)
    wgu[0, :, :I] = 0.0
    wgu[0, 0, :I] = 64.0                 # g = 64; only dx's first column is a sum over the gates
    return offs, x, dy, wgu, ints((1, I, d), 1, p, g)


@pytest.mark.parametrize("d,I", [(128, WIDEST), (WIDEST, 128)])
def test_forward(tre, d, I):
    t = base.T()
    offs, x, _, wgu, wd = inputs(d, I)
    R = ROWS + EXTRA
    y = base.sentinel((R, d), "bf16")
    q = t.full((R, 2 * I), 77, dtype=t.int8, device="cuda")
    s = t.full((R, 2, I // 64), -3.0, device="cuda")
    tre.moe_grouped_ffn_train(x, offs, wgu, wd, y_perm=y, gu_q=q, gu_s=s)
    base.sync()
    assert t.all(y[ROWS:] == base.sentinel((1,), "bf16")) and t.all(q[ROWS:] == 77) and t.all(s[ROWS:] == -3.0)
    xs = x[:ROWS].double()
    want = t.zeros((ROWS, d), dtype=t.float64, device="cuda")
    assert t.all(q[:ROWS, :I] == 127)
    assert t.all((s[:ROWS, 0].double() * 127 / 64 - 1).abs() <= 2.0 ** -22)
    for c in pieces(I):
        u = xs @ wgu[0][:, I:][:, c].double()
        assert u.abs().max() < 256        # (bf16 holds 64 u)
        blocks = u.unflatten(1, (-1, 64))
        amax = blocks.abs().amax(-1)
        sc = s[:ROWS, 1, c.start // 64:c.stop // 64].double()
        live = amax > 0
        assert t.all((sc * 127 / amax - 1).abs()[live] <= 2.0 ** -22)
        # (three roundings and the reciprocal of a quotient up to 127: below 2^-14)
        off = (q[:ROWS, I:][:, c].double().unflatten(1, (-1, 64)) - blocks / sc[..., None]).abs()
        assert t.all(off[live] <= 0.5 + 2.0 ** -14)
        want += 64.0 * u @ wd[0][c].double()
    same(y[:ROWS], want, "y")


@pytest.mark.parametrize("again", [False, True])
@pytest.mark.parametrize("d,I", [(128, WIDEST), (WIDEST, 128)])
def test_backward(tre, d, I, again):
    """again: g | u computed from x and held in 16-bit codes: g stays 64 but for float32's last places, and u is off by
    OFF at most, so du is exact, and dg = dh u and h = 64 u are off by |dh| OFF, 64 OFF and their rounding to bf16."""
    t = base.T()
    OFF, HALF, SUM = 1.01 * 64 / 65534, 2.0 ** -8, 2.0 ** -23
    offs, x, dy, wgu, wd = inputs(d, I)
    R = ROWS + EXTRA
    kw, u = {}, None
    if not again:
        g = t.Generator(device="cuda")
        g.manual_seed(7)
        u = ints((R, I), 2, 0.7, g).to(t.int8)
        s = t.ones((R, 2, I // 64), device="cuda")
        s[ROWS:] = float("nan")
        kw = dict(gu_q=t.cat([t.full((R, I), 64, dtype=t.int8, device="cuda"), u], 1), gu_s=s)
    dx, dwgu, dwd = (base.sentinel(n, "bf16") for n in ((R, d), (1, d, 2 * I), (1, I, d)))
    tre.moe_grouped_ffn_backward(x, offs, wgu, wd, dy, dx_perm=dx, dw_gate_up=dwgu, dw_down=dwd, **kw)
    base.sync()
    assert t.all(dx[ROWS:] == base.sentinel((1,), "bf16"))
    xs, dys = x[:ROWS].double(), dy[:ROWS].double()
    want_x = t.zeros((ROWS, d), dtype=t.float64, device="cuda")
    err_x = t.zeros((ROWS,), dtype=t.float64, device="cuda")

    def near(got, want, err, terms, size, name):
        err = err + terms * SUM * (size + err)
        assert t.all((got.double() - want).abs() <= err + HALF * (want.abs() + err)), name

    for c in pieces(I):
        wu = wgu[0][:, I:][:, c].double()
        v = xs @ wu if again else u[:ROWS, c].double()
        dh = dys @ wd[0][c].double().t()
        assert dh.abs().max() < 64 and v.abs().max() <= 64
        dg, du, h = dh * v, 64 * dh, 64 * v
        want_x += du @ wu.t()
        want_x[:, 0] += 64 * dg.sum(1)
        same(dwgu[0][:, I:][:, c], xs.t() @ du, "up's gradient")
        gate, down = xs.t() @ dg, h.t() @ dys
        if not again:
            same(dwgu[0][:, :I][:, c], gate, "gate's gradient")
            same(dwd[0][c], down, "down's gradient")
            continue
        edg = OFF * dh.abs() + HALF * (dg.abs() + OFF * dh.abs())
        eh = 64 * OFF + HALF * (h.abs() + 64 * OFF)
        near(dwgu[0][:, :I][:, c], gate, xs.abs().t() @ edg, ROWS, xs.abs().t() @ dg.abs(), "gate's gradient")
        near(dwd[0][c], down, eh.t() @ dys.abs(), ROWS, h.abs().t() @ dys.abs(), "down's gradient")
        err_x += 64 * edg.sum(1) + 2 * I * SUM * (64 * dg.abs().sum(1) + du.abs() @ wu[0].abs())
    if not again:
        same(dx[:ROWS], want_x, "dx")
        return
    same(dx[:ROWS, 1:], want_x[:, 1:], "dx")
    near(dx[:ROWS, 0], want_x[:, 0], err_x, 0, 0.0, "dx's first column")
