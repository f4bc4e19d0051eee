"""Plain 64-bit forms of the training operators, on the CPU: the 8-bit
checkpoint, the grouped feed-forward and its gradients, each with the bound of
its float32 error.

Bounds are first order in the float32 step, as in serving_ref: `SUM` is one
addition's relative error (a whole step, so that additions that truncate are
covered), roundings to a type are half a step of it.  Hardware functions: the
exponential of -g is off by 2^-22 + 2 |g| 2^-24 of itself (two steps, and the
rounding of g log2 e), the reciprocal by a step, so sigmoid(g) by at most
(6 + 2 |g|) 2^-23 of itself (sum, reciprocal and exponential)."""
import numpy as np

SUM = 2.0 ** -23
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
BLOCK = 64
FLOOR = 2.0 ** -100
TINY = 1e-37


def scales(v):
    """A checkpoint's scales of float64 rows [R, C] -> [R, C / 64]; NaN where a block is not finite."""
    amax = np.abs(v.reshape(v.shape[0], -1, BLOCK)).max(-1)
    return np.where(np.isfinite(amax), np.maximum(amax, FLOOR) / 127.0, np.nan)


def check_codes(q, s, v, err):
    """Codes q and scales s (numpy) of values that the kernel had within err of v: s is amax / 127 and q the nearest
    whole number of v / s, up to the values' own error and the float32 of the quotient (three roundings and the
    reciprocal: 5 steps)."""
    want, gap = scales(v), err.reshape(v.shape[0], -1, BLOCK).max(-1) / 127.0
    ok = np.isfinite(want)
    s = s.reshape(want.shape).astype(np.float64)
    assert np.array_equal(np.isnan(s), ~ok)
    assert np.all(np.abs(s - want)[ok] <= (gap + 4 * SUM * want)[ok])
    full, good = np.repeat(s, BLOCK, 1), np.repeat(ok, BLOCK, 1)
    off = np.abs(q.astype(np.float64) - v / full)
    assert np.all(np.abs(q.astype(np.int32)[good]) <= 127)
    assert np.all(off[good] <= (0.5 + err / full + 5 * SUM * 127.0)[good]), off[good].max()


def values(q, s):
    """The values that codes and scales stand for (float64)."""
    s = s.reshape(q.shape[0], -1).astype(np.float64)
    return q.astype(np.float64) * np.repeat(s, BLOCK, 1)


def product(a, ea, w, extra=0):
    """a @ w with a off by ea, and the bound of its float32 error (one addition a term, `extra` more)."""
    return a @ w, (a.shape[1] + extra) * SUM * (np.abs(a) @ np.abs(w)) + ea @ np.abs(w)


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def swiglu(g, u, eg, eu):
    """silu(g) u and its bound (|silu'| <= 1.1)."""
    s = sigmoid(g)
    silu = g * s
    es = 1.1 * eg + np.abs(silu) * (7 + 2 * np.abs(g)) * SUM
    return silu * u, es * (np.abs(u) + eu) + np.abs(silu) * eu + SUM * np.abs(silu * u) + TINY


def forward(x, wgu, wd, dtype):
    """(g | u, its bound, y before its last rounding, its bound) of one expert's rows."""
    i = wd.shape[0]
    gu, egu = product(x, np.zeros_like(x), wgu)
    h, eh = swiglu(gu[:, :i], gu[:, i:], egu[:, :i], egu[:, i:])
    eh = eh + HALF[dtype] * (np.abs(h) + eh)
    y, ey = product(h, eh, wd, 16)   # (up to 16 ranges of a split sum)
    return gu, egu, y, ey


def backward(x, dy, w, g, u, wgu, wd, dtype, eg=None, eu=None):
    """Gradients of one expert's rows at the pre-activations g, u (off by eg, eu): values and bounds of (dx, dwgu,
    dwd) before their last rounding, and of <dy, y>; w: the rows' weights, which multiply dy."""
    zero = np.zeros_like(g)
    eg, eu = (zero if eg is None else eg), (zero if eu is None else eu)
    eg, eu = eg + HALF["f32"] * np.abs(g), eu + HALF["f32"] * np.abs(u)     # read from codes in float32
    half, w = HALF[dtype], w[:, None]
    dh, edh = product(dy, np.zeros_like(dy), wd.T)
    s = sigmoid(g)
    es = (6 + 2 * np.abs(g)) * SUM * s + 0.25 * eg
    silu, d = g * s, s + g * s * (1 - s)
    h, eh = swiglu(g, u, eg, eu)
    dot = (h * dh).sum(1)
    edot = (np.abs(h) * edh + eh * (np.abs(dh) + edh) + (h.shape[1] + 16) * SUM * np.abs(h * dh)).sum(1)
    esilu = np.abs(g) * es + s * eg + SUM * np.abs(silu)
    ed = es * (1 + np.abs(silu)) + esilu + 4 * SUM * (s + np.abs(silu)) + 0.5 * eg     # |silu''| <= 0.5
    wdh, ewdh = w * dh, np.abs(w) * edh + SUM * np.abs(w * dh)

    def rounded(v, e):
        return v, e + half * (np.abs(v) + e) + TINY

    dg, edg = rounded(wdh * u * d, np.abs(u * d) * ewdh + np.abs(wdh) * (np.abs(u) * ed + np.abs(d) * eu + eu * ed)
                      + 3 * SUM * np.abs(wdh * u * d))
    du, edu = rounded(wdh * silu, np.abs(silu) * ewdh + np.abs(wdh) * esilu + SUM * np.abs(wdh * silu))
    wh, ewh = rounded(w * h, np.abs(w) * eh + SUM * np.abs(w * h))
    dgu, edgu = np.concatenate([dg, du], 1), np.concatenate([edg, edu], 1)
    dx = product(dgu, edgu, wgu.T, 16)
    n = x.shape[0]
    dwgu = x.T @ dgu, n * SUM * (np.abs(x.T) @ np.abs(dgu)) + np.abs(x.T) @ edgu
    dwd = wh.T @ dy, n * SUM * (np.abs(wh.T) @ np.abs(dy)) + ewh.T @ np.abs(dy)
    return dx, dwgu, dwd, (dot, edot)


def near(got, want, err, dtype, name):
    """Every element within its bound, the last rounding to dtype added."""
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == want.shape, name
    assert np.all(np.isfinite(got)), f"{name}: not finite"
    bound = err + HALF[dtype] * (np.abs(want) + err) + TINY
    off = np.abs(got - want)
    worst = np.unravel_index(np.argmax(off / bound), off.shape) if off.size else None
    assert np.all(off <= bound), f"{name}: {worst}: {got[worst]} for {want[worst]}, bound {bound[worst]}"
    return float((off / bound).max()) if off.size else 0.0
