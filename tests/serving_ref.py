"""Plain 64-bit forms of the serving operators, on the CPU: e4m3 blocks, the
products on them and the layer, each with the bound of its float32 error.

Bounds are first order in the float32 step.  `SUM` is one addition's relative
error, a whole step (2^-23) so that additions that truncate are covered too;
roundings to a type are half a step of it."""
import numpy as np

SUM = 2.0 ** -23
HALF_BF16 = 2.0 ** -8
HALF_F32 = 2.0 ** -24
BLOCK = 128

E4M3 = np.array([(-1.0 if c & 128 else 1.0) * (np.nan if c & 127 == 127 else (c & 7) * 2.0 ** -9 if c & 120 == 0
                 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3 & 15) - 7)) for c in range(256)])


def blocks(n):
    return -(-n // BLOCK)


def round_e4m3(v):
    """Nearest e4m3 value of |v| <= 448, ties to even."""
    v = np.asarray(v, dtype=np.float64)
    _, e = np.frexp(np.abs(v))
    step = np.exp2(np.maximum(e - 4, -9).astype(np.float64))
    return np.round(v / step) * step


def power_scale(amax):
    """Smallest 2^n >= amax / 448, n >= -126, by trial; NaN where amax is not finite."""
    amax = np.asarray(amax, dtype=np.float64)
    out = np.full(amax.shape, np.nan)
    n = np.full(amax.shape, -126)
    for p in range(-126, 128):
        n = np.where(448.0 * 2.0 ** p < amax, p + 1, n)
    ok = np.isfinite(amax)
    out[ok] = np.exp2(n[ok].astype(np.float64))
    return out


def spread(s, n, axis):
    return np.repeat(s, BLOCK, axis=axis).take(np.arange(n), axis=axis)


def quantize_rows(x):
    """(codes' values, scales) of float64 rows."""
    rows, cols = x.shape
    pad = np.zeros((rows, blocks(cols) * BLOCK))
    pad[:, :cols] = x
    amax = np.abs(pad.reshape(rows, -1, BLOCK)).max(-1)
    s = power_scale(amax)
    with np.errstate(invalid="ignore"):
        q = np.where(np.isnan(spread(s, cols, 1)), np.nan, round_e4m3(x / spread(s, cols, 1)))
    return q, s


def quantize_matrix(w):
    """(codes' values, scales) of a float64 [N, K] matrix in blocks of 128 x 128."""
    n, k = w.shape
    pad = np.zeros((blocks(n) * BLOCK, blocks(k) * BLOCK))
    pad[:n, :k] = w
    amax = np.abs(pad.reshape(blocks(n), BLOCK, -1, BLOCK)).max((1, 3))
    s = power_scale(amax)
    full = spread(spread(s, n, 0), k, 1)
    with np.errstate(invalid="ignore"):
        return np.where(np.isnan(full), np.nan, round_e4m3(w / full)), s


def codes(q):
    """Values of a float8_e4m3fn torch tensor (by its bytes) as float64 numpy."""
    import torch
    return E4M3[q.cpu().view(torch.uint8).numpy()]


def row_values(q, s):
    return codes(q) * spread(s.cpu().numpy().astype(np.float64), q.shape[1], 1)


def weight_values(q, s):
    """[E, N, K] float64 of 8-bit weights (scales [E, NB, KB], or [E, 2, NB, KB] for packed halves)."""
    v, s = codes(q), s.cpu().numpy().astype(np.float64)
    if s.ndim == 3:
        s = s[:, None]
    halves, n = s.shape[1], v.shape[1] // s.shape[1]
    full = np.concatenate([spread(spread(s[:, h], n, 1), v.shape[2], 2) for h in range(halves)], 1)
    return v * full


def product(x, w, per_block, codes8=False):
    """x [R, K] @ w [K, N] and the bound of its float32 error: K additions, and `per_block` roundings for each
    block's scale and its addition.

    codes8: both operands are 8-bit codes in an 8-bit matrix instruction.  It adds the products of 8 consecutive k
    after aligning them to the largest one's exponent, and keeps 13 binary places behind that: with 2^16 in place 0
    of a group, a product 2^3 in any other place of the group is added and 2^2 is not, while the next group's 2^-7
    still is.  The largest product itself (8 significant bits) loses nothing, so a group loses less than
    7 * 2^-13 of its largest product, which is at most the product of the two operands' largest values in it."""
    k = x.shape[1]
    bound = (k + per_block * blocks(k)) * SUM * (np.abs(x) @ np.abs(w))
    if codes8:
        top = np.abs(x).reshape(x.shape[0], k // 8, 8).max(2) @ np.abs(w).reshape(k // 8, 8, -1).max(1)
        bound += 7 * 2.0 ** -13 * top
    return x @ w, bound


def swiglu(gu, err):
    """silu(g) * u of packed [R, 2I] and its bound: |silu'| <= 1.1, |silu(g)| <= |g|; exp, divide, add and multiply
    in float32 (8 half steps cover them)."""
    i = gu.shape[1] // 2
    g, u, eg, eu = gu[:, :i], gu[:, i:], err[:, :i], err[:, i:]
    with np.errstate(over="ignore"):
        silu = g / (1.0 + np.exp(-g))
    return silu * u, 1.1 * eg * (np.abs(u) + eu) + np.abs(silu) * eu + 8 * HALF_F32 * np.abs(silu * u) + 1e-37


def layer(x, idx, w, wgu, wd, half_h, half_out, per_block=0):
    """The layer on given pairs in float64 (wgu [E, d, 2I], wd [E, I, d]) and the bound of a float32 evaluation that
    rounds h by half_h and the output by half_out (relative half steps)."""
    T, k = idx.shape
    out, err = np.zeros((T, wd.shape[2])), np.zeros((T, wd.shape[2]))
    size = np.zeros_like(out)
    for e in range(wgu.shape[0]):
        t, j = np.nonzero(idx == e)
        if not len(t):
            continue
        gu, egu = product(x[t], wgu[e], per_block)
        h, eh = swiglu(gu, egu)
        eh = eh + half_h * (np.abs(h) + eh)
        y, ey = product(h, wd[e], per_block + 16)   # + the shares of a split sum
        ey = ey + eh @ np.abs(wd[e])
        wt = w[t, j][:, None]
        np.add.at(out, t, wt * y)
        np.add.at(err, t, np.abs(wt) * ey)
        np.add.at(size, t, np.abs(wt * y))
    err = err + (k + 1) * SUM * size
    return out, err + half_out * (np.abs(out) + err) + 1e-37
