"""Checks of the training operators bit for bit, with inputs made and sums formed
on the GPU (float64), for calls too large for numpy.

The gates are 64, so that silu(g) = 64 in float32 and h = 64 u, dg = dh u, du = 64
dh, with small whole numbers everywhere else: every product and sum is a whole
number that float32 (and, before a product, bf16) holds."""
import numpy as np
import torch as t

from helpers import to_device

OFF = 1.01 * 64 / 65534      # 16-bit codes of magnitudes up to 64: u is off by that at most
HALF, SUM = 2.0 ** -8, 2.0 ** -23
EXTRA = 2                    # rows behind the last expert, where a check is not told


def gen(seed):
    g = t.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ints(shape, top, density, g, dtype=t.bfloat16):
    """Whole numbers in [-top, top], a share `density` of them drawn, the others zero."""
    v = t.randint(-top, top + 1, shape, generator=g, device="cuda", dtype=t.int8)
    if density < 1:
        v *= t.rand(shape, generator=g, device="cuda") < density
    return v.to(dtype)


def sentinel(shape, dtype):
    return t.full(shape, -7777.0, dtype=dtype, device="cuda")


def untouched(a):
    assert t.all(a == sentinel((1,), a.dtype))


def same(got, want, name):
    """want (float64, exact in float32) rounded to the output's type once."""
    f = want.float()
    assert t.equal(f.double(), want), name
    assert t.equal(got, f.to(got.dtype)), name


def near(got, want, err, terms, size, name):
    """Within err, the float32 sum of `terms` terms of magnitudes `size`, and a rounding to bf16."""
    err = err + terms * SUM * (size + err)
    off = (got.double() - want).abs()
    assert t.all(off <= err + HALF * (want.abs() + err)), f"{name}: {float(off.max())}"


def offsets(counts):
    return to_device(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))


def spans(counts):
    lo = 0
    for e, n in enumerate(counts):
        if n:
            yield e, lo, lo + n
        lo += n


def pieces(rows, n):
    """Columns of n, as many at once as keep a piece of these rows below 2^27 numbers."""
    step = max(64, min(1 << 16, (1 << 27) // max(rows, 1) // 64 * 64))
    return [slice(a, min(a + step, n)) for a in range(0, n, step)]


def weights(E, d, I, g, dtype):
    p = min(1.0, (3.0 / d) ** 0.5)       # dh: sums of d products, a few of them not zero
    wgu = ints((E, d, 2 * I), 1, min(1.0, 128.0 / d), g, dtype)
    wgu[:, :, :I] = 0.0
    wgu[:, 0, :I] = 64.0                 # x's first column is 1: g = 64; only dx's first column sums over the gates
    return wgu, ints((E, I, d), 1, p, g, dtype)


def rows_of(R, d, g, dtype):
    x, dy = ints((R, d), 1, 1.0, g, dtype), ints((R, d), 1, min(1.0, (3.0 / d) ** 0.5), g, dtype)
    x[:, 0] = 1.0
    return x, dy


def checkpoint(R, I, seed):
    """u of whole numbers up to 2 and the checkpoint of 64 | u."""
    u = ints((R, I), 2, 0.7, gen(seed), t.int8)
    q = t.empty((R, 2 * I), dtype=t.int8, device="cuda")
    q[:, :I] = 64
    q[:, I:] = u
    return u, q, t.ones((R, 2, I // 64), device="cuda")


def check_codes(q, s, u, c, I):
    """Codes and scales of the columns c of 64 | u."""
    n = u.shape[0]
    blocks = u.unflatten(1, (-1, 64))
    amax = blocks.abs().amax(-1)
    at = slice(c.start // 64, c.stop // 64)
    assert t.all(q[:, :I][:, c] == 127) and t.all((s[:, 0, at].double() * 127 / 64 - 1).abs() <= 2.0 ** -22)
    sc, live = s[:, 1, at].double(), amax > 0
    assert t.all((sc * 127 / amax - 1).abs()[live] <= 2.0 ** -22)
    # (three roundings and the reciprocal of a quotient up to 127: below 2^-14)
    off = (q[:, I:][:, c].double().reshape(n, -1, 64) - blocks / sc[..., None]).abs()
    assert t.all(off[live] <= 0.5 + 2.0 ** -14)


def forward_rows(xs, wgu, wd, I, q, s):
    """y of one expert's rows (float64), their codes checked."""
    want = t.zeros((xs.shape[0], wd.shape[1]), dtype=t.float64, device="cuda")
    for c in pieces(max(xs.shape), I):
        u = xs @ wgu[:, I:][:, c].double()
        assert u.abs().max() < 256        # (bf16 holds 64 u)
        check_codes(q, s, u, c, I)
        want += 64.0 * u @ wd[c].double()
    return want


def check_forward(tre, counts, d, I, dtype=t.bfloat16, extra=EXTRA):
    E, R = len(counts), sum(counts)
    g = gen(d + I + R)
    wgu, wd = weights(E, d, I, g, dtype)
    x, _ = rows_of(R + extra, d, g, dtype)
    x[R:] = float("nan")
    y = sentinel((R + extra, d), dtype)
    q = t.full((R + extra, 2 * I), 77, dtype=t.int8, device="cuda")
    s = t.full((R + extra, 2, I // 64), -3.0, device="cuda")
    tre.moe_grouped_ffn_train(x, offsets(counts), wgu, wd, y_perm=y, gu_q=q, gu_s=s)
    t.cuda.synchronize()
    untouched(y[R:])
    assert t.all(q[R:] == 77) and t.all(s[R:] == -3.0)
    for e, lo, hi in spans(counts):
        same(y[lo:hi], forward_rows(x[lo:hi].double(), wgu[e], wd[e], I, q[lo:hi], s[lo:hi]), f"y of expert {e}")


def backward_rows(xs, dys, wgu, wd, I, v_of, dwgu, dwd, w, again, name):
    """Checks one expert's weight gradients; returns (dx's rows, the bound of its first column, <dh, h>)."""
    n, d = xs.shape
    want_x = t.zeros((n, d), dtype=t.float64, device="cuda")
    err_x = t.zeros((n,), dtype=t.float64, device="cuda")
    dot = t.zeros((n,), dtype=t.float64, device="cuda")
    for c in pieces(max(n, d), I):
        wu = wgu[:, I:][:, c].double()
        v = xs @ wu if again else v_of[:, c].double()
        dh = dys @ wd[c].double().t()
        assert dh.abs().max() < 64 and v.abs().max() <= 64
        dot += (64 * v * dh).sum(1)
        h = 64 * v
        if w is not None:
            dh, h = dh * w[:, None], h * w[:, None]
        dg, du = dh * v, 64 * dh
        want_x += du @ wu.t()
        want_x[:, 0] += 64 * dg.sum(1)
        same(dwgu[:, I:][:, c], xs.t() @ du, f"up's gradient of {name}")
        gate, down = xs.t() @ dg, h.t() @ dys
        if not again:
            same(dwgu[:, :I][:, c], gate, f"gate's gradient of {name}")
            same(dwd[c], down, f"down's gradient of {name}")
            continue
        edg = OFF * dh.abs() + HALF * (dg.abs() + OFF * dh.abs())
        eh = 64 * OFF + HALF * (h.abs() + 64 * OFF)
        near(dwgu[:, :I][:, c], gate, xs.abs().t() @ edg, n, xs.abs().t() @ dg.abs(), f"gate's gradient of {name}")
        near(dwd[c], down, eh.t() @ dys.abs(), n, h.abs().t() @ dys.abs(), f"down's gradient of {name}")
        err_x += 64 * edg.sum(1) + 2 * I * SUM * (64 * dg.abs().sum(1) + du.abs() @ wu[0].abs())
    return want_x, err_x, dot


def check_backward(tre, counts, d, I, again, dtype=t.bfloat16, extra=EXTRA):
    """again (bf16): g | u computed from x and held in 16-bit codes: g stays 64 but for float32's last places, and u is
    off by OFF at most, so du is exact, and dg = dh u and h = 64 u are off by |dh| OFF, 64 OFF and their rounding."""
    E, R = len(counts), sum(counts)
    g = gen(d + I + R)
    wgu, wd = weights(E, d, I, g, dtype)
    x, dy = rows_of(R + extra, d, g, dtype)
    x[R:], dy[R:] = float("nan"), float("inf")
    u, kw = None, {}
    if not again:
        u, q, s = checkpoint(R + extra, I, 7)
        s[R:] = float("nan")
        kw = dict(gu_q=q, gu_s=s)
    dx, dwgu, dwd = sentinel((R + extra, d), dtype), sentinel((E, d, 2 * I), dtype), sentinel((E, I, d), dtype)
    tre.moe_grouped_ffn_backward(x, offsets(counts), wgu, wd, dy, dx_perm=dx, dw_gate_up=dwgu, dw_down=dwd, **kw)
    t.cuda.synchronize()
    untouched(dx[R:])
    for e, n in enumerate(counts):
        if n == 0:
            assert not t.any(dwgu[e]) and not t.any(dwd[e])
    for e, lo, hi in spans(counts):
        want, err, _ = backward_rows(x[lo:hi].double(), dy[lo:hi].double(), wgu[e], wd[e], I,
                                     None if again else u[lo:hi], dwgu[e], dwd[e], None, again, f"expert {e}")
        if again:
            same(dx[lo:hi, 1:], want[:, 1:], f"dx of expert {e}")
            near(dx[lo:hi, 0], want[:, 0], err, 0, 0.0, f"dx's first column of expert {e}")
        else:
            same(dx[lo:hi], want, f"dx of expert {e}")


def check_layer(tre, idx, d, E, I, dtype=t.bfloat16):
    """A step on given pairs idx [T, k] (some -1), weights powers of two: the forward with its checkpoint, then the
    backward from an exact one."""
    T_, k = idx.shape
    g = gen(d + I + T_)
    wgu, wd = weights(E, d, I, g, dtype)
    x, dout = rows_of(T_, d, g, dtype)
    idx = to_device(idx)
    w = t.exp2(t.randint(-2, 2, (T_, k), generator=g, device="cuda").float())
    out, _, _, kept = tre.moe_forward_train_q8(x, wgu, wd, k, topk_idx=idx, topk_w=w, out=sentinel((T_, d), dtype))
    offs = kept.expert_offsets.tolist()
    counts = [b - a for a, b in zip(offs, offs[1:])]
    u, q, s = checkpoint(T_ * k, I, 9)
    r = tre.moe_backward_q8(x, wgu, wd, k, dout, idx, w, kept._replace(gu_q=q, gu_s=s), dx=sentinel((T_, d), dtype),
                            dw_gate_up=sentinel((E, d, 2 * I), dtype), dw_down=sentinel((E, I, d), dtype))
    t.cuda.synchronize()
    flat = idx.flatten()
    order = t.argsort(t.where(flat >= 0, flat, E), stable=True)[:offs[-1]]
    assert counts == t.bincount(flat[flat >= 0], minlength=E).tolist()
    assert t.equal(kept.row_token[:offs[-1]].long(), order // k) and t.equal(kept.pair_row[order].long(),
                                                                            t.arange(offs[-1], device="cuda"))
    want_o, want_x = (t.zeros((T_, d), dtype=t.float64, device="cuda") for _ in range(2))
    want_w = t.zeros(T_ * k, dtype=t.float64, device="cuda")
    for e, lo, hi in spans(counts):
        tok, wp = order[lo:hi] // k, w.flatten()[order[lo:hi]].double()
        xs = x[tok].double()
        y = forward_rows(xs, wgu[e], wd[e], I, kept.gu_q[lo:hi], kept.gu_s[lo:hi])
        want_o.index_add_(0, tok, y * wp[:, None])
        dx, _, dot = backward_rows(xs, dout[tok].double(), wgu[e], wd[e], I, u[lo:hi], r["dw_gate_up"][e],
                                   r["dw_down"][e], wp, False, f"expert {e}")
        want_x.index_add_(0, tok, dx)
        want_w[order[lo:hi]] = dot
    same(out, want_o, "out")
    same(r["dx"], want_x, "dx")
    assert t.equal(r["dtopk_w"].double().flatten(), want_w)
    return counts
