"""The training operators on the GPU against their plain 64-bit forms
(training_ref): gradients bit for bit where every sum is exact, and within
bounds that count the roundings of the formulas elsewhere.  Outputs start as a
sentinel, so that what a call leaves unwritten, or should have left, shows."""
import numpy as np
import pytest

import training_ref as ref
import workloads
from helpers import as_f64, to_device, to_host

pytestmark = pytest.mark.gpu

# rows of each expert, by the tiles that they lead to (bf16)
COUNTS = {
    "64-row tiles": [5, 0, 64, 1, 70],
    "128-row tiles": [100, 129, 0],
    "tall tiles": [256, 288, 0, 257],
    "tall and not": [320, 33, 511, 289],
    "256-row tiles": [800, 545],
    "many experts": [(7 * e) % 4 for e in range(130)],
    "one row": [0, 1],
    "one expert": [77],
}
WIDTHS = [(64, 64), (128, 192), (320, 576), (192, 1024)]


@pytest.fixture(scope="module")
def tre():
    import torch
    assert torch.cuda.is_available(), "the GPU tests need an MI355X"
    import token_routing_expert_amd as m
    m.load()
    return m


def T():
    import torch
    return torch


def sync():
    T().cuda.synchronize()


def torch_type(dtype):
    return T().float32 if dtype == "f32" else T().bfloat16


def put(a, dtype):
    """float64 -> a GPU tensor of dtype."""
    a = np.asarray(a, dtype=np.float32)
    return to_device(a if dtype == "f32" else workloads.bf16_bits(a))


def rand(shape, dtype, seed, std=1.0):
    """(GPU tensor, its float64 values)."""
    a = (np.random.default_rng(seed).standard_normal(shape) * std).astype(np.float32)
    a = a if dtype == "f32" else workloads.bf16_bits(a)
    return to_device(a), as_f64(a)


def rounded(v, dtype):
    """float64 values, exact in float32, as dtype rounds them."""
    f = v.astype(np.float32)
    assert np.array_equal(f.astype(np.float64), v)
    return as_f64(f if dtype == "f32" else workloads.bf16_bits(f))


def host(t):
    return as_f64(to_host(t))


def offsets(counts):
    return to_device(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))


def spans(counts):
    ends = np.cumsum(counts)
    return [(e, ends[e] - n, ends[e]) for e, n in enumerate(counts) if n]


def sentinel(shape, dtype):
    return T().full(shape, -7777.0, dtype=torch_type(dtype), device="cuda")


def sparse_ints(shape, density, seed, top=1):
    rng = np.random.default_rng(seed)
    a = rng.integers(-top, top + 1, shape).astype(np.float64)
    return a * (rng.random(shape) < density)


# ---- gradients, exactly ------------------------------------------------------------------
#
# g = 64 everywhere: sigmoid(64) is 1 in float32, so h = 64 u, dg = dh u and du =
# 64 dh.  u, dy and the weights are small whole numbers, so every product and
# sum is a whole number that float32 (and, before a product, bf16) holds.

def exact_inputs(rows, E, d, I, seed):
    p = min(1.0, (3.0 / d) ** 0.5)       # dh: sums of d products, a few of them not zero
    x = sparse_ints((rows, d), 0.5, seed, 2)
    dy = sparse_ints((rows, d), p, seed + 1)
    wgu = sparse_ints((E, d, 2 * I), 0.5, seed + 2)
    wd = sparse_ints((E, I, d), p, seed + 3)
    u = sparse_ints((rows, I), 0.7, seed + 4, 2)
    return x, dy, wgu, wd, u


def exact_checkpoint(u):
    q = np.concatenate([np.full_like(u, 64.0), u], 1).astype(np.int8)
    return to_device(q), T().ones((u.shape[0], 2, u.shape[1] // 64), dtype=T().float32, device="cuda")


def exact_gradients(x, dy, w, wgu, wd, u):
    """dx, dwgu, dwd, <dh, h> of one expert's rows."""
    dh = dy @ wd.T
    assert np.abs(dh).max(initial=0) < 64      # (bf16 holds dh u and 64 dh)
    dgu = np.concatenate([dh * u, 64 * dh], 1) * w[:, None]
    return dgu @ wgu.T, x.T @ dgu, (64 * u * w[:, None]).T @ dy, (64 * u * dh).sum(1)


@pytest.mark.parametrize("d,I", WIDTHS)
@pytest.mark.parametrize("case", list(COUNTS))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_grouped_backward_exact(tre, case, d, I, dtype):
    counts = COUNTS[case]
    E, R = len(counts), sum(counts)
    x, dy, wgu, wd, u = exact_inputs(R, E, d, I, R + d + I)
    q, s = exact_checkpoint(u)
    extra = 3                                   # rows behind the last expert
    pad = np.zeros((extra, d))
    xs, dys = put(np.concatenate([x, pad + 5]), dtype), put(np.concatenate([dy, pad + 5]), dtype)
    q = T().cat([q, T().full((extra, 2 * I), 9, dtype=T().int8, device="cuda")])
    s = T().cat([s, T().full((extra, 2, I // 64), float("nan"), device="cuda")])
    dx, dwgu, dwd = sentinel((R + extra, d), dtype), sentinel((E, d, 2 * I), dtype), sentinel((E, I, d), dtype)
    tre.moe_grouped_ffn_backward(xs, offsets(counts), put(wgu, dtype), put(wd, dtype), dys, gu_q=q, gu_s=s, dx_perm=dx,
                                 dw_gate_up=dwgu, dw_down=dwd)
    sync()
    want_x, want_gu, want_d = np.zeros((R, d)), np.zeros((E, d, 2 * I)), np.zeros((E, I, d))
    for e, lo, hi in spans(counts):
        want_x[lo:hi], want_gu[e], want_d[e], _ = exact_gradients(x[lo:hi], dy[lo:hi], np.ones(hi - lo), wgu[e], wd[e],
                                                                  u[lo:hi])
    assert np.array_equal(host(dx[:R]), rounded(want_x, dtype))
    assert np.array_equal(host(dwgu), rounded(want_gu, dtype))
    assert np.array_equal(host(dwd), rounded(want_d, dtype))
    assert T().all(dx[R:] == -7777.0) or dtype == "bf16" and T().all(dx[R:] == T().tensor(-7777.0).bfloat16().item())


def route_given(T_, E, k, seed, drop=0.1, twice=False):
    """Given pairs: k experts a token (twice: an expert may come again), some dropped; weights that are powers of two."""
    rng = np.random.default_rng(seed)
    idx = (rng.integers(0, E, (T_, k)) if twice or k > E
           else np.argsort(rng.random((T_, E)), 1)[:, :k]).astype(np.int32)
    idx[rng.random((T_, k)) < drop] = -1
    return idx, np.exp2(rng.integers(-2, 2, (T_, k))).astype(np.float32)


def grouping(tre, x, idx, E):
    _, tok, row, offs = tre.moe_permute(x, to_device(idx), idx.shape[1], E, move_rows=False)
    return offs, tok, row


def group_numpy(idx, E):
    """(tokens, pairs) of each expert's rows, in grouped order."""
    flat = idx.reshape(-1)
    return [np.nonzero(flat == e)[0] for e in range(E)]


@pytest.mark.parametrize("T_,d,E,k,I,twice", [
    (1, 64, 2, 1, 64, False), (37, 128, 5, 2, 192, False), (300, 320, 3, 3, 576, False), (700, 192, 4, 2, 1024, False),
    (450, 128, 3, 2, 320, True), (97, 64, 4, 9, 128, True), (64, 192, 200, 4, 64, False), (30, 64, 3, 5, 64, True)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_backward_exact(tre, T_, d, E, k, I, twice, dtype):
    idx, w = route_given(T_, E, k, T_ + k, twice=twice)
    x, dout, wgu, wd, _ = exact_inputs(T_, E, d, I, T_ + d)
    u = sparse_ints((T_ * k, I), 0.7, T_, 2)
    xs = put(x, dtype)
    kept = tre.Checkpoint(*grouping(tre, xs, idx, E), *exact_checkpoint(u))
    dx, dwgu, dwd = sentinel((T_, d), dtype), sentinel((E, d, 2 * I), dtype), sentinel((E, I, d), dtype)
    r = tre.moe_backward_q8(xs, put(wgu, dtype), put(wd, dtype), k, put(dout, dtype), to_device(idx), to_device(w),
                            kept, dx=dx, dw_gate_up=dwgu, dw_down=dwd)
    sync()
    assert set(r) == {"dx", "dw_gate_up", "dw_down", "dtopk_w"} and r["dx"] is dx
    want_x, want_w = np.zeros((T_, d)), np.zeros(T_ * k)
    at = 0
    for e, pairs in enumerate(group_numpy(idx, E)):
        t, n = pairs // k, len(pairs)
        rx, gu, dn, dot = exact_gradients(x[t], dout[t], w.reshape(-1)[pairs].astype(np.float64), wgu[e], wd[e],
                                          u[at:at + n])
        np.add.at(want_x, t, rx)
        want_w[pairs] = dot
        assert np.array_equal(host(dwgu[e]), rounded(gu, dtype)), e
        assert np.array_equal(host(dwd[e]), rounded(dn, dtype)), e
        at += n
    assert np.array_equal(host(dx), rounded(want_x, dtype))
    assert np.array_equal(host(r["dtopk_w"]).reshape(-1), want_w)


# ---- the forward and its checkpoint ---------------------------------------------------------

@pytest.mark.parametrize("d,I", WIDTHS)
@pytest.mark.parametrize("case", list(COUNTS))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_grouped_train(tre, case, d, I, dtype):
    counts = COUNTS[case]
    E, R = len(counts), sum(counts)
    x, vx = rand((R + 3, d), dtype, R + d)
    wgu, vgu = rand((E, d, 2 * I), dtype, d, std=d ** -0.5)
    wd, vd = rand((E, I, d), dtype, I, std=I ** -0.5)
    y = sentinel((R + 3, d), dtype)
    q = T().full((R + 3, 2 * I), 77, dtype=T().int8, device="cuda")
    s = T().full((R + 3, 2, I // 64), -3.0, device="cuda")
    out = tre.moe_grouped_ffn_train(x, offsets(counts), wgu, wd, y_perm=y, gu_q=q, gu_s=s)
    sync()
    assert out[0] is y and out[1] is q and out[2] is s
    for e, lo, hi in spans(counts):
        gu, egu, vy, ey = ref.forward(vx[lo:hi], vgu[e], vd[e], dtype)
        ref.near(host(y[lo:hi]), vy, ey, dtype, f"y of expert {e}")
        ref.check_codes(q[lo:hi].cpu().numpy(), s[lo:hi].cpu().numpy(), gu, egu)
    assert T().all(q[R:] == 77) and T().all(s[R:] == -3.0) and T().all(y[R:] == sentinel((1,), dtype))


@pytest.mark.parametrize("rows,I", [(1, 64), (5, 192), (77, 2880)])
def test_checkpoint_values(tre, rows, I):
    rng = np.random.default_rng(I)
    q = rng.integers(-127, 128, (rows, 2 * I)).astype(np.int8)
    s = np.exp(3 * rng.standard_normal((rows, 2, I // 64))).astype(np.float32)
    s[0, 0, 0] = np.nan
    want = np.float32(ref.values(q, s))           # one rounding: the product is exact in 64 bits
    for dtype in ("f32", "bf16"):
        got = tre.moe_checkpoint_values(to_device(q), to_device(s), torch_type(dtype))
        sync()
        exact = want if dtype == "f32" else as_f64(workloads.bf16_bits(want))
        live = ~np.isnan(want)
        assert np.array_equal(host(got)[live], exact[live].astype(np.float64)) and np.all(np.isnan(host(got)[~live]))


def kept_gates(rows, I, seed):
    """A checkpoint of gates and ups of many sizes: (q, s, values)."""
    rng = np.random.default_rng(seed)
    v = rng.standard_normal((rows, 2 * I)) * np.exp(rng.standard_normal((rows, 1)))
    s = ref.scales(v).astype(np.float32)
    q = np.round(v / np.repeat(s.astype(np.float64), 64, 1)).astype(np.int8)
    return to_device(q), to_device(s.reshape(rows, 2, -1)), ref.values(q, s)


@pytest.mark.parametrize("again", [False, True])
@pytest.mark.parametrize("d,I", [(128, 192), (320, 576)])
@pytest.mark.parametrize("case", list(COUNTS))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_grouped_backward(tre, case, d, I, dtype, again):
    """Gates of both signs and many sizes; again: g | u computed from x."""
    counts = COUNTS[case]
    E, R = len(counts), sum(counts)
    x, vx = rand((R, d), dtype, R + d)
    dy, vdy = rand((R, d), dtype, R + I, std=1e-3)
    wgu, vgu = rand((E, d, 2 * I), dtype, d, std=d ** -0.5)
    wd, vd = rand((E, I, d), dtype, I, std=I ** -0.5)
    kw = {}
    if not again:
        q, s, v = kept_gates(R, I, R)
        kw = dict(gu_q=q, gu_s=s)
    dx, dwgu, dwd = tre.moe_grouped_ffn_backward(x, offsets(counts), wgu, wd, dy, **kw)
    sync()
    for e in range(E):
        if counts[e] == 0:
            assert not T().any(dwgu[e]) and not T().any(dwd[e])
    for e, lo, hi in spans(counts):
        if again:
            gu, egu = ref.product(vx[lo:hi], np.zeros((hi - lo, d)), vgu[e])
            if dtype == "bf16":   # 16-bit codes in between: half a step of amax / 32767, and their float32
                amax = np.abs(gu + egu).reshape(hi - lo, -1, 64).max(-1)
                egu = egu + np.repeat(amax, 64, 1) * (0.5 / 32767 + 4 * ref.SUM)
        else:
            gu, egu = v[lo:hi], np.zeros((hi - lo, 2 * I))
        a, b, c, _ = ref.backward(vx[lo:hi], vdy[lo:hi], np.ones(hi - lo), gu[:, :I], gu[:, I:], vgu[e], vd[e], dtype,
                                  egu[:, :I], egu[:, I:])
        ref.near(host(dx[lo:hi]), *a, dtype, f"dx of expert {e}")
        ref.near(host(dwgu[e]), *b, dtype, f"dw_gate_up of expert {e}")
        ref.near(host(dwd[e]), *c, dtype, f"dw_down of expert {e}")


@pytest.mark.parametrize("T_,d,E,k,I", [(1, 64, 3, 2, 128), (50, 128, 8, 2, 256), (400, 192, 3, 2, 320),
                                        (333, 128, 2, 1, 192), (90, 64, 150, 4, 64), (600, 128, 5, 3, 1024)])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_step(tre, T_, d, E, k, I, given, dtype):
    """A training step as it is used: route, forward, keep, backward; against the 64-bit forms at the kept values."""
    x, vx = rand((T_, d), dtype, T_)
    wgu, vgu = rand((E, d, 2 * I), dtype, d, std=d ** -0.5)
    wd, vd = rand((E, I, d), dtype, I, std=I ** -0.5)
    dout, vdo = rand((T_, d), dtype, T_ + 1, std=1e-3)
    logits = None
    if given:
        idx, w = route_given(T_, E, k, T_, twice=T_ == 400)
        ti, tw = to_device(idx), to_device(w)
    else:
        logits = to_device(np.random.default_rng(T_).standard_normal((T_, E)).astype(np.float32))
        ti = tw = None
    out, ti, tw, kept = tre.moe_forward_train_q8(x, wgu, wd, k, logits=logits, topk_idx=ti, topk_w=tw)
    r = tre.moe_backward_q8(x, wgu, wd, k, dout, ti, tw, kept, want_dlogits=not given)
    sync()
    if not given:
        ri, rw = tre.moe_route_topk(logits, k)
        assert T().equal(ri, ti) and T().equal(rw, tw)
    idx, w = ti.cpu().numpy(), tw.cpu().numpy().astype(np.float64)
    q, s = kept.gu_q.cpu().numpy(), kept.gu_s.cpu().numpy()
    row = kept.pair_row.cpu().numpy()
    vo, eo = np.zeros((T_, d)), np.zeros((T_, d))
    wx, ex, size = np.zeros((T_, d)), np.zeros((T_, d)), np.zeros((T_, d))
    dw, edw = np.zeros(T_ * k), np.zeros(T_ * k)
    at = 0
    for e, pairs in enumerate(group_numpy(idx, E)):
        t, n = pairs // k, len(pairs)
        assert np.array_equal(row[pairs], np.arange(at, at + n))
        assert np.array_equal(kept.row_token[at:at + n].cpu().numpy(), t)
        if n == 0:
            assert not T().any(r["dw_gate_up"][e]) and not T().any(r["dw_down"][e])
            continue
        wp = w.reshape(-1)[pairs]
        gu, egu, vy, ey = ref.forward(vx[t], vgu[e], vd[e], dtype)
        ref.check_codes(q[at:at + n], s[at:at + n], gu, egu)
        np.add.at(vo, t, wp[:, None] * vy)
        np.add.at(eo, t, wp[:, None] * (ey + (k + 10) * ref.SUM * np.abs(vy)))
        v = ref.values(q[at:at + n], s[at:at + n])
        a, b, c, dot = ref.backward(vx[t], vdo[t], wp, v[:, :I], v[:, I:], vgu[e], vd[e], dtype)
        np.add.at(wx, t, a[0])
        np.add.at(ex, t, a[1])
        np.add.at(size, t, np.abs(a[0]))
        dw[pairs], edw[pairs] = dot
        ref.near(host(r["dw_gate_up"][e]), *b, dtype, f"dw_gate_up of expert {e}")
        ref.near(host(r["dw_down"][e]), *c, dtype, f"dw_down of expert {e}")
        at += n
    assert np.array_equal(kept.expert_offsets.cpu().numpy()[-1], at)
    assert np.all(row[idx.reshape(-1) < 0] == -1)
    ref.near(host(out), vo, eo, dtype, "out")
    ref.near(host(r["dx"]), wx, ex + (k + 10) * ref.SUM * size, dtype, "dx")
    ref.near(host(r["dtopk_w"]).reshape(-1), dw, edw, "f32", "dtopk_w")
    if not given:
        dw, edw = dw.reshape(T_, k), edw.reshape(T_, k)
        inner, einner = (w * dw).sum(1, keepdims=True), (w * edw + (k + 2) * ref.SUM * np.abs(w * dw)).sum(1, keepdims=True)
        want, err = np.zeros((T_, E)), np.zeros((T_, E))
        np.put_along_axis(want, idx.astype(np.int64), w * (dw - inner), 1)
        np.put_along_axis(err, idx.astype(np.int64), w * (edw + einner + 2 * ref.SUM * (np.abs(dw) + np.abs(inner))), 1)
        ref.near(host(r["dlogits"]), want, err, "f32", "dlogits")


def test_dlogits_of_an_expert_named_twice(tre):
    """dlogits sums the pairs of one expert, as the formula's softmax over the pairs gives."""
    T_, d, E, k, I = 6, 64, 4, 3, 64
    idx = np.array([[1, 1, 2], [0, 3, 0], [2, 2, 2], [-1, 1, 1], [3, -1, 0], [-1, -1, -1]], dtype=np.int32)
    x, dout, wgu, wd, _ = exact_inputs(T_, E, d, I, 3)
    u = sparse_ints((T_ * k, I), 0.7, 4, 2)
    w = np.full((T_, k), 0.25, dtype=np.float32)
    xs = put(x, "f32")
    kept = tre.Checkpoint(*grouping(tre, xs, idx, E), *exact_checkpoint(u))
    r = tre.moe_backward_q8(xs, put(wgu, "f32"), put(wd, "f32"), k, put(dout, "f32"), to_device(idx), to_device(w), kept,
                            want_dlogits=True)
    sync()
    dw = host(r["dtopk_w"])
    assert np.all(dw[idx < 0] == 0)
    want = np.zeros((T_, E))
    for t in range(T_):
        for j in range(k):
            if idx[t, j] >= 0:
                want[t, idx[t, j]] += 0.25 * (dw[t, j] - 0.25 * dw[t].sum())
    assert np.array_equal(host(r["dlogits"]), want)


# ---- values that are not finite, huge or tiny ---------------------------------------------------

@pytest.mark.parametrize("case", ["64-row tiles", "128-row tiles", "tall tiles", "256-row tiles"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_checkpoint_of_extreme_rows(tre, case, dtype):
    """Zeros, values below the floor, near the largest float32, infinity and NaN: each shows in its own blocks only."""
    counts, d, I = COUNTS[case], 128, 192
    E, R = len(counts), sum(counts)
    rng = np.random.default_rng(3)
    x = np.zeros((R, d))
    x[:, 0] = 1.0                       # rows pick the first row of the weights, times their size
    sizes = {0: 0.0, 1: 2.0 ** -110, 2: 2.0 ** 100, 3: 2.0 ** -60, 4: np.inf, 6: np.nan}
    for r, v in sizes.items():
        if r < R:
            x[r, 0] = v
    wgu = np.zeros((E, d, 2 * I))
    wgu[:, 0] = rng.standard_normal((E, 2 * I))
    wgu[:, 0, 7] = 0.0                  # 0 * inf: NaN beside infinities
    vgu = as_f64(to_host(put(wgu, dtype)))
    y, q, s = tre.moe_grouped_ffn_train(put(x, dtype), offsets(counts), put(wgu, dtype),
                                        put(rng.standard_normal((E, I, d)) * 0.1, dtype))
    sync()
    q, s = q.cpu().numpy(), s.cpu().numpy()
    for e, lo, hi in spans(counts):
        for r in range(lo, hi):
            if r in (4, 6):
                assert np.all(np.isnan(s[r])), r
                assert np.all(np.isnan(host(tre.moe_checkpoint_values(to_device(q[r:r + 1]), to_device(s[r:r + 1]),
                                                                      T().float32))))
                continue
            v = x[r, 0] * vgu[e, 0][None]
            ref.check_codes(q[r:r + 1], s[r:r + 1], v, np.abs(v) * ref.SUM)
    if R > 1:
        assert np.all(q[0] == 0) and np.all(q[1] == 0) and np.all(np.abs(s[0] * 127 / 2.0 ** -100 - 1) < 1e-6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_of_extreme_gates(tre, dtype):
    """Gates up to +-2^100: the gradients of the formula, where it is finite."""
    counts, d, I = [40, 90], 64, 64
    R = sum(counts)
    top = np.array([0.0, 2.0 ** -100, 1e-20, 1.0, 30.0, 90.0, 104.0, 1e4, 1e20, 2.0 ** 100])
    sizes = np.tile(top, R)[:R]
    codes = np.random.default_rng(1).integers(-127, 128, (R, 2 * I)).astype(np.int8)
    codes[:, 0] = 127
    s = np.ones((R, 2, 1), dtype=np.float32) / 127
    s[:, 0, 0] = (np.maximum(sizes, 2.0 ** -100) / 127).astype(np.float32)
    v = ref.values(codes, s)
    x, vx = rand((R, d), dtype, 1)
    dy, vdy = rand((R, d), dtype, 2, std=2.0 ** -60)
    wgu, vgu = rand((2, d, 2 * I), dtype, 3, std=0.1)
    wd, vd = rand((2, I, d), dtype, 4, std=0.1)
    dx, dwgu, dwd = tre.moe_grouped_ffn_backward(x, offsets(counts), wgu, wd, dy, gu_q=to_device(codes), gu_s=to_device(s))
    sync()
    # each row on its own (a weight gradient would only show the largest gate's)
    for e, lo, hi in spans(counts):
        a, b, c, _ = ref.backward(vx[lo:hi], vdy[lo:hi], np.ones(hi - lo), v[lo:hi, :I], v[lo:hi, I:], vgu[e], vd[e],
                                  dtype)
        ref.near(host(dx[lo:hi]), *a, dtype, f"dx of expert {e}")
        ref.near(host(dwgu[e]), *b, dtype, f"dw_gate_up of expert {e}")
        ref.near(host(dwd[e]), *c, dtype, f"dw_down of expert {e}")


@pytest.mark.parametrize("case", ["64-row tiles", "128-row tiles", "tall tiles", "256-row tiles"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_stays_in_its_row_and_expert(tre, case, dtype):
    counts, d, I = COUNTS[case], 128, 128
    E, R = len(counts), sum(counts)
    q, s, _ = kept_gates(R, I, 2)
    bad = R - 1
    e_bad = max(e for e, n in enumerate(counts) if n)
    s[bad, 1, 1] = float("nan")
    x, _ = rand((R, d), dtype, 1)
    dy, _ = rand((R, d), dtype, 2)
    wgu, _ = rand((E, d, 2 * I), dtype, 3, std=0.1)
    wd, _ = rand((E, I, d), dtype, 4, std=0.1)
    dx, dwgu, dwd = tre.moe_grouped_ffn_backward(x, offsets(counts), wgu, wd, dy, gu_q=q, gu_s=s)
    sync()
    assert np.all(np.isnan(host(dx[bad]))) and np.all(np.isfinite(host(dx[:bad])))
    for e in range(E):
        assert np.all(np.isfinite(host(dwgu[e]))) == (e != e_bad) and np.all(np.isfinite(host(dwd[e]))) == (e != e_bad)
    # down: h of the bad columns only
    assert np.all(np.isfinite(host(dwd[e_bad])[:64])) and np.all(np.isnan(host(dwd[e_bad])[64:]))


# ---- empty batches, arrays out of range ---------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_rows(tre, dtype):
    E, d, I, k = 3, 64, 128, 2
    wgu, wd = rand((E, d, 2 * I), dtype, 1)[0], rand((E, I, d), dtype, 2)[0]
    x = T().empty((0, d), dtype=torch_type(dtype), device="cuda")
    y, q, s = tre.moe_grouped_ffn_train(x, offsets([0, 0, 0]), wgu, wd)
    assert y.shape == (0, d) and q.shape == (0, 2 * I) and s.shape == (0, 2, 2)
    for kw in ({}, dict(gu_q=q, gu_s=s)):
        dx, dwgu, dwd = tre.moe_grouped_ffn_backward(x, offsets([0, 0, 0]), wgu, wd, x, dw_gate_up=sentinel(wgu.shape, dtype),
                                                     dw_down=sentinel(wd.shape, dtype), **kw)
        sync()
        assert dx.shape == (0, d) and not T().any(dwgu) and not T().any(dwd)
    out, ti, tw, kept = tre.moe_forward_train_q8(x, wgu, wd, k, logits=T().empty((0, E), device="cuda"))
    r = tre.moe_backward_q8(x, wgu, wd, k, x, ti, tw, kept, want_dlogits=True)
    sync()
    assert out.shape == (0, d) and r["dlogits"].shape == (0, E) and not T().any(r["dw_gate_up"])
    # rows, but no expert has one; and tokens whose pairs are all another rank's
    x, _ = rand((9, d), dtype, 3)
    dx, dwgu, dwd = tre.moe_grouped_ffn_backward(x, offsets([0, 0, 0]), wgu, wd, x, dx_perm=sentinel((9, d), dtype))
    idx = T().full((9, k), -1, dtype=T().int32, device="cuda")
    out, ti, tw, kept = tre.moe_forward_train_q8(x, wgu, wd, k, topk_idx=idx, topk_w=T().ones((9, k), device="cuda"))
    r = tre.moe_backward_q8(x, wgu, wd, k, x, ti, tw, kept)
    sync()
    assert T().all(dx == sentinel((1,), dtype)) and not T().any(dwgu) and not T().any(dwd)
    assert not T().any(out) and not T().any(r["dx"]) and not T().any(r["dw_down"]) and not T().any(r["dtopk_w"])


@pytest.mark.parametrize("bad", [[0, -5, 300, 20], [-9, 900, 900, 2 ** 31 - 1], [700, 600, 10, 5],
                                 [-2 ** 31, -1, 600, 601], [600, 600, 600, 600]])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_arrays_out_of_range(tre, bad, dtype):
    """Offsets, row indices and tokens outside their arrays give whatever values, inside the outputs."""
    E, d, I, R = 3, 64, 128, 600
    offs = to_device(np.array(bad, dtype=np.int32))
    wgu, wd = rand((E, d, 2 * I), dtype, 1)[0], rand((E, I, d), dtype, 2)[0]
    guard = 4096
    whole = sentinel((R + 2 * guard, d), dtype)
    x, _ = rand((R, d), dtype, 3)
    y, q, s = tre.moe_grouped_ffn_train(x, offs, wgu, wd, y_perm=whole[guard:guard + R])
    tre.moe_grouped_ffn_backward(x, offs, wgu, wd, x, gu_q=q, gu_s=s, dx_perm=whole[guard:guard + R])
    tre.moe_grouped_ffn_backward(x, offs, wgu, wd, x, dx_perm=whole[guard:guard + R])
    # (pairs: two a token)
    rng = np.random.default_rng(1)
    wild = to_device(rng.integers(-2 ** 31, 2 ** 31, R).astype(np.int32))
    near = to_device(rng.integers(-3, R + 3, R).astype(np.int32))
    for tok, row in ((wild, near), (near, wild)):
        kept = tre.Checkpoint(offs, tok, row, q, s)
        tre.moe_backward_q8(x[:R // 2], wgu, wd, 2, x[:R // 2], near.view(-1, 2), T().ones((R // 2, 2), device="cuda"), kept,
                            want_dlogits=True, dx=whole[guard:guard + R // 2])
    sync()
    edge = sentinel((1,), dtype)
    assert T().all(whole[:guard] == edge) and T().all(whole[guard + R:] == edge)


# ---- streams, graphs, workspaces, builds ----------------------------------------------------------

def layer_step(tre, dtype, seed=0, T_=160, d=128, E=4, k=2, I=192):
    """A layer's inputs and a function that runs its training step on given buffers."""
    x, dout = rand((T_, d), dtype, seed)[0], rand((T_, d), dtype, seed + 1)[0]
    wgu, wd = rand((E, d, 2 * I), dtype, seed + 2, std=0.1)[0], rand((E, I, d), dtype, seed + 3, std=0.1)[0]
    logits = to_device(np.random.default_rng(seed).standard_normal((T_, E)).astype(np.float32))
    dt = 0 if dtype == "f32" else 1
    ws = T().empty(max(tre.moe_forward_train_q8_workspace_size(T_, d, E, k, I, dt),
                       tre.moe_backward_q8_workspace_size(T_, d, E, k, I, dt)), dtype=T().uint8, device="cuda")

    def run(workspace=None, stream=None):
        w = ws if workspace is None else workspace
        out, ti, tw, kept = tre.moe_forward_train_q8(x, wgu, wd, k, logits=logits, workspace=w, stream=stream)
        r = tre.moe_backward_q8(x, wgu, wd, k, dout, ti, tw, kept, want_dlogits=True, workspace=w, stream=stream)
        return [out, ti, tw, *kept, *r.values()]
    return run, ws


def grouped_step(tre, dtype, seed=0, counts=(70, 0, 300), d=128, I=192):
    R, E = sum(counts), len(counts)
    x, dy = rand((R, d), dtype, seed)[0], rand((R, d), dtype, seed + 1)[0]
    wgu, wd = rand((E, d, 2 * I), dtype, seed + 2, std=0.1)[0], rand((E, I, d), dtype, seed + 3, std=0.1)[0]
    offs = offsets(counts)
    dt = 0 if dtype == "f32" else 1
    ws = T().empty(max(tre.moe_grouped_ffn_train_workspace_size(R, E, d, I, dt),
                       tre.moe_grouped_ffn_backward_workspace_size(R, E, d, I, dt)), dtype=T().uint8, device="cuda")

    def run(workspace=None, stream=None):
        w = ws if workspace is None else workspace
        y, q, s = tre.moe_grouped_ffn_train(x, offs, wgu, wd, workspace=w, stream=stream)
        g = tre.moe_grouped_ffn_backward(x, offs, wgu, wd, dy, gu_q=q, gu_s=s, workspace=w, stream=stream)
        a = tre.moe_grouped_ffn_backward(x, offs, wgu, wd, dy, workspace=w, stream=stream)
        return [y, q, s, *g, *a]
    return run, ws


STEPS = [("layer", layer_step), ("grouped", grouped_step)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("make", [m for _, m in STEPS], ids=[n for n, _ in STEPS])
def test_graph_replays(tre, make, dtype):
    """Captured, replayed with eager work in between, and two graphs on one workspace: always the eager bits."""
    run, ws = make(tre, dtype)
    want = [t.clone() for t in run()]
    other, _ = make(tre, dtype, seed=50)
    want2 = [t.clone() for t in other(workspace=ws)]
    sync()
    graphs = []
    for f in (run, other):
        side = T().cuda.Stream()
        side.wait_stream(T().cuda.current_stream())
        with T().cuda.stream(side):
            f(workspace=ws)
        T().cuda.current_stream().wait_stream(side)
        g = T().cuda.CUDAGraph()
        with T().cuda.graph(g):
            outs = f(workspace=ws)
        graphs.append((g, outs))
    for i in range(4):
        for (g, outs), w in zip(graphs, (want, want2)):
            for t in outs:
                t.zero_() if i % 2 else None
            g.replay()
            if i == 1:
                other(workspace=None)
            sync()
            for a, b in zip(outs, w):
                assert T().equal(a.view(T().uint8), b.view(T().uint8)), i
        ws.fill_(255 if i % 2 else 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("make", [m for _, m in STEPS], ids=[n for n, _ in STEPS])
def test_two_streams(tre, make, dtype):
    """Two steps at once, each on a stream and a workspace of its own, given as an argument or as the current one."""
    runs = [make(tre, dtype, seed=s) for s in (0, 100)]
    want = [[t.clone() for t in run()] for run, _ in runs]
    sync()
    streams = [T().cuda.Stream(), T().cuda.Stream()]
    for _ in range(3):
        got = []
        for (run, _), st in zip(runs, streams):
            st.wait_stream(T().cuda.current_stream())
            if st is streams[0]:
                got.append(run(stream=st))
            else:
                with T().cuda.stream(st):
                    got.append(run())
        sync()
        for g, w in zip(got, want):
            for a, b in zip(g, w):
                assert T().equal(a.view(T().uint8), b.view(T().uint8))


@pytest.mark.parametrize("case", list(COUNTS))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_device_checked_build_equals_release(tre, case, dtype):
    counts = COUNTS[case]
    run, _ = grouped_step(tre, dtype, counts=counts)
    layer, _ = layer_step(tre, dtype, T_=max(1, sum(counts) // 2), E=max(2, min(len(counts), 8)))
    want = [t.clone() for t in run() + layer()]
    sync()
    release = tre._lib
    try:
        tre._lib = tre.open_library(tre.DEBUG_LIB_PATH)
        got = run() + layer()
        sync()
    finally:
        tre._lib = release
    # (rows of the checkpoint behind the last expert do not exist here: every pair has an expert)
    for a, b in zip(got, want):
        assert T().equal(a.view(T().uint8), b.view(T().uint8))


def test_steps_of_one_size_share_their_buffers(tre):
    """A Checkpoint filled again, outputs and workspaces given: nothing of an earlier step is left."""
    run, _ = layer_step(tre, "bf16")
    T_, d, E, k, I = 160, 128, 4, 2, 192
    steps = []
    for seed in (0, 9):
        x, dout = rand((T_, d), "bf16", seed)[0], rand((T_, d), "bf16", seed + 1)[0]
        logits = to_device(np.random.default_rng(seed).standard_normal((T_, E)).astype(np.float32))
        steps.append((x, dout, logits))
    wgu, wd = rand((E, d, 2 * I), "bf16", 2, std=0.1)[0], rand((E, I, d), "bf16", 3, std=0.1)[0]

    def step(x, dout, logits, kept=None, **g):
        out, ti, tw, kept = tre.moe_forward_train_q8(x, wgu, wd, k, logits=logits, kept=kept)
        return kept, [out, *tre.moe_backward_q8(x, wgu, wd, k, dout, ti, tw, kept, want_dlogits=True, **g).values()]
    want = [[t.clone() for t in step(*s)[1]] for s in steps]
    kept, first = step(*steps[0])
    grads = dict(dx=first[1], dw_gate_up=first[2], dw_down=first[3])
    for i in (1, 0, 1):
        again, got = step(*steps[i], kept=kept, **grads)
        sync()
        assert again is kept and got[1] is grads["dx"]
        for a, b in zip(got, want[i]):
            assert T().equal(a, b)


def test_binding_checks(tre):
    d, I, E, R = 64, 64, 2, 8
    x, _ = rand((R, d), "bf16", 1)
    wgu, wd = rand((E, d, 2 * I), "bf16", 2)[0], rand((E, I, d), "bf16", 3)[0]
    offs = offsets([4, 4])
    y, q, s = tre.moe_grouped_ffn_train(x, offs, wgu, wd)
    back = tre.moe_grouped_ffn_backward
    for bad in (lambda: tre.moe_grouped_ffn_train(x.float(), offs, wgu, wd),
                lambda: tre.moe_grouped_ffn_train(x, offs, wgu[:, :, :-1], wd),
                lambda: tre.moe_grouped_ffn_train(x, offs.long(), wgu, wd),
                lambda: tre.moe_grouped_ffn_train(x.cpu(), offs, wgu, wd),
                lambda: back(x, offs, wgu, wd, x, gu_q=q),
                lambda: back(x, offs, wgu, wd, x, gu_q=q.view(T().uint8), gu_s=s),
                lambda: back(x, offs, wgu, wd, x[:4], gu_q=q, gu_s=s),
                lambda: back(x.t(), offs, wgu, wd, x.t()),
                lambda: back(x, offs, wgu, wd, x, workspace=T().empty(16, dtype=T().uint8, device="cuda")),
                lambda: tre.moe_checkpoint_values(q, s[:, :1], T().float32),
                lambda: tre.moe_forward_train_q8(x, wgu, wd, 2)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        tre.moe_checkpoint_values(q, s, T().float16)
    with pytest.raises(tre.MoeError):
        tre.moe_forward_train_q8(x, wgu, wd, 3, logits=T().zeros((R, E), device="cuda"))
