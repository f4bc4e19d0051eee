"""The serving operators on the GPU at the ends of their ranges: gates whose
SwiGLU factors leave float32 though the product does not, layers whose weights
pass 2^31 bytes, the widest layers and the most experts, the same rows in calls
of different sizes, the steps captured, on side streams and with offsets out of
range, and what the binding takes and refuses."""
import numpy as np
import pytest

import serving_ref as ref
from helpers import to_device
from test_serving_gpu import (T, check_codes, few_call, few_weights, offsets_of, product_tolerance,   # noqa: F401
                              rand, random_codes, random_scales, routed, sync, tre, weights8)   # (tre: the fixture)

pytestmark = pytest.mark.gpu


# (gate, up): below -88.73 the definition's denominator 1 + e^-g passes float32's range and the result is a zero;
# between, and far above, the result is an ordinary number although g * u or 1 / (1 + e^-g) alone is not.
GATES = [(-20.0, 1e38), (-60.0, -3e38), (-86.0, 1e37), (-87.0, 1e38), (-87.4, -1e38), (-88.0, 1e38), (-88.7, 1e38),
         (-88.8, 1.0), (-89.0, 1e38), (-100.0, 1e30), (-150.0, -1.0), (-1e4, 1e38), (-1e20, 1e20), (-3e38, 3e38),
         (-3e38, 1.0), (-1.0, 1e38), (-1e-30, 1e38), (0.0, 1e38), (1e-30, -1e38), (1.0, 3e37), (20.0, 1e37),
         (89.0, 1e36), (1e20, 1e18), (3e38, 1.0), (3e38, 1e-30)]


@pytest.mark.parametrize("rows", [10, 40, 80, 160])   # tiles of 32 and 64 rows (bf16 inside), 128 and 288 (8 bits)
def test_gate_up_extreme_gates(tre, rows):
    """Finite gates and ups whose silu(gate) * up is finite never give NaN codes, and give that product."""
    torch = T()
    E, d, I = 32, 512, 1024                            # 8 column tiles an expert: a tile for every compute unit
    g, u = (np.resize(np.array(v, np.float32), E * rows).astype(np.float64) for v in zip(*GATES))
    # row r's gate comes from its first k and its first scale, its up from the second block of k and that scale
    x = torch.zeros((E * rows, d))
    x[:, 0], x[:, 128] = torch.from_numpy(np.sign(g)), torch.from_numpy(np.sign(u))
    xs = np.ones((E * rows, 4), np.float32)
    xs[:, 0], xs[:, 1] = np.abs(g), np.abs(u)
    w = torch.zeros((E, 2 * I, d))
    w[:, :I, 0] = 1.0
    w[:, I:, 128] = torch.tensor([1.0, 0.5, -1.0, 0.25]).repeat(I // 4)
    f8 = torch.float8_e4m3fn
    hq, hs = tre.moe_gate_up_swiglu_fp8(x.to(f8).cuda(), to_device(xs), offsets_of([rows] * E), w.to(f8).cuda(),
                                        torch.ones((E, 2, I // 128, d // 128), device="cuda"))
    sync()
    ups = u[:, None] * np.resize([1.0, 0.5, -1.0, 0.25], I)
    with np.errstate(over="ignore"):
        silu = (g / (1.0 + np.exp(-g)))[:, None]
    h = silu * ups
    # exponential, its correction, sum, reciprocal and two products: 8 half steps; 1e-37 covers results below
    # float32's normal range; where the denominator passes it, |silu| <= 88.73 e^-88.73 = 2.7e-37 may become zero
    bound = 8 * ref.HALF_F32 * np.abs(h) + 1e-37 + np.where(g < -88.72, 2.7e-37, 0.0)[:, None] * np.abs(ups)
    check_codes(hq, hs, h, bound, f"{rows} rows an expert")


# ---- layers whose weights pass 2^31 bytes -------------------------------------------------------

BIG_E, BIG_D, BIG_I = 3, 16384, 40960     # 1.34e9 gate/up codes an expert, 4.0e9 in all


@pytest.fixture(scope="module")
def big(tre):
    """Codes +-0.5 and +-1 and scales 0.5 and 1: every product is a multiple of 2^-4, and a sum over the widest side
    stays below 2^16, so float32 sums are exact in any order."""
    torch = T()
    g = torch.Generator(device="cuda").manual_seed(1)

    def codes(*shape):
        q = torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=g)
        return q.bitwise_and_(0x88).bitwise_or_(0x30).view(torch.float8_e4m3fn)

    def scales(*shape):
        return torch.randint(1, 3, shape, device="cuda", generator=g).float() * 0.5

    nb, db = ref.blocks(BIG_I), ref.blocks(BIG_D)
    yield codes, scales, (codes(BIG_E, 2 * BIG_I, BIG_D), scales(BIG_E, 2, nb, db), codes(BIG_E, BIG_D, BIG_I),
                          scales(BIG_E, db, nb))
    torch.cuda.empty_cache()


def spread64(q, s, rows=1):
    """What codes [n, k] and scales [n / rows, k / 128] stand for, in 64 bits."""
    s = s.double().repeat_interleave(128, 1)[:, :q.shape[1]].repeat_interleave(rows, 0)[:q.shape[0]]
    return q.float().double() * s


def times(a, q, s, mul=lambda w: w):
    """a [n, K] @ mul(w) of one expert's [N, K] codes, in pieces of whole blocks."""
    return T().cat([a @ mul(spread64(q[n:n + 4096], s[n // 128:n // 128 + 32], 128)).t().contiguous()
                    for n in range(0, q.shape[0], 4096)], 1)


def gate_up64(a, w, e, mul=lambda w: w):
    return T().cat([times(a, w[0][e, i * BIG_I:(i + 1) * BIG_I], w[1][e, i], mul) for i in (0, 1)], 1)


@pytest.mark.parametrize("counts", [[3, 0, 5], [500, 30, 700]], ids=["low_tiles", "high_tiles"])
def test_products_past_two_gib(tre, big, counts):
    torch = T()
    codes, scales, w = big
    R, offs = sum(counts), offsets_of(counts)
    xq, xs = codes(R, BIG_D), scales(R, ref.blocks(BIG_D)) * 0.25
    hq, hs = tre.moe_gate_up_swiglu_fp8(xq, xs, offs, w[0], w[1])
    aq, as_ = codes(R, BIG_I), scales(R, ref.blocks(BIG_I))
    y = tre.moe_down_proj_fp8(aq, as_, offs, w[2], w[3])
    at = 0
    for e, n in enumerate(counts):
        rows = torch.unique(torch.linspace(at, at + n - 1, min(n, 6), device="cuda").long()) if n else []
        at += n
        if not n:
            continue
        exact = times(spread64(aq.view(torch.uint8)[rows].view(aq.dtype), as_[rows]), w[2][e], w[3][e])
        assert torch.equal(y[rows], exact.float().to(torch.bfloat16)), (e, n)
        gu = gate_up64(spread64(xq.view(torch.uint8)[rows].view(xq.dtype), xs[rows]), w, e).cpu().numpy()
        h, eh = ref.swiglu(gu, np.zeros_like(gu))
        check_codes(hq.view(torch.uint8)[rows].view(hq.dtype), hs[rows], h, eh, f"expert {e} of {counts}")
    whole = tre.moe_grouped_ffn_fp8(xq, xs, offs, *w)
    assert torch.equal(whole, tre.moe_down_proj_fp8(hq, hs, offs, w[2], w[3]))


def test_few_tokens_past_two_gib(tre, big):
    torch = T()
    _, _, w = big
    ids, T_, k = np.array([[0, 2], [2, -1], [1, 2]], np.int32), 3, 2
    wts = np.random.default_rng(2).random((T_, k)).astype(np.float32)
    x = torch.randn((T_, BIG_D), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)).mul(0.01)
    x = x.to(torch.bfloat16)
    out, _, _ = tre.moe_forward_few_fp8(x, *w, k, topk_idx=to_device(ids), topk_w=to_device(wts))
    want, err, size = (np.zeros((T_, BIG_D)) for _ in range(3))
    for e in range(BIG_E):
        t, j = np.nonzero(ids == e)
        xe = x[torch.from_numpy(t).cuda()].double()
        # as serving_ref.layer bounds it: a float32 step for each addition and each block's scale, h and the output
        # rounded to bf16
        step = (BIG_D + 3 * ref.blocks(BIG_D)) * ref.SUM
        h, eh = ref.swiglu(gate_up64(xe, w, e).cpu().numpy(), step * gate_up64(xe.abs(), w, e, torch.abs).cpu().numpy())
        eh = eh + ref.HALF_BF16 * (np.abs(h) + eh)
        h, eh = torch.from_numpy(h).cuda(), torch.from_numpy(eh).cuda()
        step = (BIG_I + 19 * ref.blocks(BIG_I)) * ref.SUM
        y = times(h, w[2][e], w[3][e]).cpu().numpy()
        ey = times(step * h.abs() + eh, w[2][e], w[3][e], torch.abs).cpu().numpy()
        wt = wts[t, j].astype(np.float64)[:, None]
        np.add.at(want, t, wt * y)
        np.add.at(err, t, wt * ey)
        np.add.at(size, t, np.abs(wt * y))
    err = err + (k + 1) * ref.SUM * size
    tol = err + ref.HALF_BF16 * (np.abs(want) + err)
    got = out.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)
    # the roundings of h are independent of each other and of the weights' signs, so in the norm they add in
    # quadrature and make at most a half step of y; the output's rounding makes another
    assert np.linalg.norm(got - want) <= 2 * ref.HALF_BF16 * np.linalg.norm(want)


# ---- the same rows in calls of different sizes ----------------------------------------------------

def test_rows_alone_and_among_others(tre):
    """Tiles of other heights sum a block in other arithmetic: what a row gives in a small call and in a large one
    stays within the header's bound of the exact value, so within twice that of each other."""
    torch = T()
    E, d, I, n, more = 16, 576, 2048, 8, 300
    w, wgu, wd = weights8(E, d, I, 210)
    few, many = offsets_of([n] * E), offsets_of([more] * E)
    pick = torch.cat([torch.arange(n) + e * more for e in range(E)]).cuda()
    xq, xs = random_codes((E * more, d), 211), random_scales((E * more, ref.blocks(d)), 212, 0.002, 0.02)
    aq, as_ = random_codes((E * more, I), 213), random_scales((E * more, ref.blocks(I)), 214, 0.01, 0.02)

    def picked(q, s):
        return q.view(torch.uint8)[pick].view(q.dtype), s[pick]

    (xq1, xs1), (aq1, as1) = picked(xq, xs), picked(aq, as_)
    small = tre.moe_gate_up_swiglu_fp8(xq1, xs1, few, w[0], w[1])
    large = picked(*tre.moe_gate_up_swiglu_fp8(xq, xs, many, w[0], w[1]))
    y1 = tre.moe_down_proj_fp8(aq1, as1, few, w[2], w[3])
    y2 = tre.moe_down_proj_fp8(aq, as_, many, w[2], w[3])[pick]
    sync()
    x, a = ref.row_values(xq1, xs1), ref.row_values(aq1, as1)
    for e in range(E):
        r = slice(e * n, (e + 1) * n)
        check_codes(small[0][r], small[1][r], *ref.swiglu(*ref.product(x[r], wgu[e], 3)), f"few rows, expert {e}")
        check_codes(large[0][r], large[1][r], *ref.swiglu(*ref.product(x[r], wgu[e], 3, codes8=True)),
                    f"many rows, expert {e}")
        want, bound = ref.product(a[r], wd[e], 3, codes8=True)
        tol = product_tolerance(want, bound)
        for y in (y1, y2):
            assert np.all(np.abs(y[r].double().cpu().numpy() - want) <= tol), e


# ---- each step by itself: captured, on a side stream, in its own rows only -------------------------------

def steps(tre, seed):
    """Calls of the operators that the layers are made of, each (call, its outputs, what it reads and may change)."""
    torch = T()
    E, d, I, R = 4, 192, 320, 90
    w, _, _ = weights8(E, d, I, seed)
    wb = rand((E, d, 2 * I), "bf16", seed, 0.05)[0], rand((E, I, d), "bf16", seed + 1, 0.05)[0]
    x, offs = rand((R, d), "bf16", seed + 2)[0], offsets_of([30, 0, 41, 19])
    xq, xs = random_codes((R, d), seed + 3), random_scales((R, ref.blocks(d)), seed + 4, 0.002, 0.02)
    aq, as_ = random_codes((R, I), seed + 5), random_scales((R, ref.blocks(I)), seed + 6, 0.01, 0.02)
    f8 = lambda *n: torch.full(n, 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)   # noqa: E731
    f32 = lambda *n: torch.full(n, float("nan"), device="cuda")                                       # noqa: E731
    y = [torch.full((R, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ws = torch.full((tre.load().moe_grouped_ffn_fp8_workspace_size(R, I),), 0xFF, dtype=torch.uint8, device="cuda")
    q, h = (f8(R, d), f32(R, ref.blocks(d))), (f8(R, I), f32(R, ref.blocks(I)))
    return {
        "rows": (lambda st=None: tre.moe_quantize_rows(x, q=q[0], scale=q[1], stream=st), q, x),
        "weights": (lambda st=None: tre.moe_quantize_weights(*wb, stream=st), None, wb[0]),
        "gate_up": (lambda st=None: tre.moe_gate_up_swiglu_fp8(xq, xs, offs, *w[:2], h_q=h[0], h_s=h[1], stream=st), h, xs),
        "down": (lambda st=None: tre.moe_down_proj_fp8(aq, as_, offs, *w[2:], y_perm=y[0], stream=st), y[:1], as_),
        "ffn": (lambda st=None: tre.moe_grouped_ffn_fp8(xq, xs, offs, *w, y_perm=y[1], workspace=ws, stream=st), y[1:], xs),
    }


def bits(out):
    return [t.view(T().uint8).clone() for t in (out if isinstance(out, (tuple, list)) else [out])]


STEPS = ["rows", "weights", "gate_up", "down", "ffn"]


@pytest.mark.parametrize("step", STEPS)
def test_steps_replayed(tre, step):
    """Captured once, replayed on changing inputs: the eager call's bits each time."""
    torch = T()
    call, out, source = steps(tre, 230)[step]
    call()
    sync()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call()                      # (the weights' outputs belong to the graph)
    for r in range(4):
        source.mul_(0.75 if r % 2 else 1.5)
        g.replay()
        replayed = bits(got)
        for t in out or ():
            t.view(torch.uint8).fill_(0x7F)
        eager = bits(call())
        sync()
        assert all(torch.equal(a, b) for a, b in zip(replayed, eager)), r


@pytest.mark.parametrize("step", STEPS)
def test_steps_on_side_streams(tre, step):
    """Two streams at once, each with its own inputs: the bits of the calls by themselves."""
    torch = T()
    pairs = [steps(tre, 240 + 20 * i)[step][0] for i in range(2)]
    want = [bits(call()) for call in pairs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    sync()
    for _ in range(5):
        got = [call(st) for call, st in zip(pairs, streams)]
        sync()
        for o, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(bits(o), w))


@pytest.mark.parametrize("counts", [[30, 0, 3], [300, 0, 140]])
def test_gate_up_leaves_other_rows(tre, counts):
    """Rows of codes and scales behind the last expert's stay as they were."""
    torch = T()
    d, I, R, spare = 128, 320, sum(counts), 70
    w, _, _ = weights8(3, d, I, 250)
    xq, xs = random_codes((R + spare, d), 251), random_scales((R + spare, 1), 252, 0.002, 0.02)
    hq = torch.full((R + spare, I), 0x55, dtype=torch.uint8, device="cuda")
    hs = torch.full((R + spare, ref.blocks(I)), -3.0, device="cuda")
    tre.moe_gate_up_swiglu_fp8(xq, xs, offsets_of(counts), *w[:2], h_q=hq.view(torch.float8_e4m3fn), h_s=hs)
    sync()
    assert torch.all(hq[R:] == 0x55) and torch.all(hs[R:] == -3.0) and torch.all(hs[:R] > 0)


@pytest.mark.parametrize("offsets", [[0, -5, 60, 40], [70, 10, 1 << 30, 64], [-9, -8, -7, -6], [64, 3, 2, 1]])
def test_offsets_out_of_range(tre, offsets):
    """Offsets that fall, or leave [0, max_rows], are taken back into it: nothing outside the outputs is written, and
    an expert whose own two offsets are in order gets its product."""
    torch = T()
    d, I, R = 192, 128, 64
    w, _, wd = weights8(3, d, I, 260)
    aq, as_ = random_codes((R, I), 261), random_scales((R, 1), 262, 0.01, 0.02)
    xq, xs = random_codes((R, d), 263), random_scales((R, 2), 264, 0.002, 0.02)
    y = torch.full((3 * R, d), 7.0, dtype=torch.bfloat16, device="cuda")
    hq, hs = torch.full((3 * R, I), 0x55, dtype=torch.uint8, device="cuda"), torch.full((3 * R, 1), -3.0, device="cuda")
    offs = to_device(np.array(offsets, np.int32))
    tre.moe_down_proj_fp8(aq, as_, offs, *w[2:], y_perm=y[R:2 * R])
    tre.moe_gate_up_swiglu_fp8(xq, xs, offs, *w[:2], h_q=hq[R:2 * R].view(torch.float8_e4m3fn), h_s=hs[R:2 * R])
    sync()
    for t, v in ((y, 7.0), (hq, 0x55), (hs, -3.0)):
        assert torch.all(t[:R] == v) and torch.all(t[2 * R:] == v)
    clip = np.clip(offsets, 0, R)
    owners = [[e for e in range(3) if clip[e] <= r < clip[e + 1]] for r in range(R)]
    a = ref.row_values(aq, as_)
    for r in range(R):
        if len(owners[r]) == 1:
            want, bound = ref.product(a[r:r + 1], wd[owners[r][0]], 3, codes8=True)
            err = np.abs(y[R + r].double().cpu().numpy() - want[0])
            assert np.all(err <= product_tolerance(want, bound)[0]), r
        elif not owners[r]:
            assert torch.all(y[R + r] == 7.0), r


# ---- the binding ------------------------------------------------------------------------------------

def test_max_rows_without_row_token(tre):
    """Without row_token the rows are x_q's: another max_rows is refused, not passed over."""
    torch = T()
    f8 = torch.float8_e4m3fn
    xq, xs = torch.ones((6, 64), device="cuda").to(f8), torch.ones((6, 1), device="cuda")
    w, ws = torch.ones((2, 128, 64), device="cuda").to(f8), torch.ones((2, 2, 1, 1), device="cuda")
    offs = offsets_of([2, 4])
    for rows in (0, 4, 7):
        with pytest.raises(ValueError, match="max_rows"):
            tre.moe_gate_up_swiglu_fp8(xq, xs, offs, w, ws, max_rows=rows)
    a = tre.moe_gate_up_swiglu_fp8(xq, xs, offs, w, ws, max_rows=6)
    token = to_device(np.arange(6, dtype=np.int32))
    b = tre.moe_gate_up_swiglu_fp8(xq, xs, offs, w, ws, row_token=token)
    c = tre.moe_gate_up_swiglu_fp8(xq, xs, offs, w, ws, row_token=token, max_rows=5)
    assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])
    assert c[0].shape == (5, 64) and c[1].shape == (5, 1)


@pytest.mark.parametrize("form", ["bf16", "f32", "fp8", "layer8"])
def test_flat_pairs(tre, form):
    """Pairs as moe_permute takes them, [T * k] instead of [T, k], as moe_forward does; another length is refused."""
    torch = T()
    T_, d, E, k, I = 5, 128, 4, 2, 64
    w, _, _ = few_weights("fp8" if form == "layer8" else form, E, d, I, 200)
    x, _ = rand((T_, d), "f32" if form == "f32" else "bf16", 201)
    call = (lambda **kw: tre.moe_forward_fp8(x, *w, k, **kw)) if form == "layer8" else \
        (lambda **kw: few_call(tre, form, x, w, k, **kw))
    idx, wt = tre.moe_route_topk(routed(T_, E, k, 202)[0], k)
    want = call(topk_idx=idx, topk_w=wt)[0]
    out, i2, w2 = call(topk_idx=idx.reshape(-1), topk_w=wt.reshape(-1))
    sync()
    assert torch.equal(out, want) and i2.shape == (T_ * k,) and w2.shape == (T_ * k,)
    for i, v in ((idx.reshape(-1)[1:], wt), (idx, wt.reshape(-1)[1:]), (idx.reshape(k, T_), wt)):
        with pytest.raises(ValueError):
            call(topk_idx=i, topk_w=v)


@pytest.mark.parametrize("form", ["bf16", "f32", "fp8", "layer8"])
@pytest.mark.parametrize("given", [False, True])
def test_no_tokens(tre, form, given):
    """An empty batch, as the last step of a server may hold: empty outputs, whatever allocates them."""
    torch = T()
    d, E, k, I = 128, 4, 2, 64
    w, _, _ = few_weights("fp8" if form == "layer8" else form, E, d, I, 220)
    x = torch.empty((0, d), dtype=torch.float32 if form == "f32" else torch.bfloat16, device="cuda")
    pairs = dict(topk_idx=torch.empty((0, k), dtype=torch.int32, device="cuda"), topk_w=torch.empty((0, k), device="cuda"))
    kw = pairs if given else dict(logits=torch.empty((0, E), device="cuda"))
    out, idx, wt = tre.moe_forward_fp8(x, *w, k, **kw) if form == "layer8" else few_call(tre, form, x, w, k, **kw)
    sync()
    assert out.shape == (0, d) and idx.shape == (0, k) and wt.shape == (0, k)


# ---- the widest layers and the most experts -----------------------------------------------------------

WIDE, PIECE = (1 << 22) - 64, 1 << 19


def long_times(a, q):
    """a [n, K] @ codes [N, K] transposed in 64 bits, in pieces of either side."""
    out = T().zeros((a.shape[0], q.shape[0]), dtype=T().float64, device="cuda")
    for n in range(0, q.shape[0], PIECE):
        rows = q[n:n + PIECE]
        for k in range(0, a.shape[1], PIECE):
            part = rows[:, k:k + PIECE].float().double()
            out[:, n:n + PIECE] += a[:, k:k + PIECE].double() @ part.t().contiguous()
    return out


@pytest.mark.parametrize("d,I", [(WIDE, 64), (64, WIDE)])
def test_widest_layers(tre, d, I):
    """Widths next to 2^22.  Codes are +-0.5 and +-1 and every scale 1, so block sums are exact, and so is their sum
    while it stays below 2^22, which random signs see to (checked)."""
    torch = T()
    g = torch.Generator(device="cuda").manual_seed(d)

    def codes(*shape):
        q = torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=g)
        return q.bitwise_and_(0x88).bitwise_or_(0x30).view(torch.float8_e4m3fn)

    def product(a, q):
        pieces = torch.stack([long_times(a[:, k:k + PIECE], q[:, k:k + PIECE]) for k in range(0, a.shape[1], PIECE)])
        assert float(pieces.cumsum(0).abs().max()) < 2.0 ** 21
        return pieces.sum(0)

    R, ones = 37, lambda *shape: torch.ones(shape, device="cuda")   # noqa: E731
    nb, db = ref.blocks(I), ref.blocks(d)
    gq, dq, xq, aq = codes(1, 2 * I, d), codes(1, d, I), codes(R, d), codes(R, I)
    offs, shrink = offsets_of([R]), 2.0 ** -11 if d > I else 2.0 ** -4     # gates of ordinary size
    hq, hs = tre.moe_gate_up_swiglu_fp8(xq, ones(R, db) * shrink, offs, gq, ones(1, 2, nb, db))
    y = tre.moe_down_proj_fp8(aq, ones(R, nb), offs, dq, ones(1, db, nb))
    rows = torch.tensor([0, 15, 16, 31, 32, 36], device="cuda")
    pick = lambda q: q.view(torch.uint8)[rows].view(q.dtype).float()       # noqa: E731
    for n in (0, d - 64) if d > I else (0,):                               # the first and the last columns
        want = product(pick(aq), dq[0, n:n + 64])
        assert torch.equal(y[rows, n:n + 64], want.float().to(torch.bfloat16))
    for n in (0, I - 64) if I > d else (0,):
        gu = torch.cat([product(pick(xq), gq[0, i * I + n:i * I + n + 64]) for i in (0, 1)], 1) * shrink
        h, eh = ref.swiglu(gu.cpu().numpy(), np.zeros(gu.shape))
        # the block's scale comes from all of its 128 columns: only the codes' values are compared here
        got = hq[rows, n:n + 64].double() * hs[rows, n // 128].double()[:, None]
        top = hs[rows, n // 128].double().cpu().numpy()[:, None]
        err = np.abs(got.cpu().numpy() - h)
        assert np.all(err <= eh + np.maximum(2.0 ** -4 * (np.abs(h) + eh), 2.0 ** -10 * top)), n
    # the few-token layer, two tokens
    x = torch.randn((2, d), device="cuda", generator=g).mul(0.5 * shrink).to(torch.bfloat16)
    idx, wt = to_device(np.zeros((2, 1), np.int32)), ones(2, 1)
    out, _, _ = tre.moe_forward_few_fp8(x, gq, ones(1, 2, nb, db), dq, ones(1, db, nb), 1, topk_idx=idx, topk_w=wt)
    gate, up = long_times(x, gq[0]).chunk(2, 1)
    want = long_times(gate / (1 + torch.exp(-gate)) * up, dq[0])
    err = float((out.double() - want).norm() / want.norm())
    # h and the output are rounded to bf16 (independent errors: a half step each in the norm); float32 sums of 2^22
    # terms of random signs add 2^11 steps of 2^-24 to either product
    assert err <= 2 * ref.HALF_BF16 + 2 * 2.0 ** -13, err


@pytest.mark.parametrize("E", [65, 129, 256])
def test_many_experts(tre, E):
    """Groups over all four waves of experts: rows in the first, the last and every third one, exactly."""
    torch = T()
    counts = [(e % 5) * 9 if e % 3 == 0 or e == E - 1 else 0 for e in range(E)]
    counts[0], counts[-1] = 40, 33
    R, K, N = sum(counts), 192, 128
    g = torch.Generator(device="cuda").manual_seed(E)

    def codes(*shape):
        q = torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=g)
        return q.bitwise_and_(0x88).bitwise_or_(0x30).view(torch.float8_e4m3fn)

    aq, as_ = codes(R, K), torch.ones((R, 2), device="cuda")
    w, ws = codes(E, N, K), torch.ones((E, 1, 2), device="cuda")
    y = tre.moe_down_proj_fp8(aq, as_, offsets_of(counts), w, ws)
    at = 0
    for e, n in enumerate(counts):
        want = aq[at:at + n].float().double() @ w[e].float().double().t().contiguous()
        assert torch.equal(y[at:at + n], want.float().to(torch.bfloat16)), e
        at += n
