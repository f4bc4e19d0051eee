"""The serving operators on the GPU against their plain 64-bit forms
(serving_ref): e4m3 blocks bit for bit; products and layers within bounds that
count the roundings of the formulas.  Outputs start as NaN (or a sentinel), so
that what a call leaves unwritten shows."""
import numpy as np
import pytest

import oracle
import serving_ref as ref
from helpers import as_f64, to_device, to_host
import workloads

pytestmark = pytest.mark.gpu


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


def say(msg):
    print("  " + msg, flush=True)


def rand(shape, dtype, seed, std=1.0):
    """(GPU tensor, its float64 values)."""
    a = (np.random.default_rng(seed).standard_normal(shape) * std).astype(np.float32)
    a = a if dtype == "f32" else workloads.bf16_bits(a)
    return to_device(a), as_f64(a)


def random_codes(shape, seed):
    a = np.random.default_rng(seed).standard_normal(shape) * 100
    return T().from_numpy(np.clip(a, -448, 448).astype(np.float32)).to("cuda").to(T().float8_e4m3fn)


def random_scales(shape, seed, lo=1e-4, hi=2e-4):
    return to_device(np.random.default_rng(seed).uniform(lo, hi, shape).astype(np.float32))


def weights8(E, d, I, seed):
    """Random 8-bit weights of a layer with scales that are no powers of two, and their values as [E, K, N]."""
    nb, db = ref.blocks(I), ref.blocks(d)
    w = (random_codes((E, 2 * I, d), seed), random_scales((E, 2, nb, db), seed + 1),
         random_codes((E, d, I), seed + 2), random_scales((E, db, nb), seed + 3))
    return w, ref.weight_values(*w[:2]).transpose(0, 2, 1), ref.weight_values(*w[2:]).transpose(0, 2, 1)


# ---- quantisation: bit for bit ----------------------------------------------------------

def edge_rows(cols, dtype):
    """Rows with the blocks in which a scale or a code can go wrong."""
    big = 3.3895313892515355e38      # the largest bf16
    rows = [np.zeros(cols), np.full(cols, -0.0), np.full(cols, 448.0), np.full(cols, 449.0 if dtype == "f32" else 450.0),
            np.full(cols, 2.0 ** -126), np.full(cols, -2.0 ** -133), np.full(cols, big), np.full(cols, 1.0)]
    for bad in (np.inf, -np.inf, np.nan):
        r = np.linspace(-3, 3, cols)
        r[cols // 2] = bad
        rows.append(r)
    r = np.full(cols, 2.0 ** -60)     # one huge value: the others fall below the smallest code
    r[5] = 1e30
    rows.append(r)
    r = np.tile(np.array([448.0, 17.0, 18.0, 19.0, 0.0146484375, 0.0029296875, 0.0009765625, -0.0048828125]),
                cols // 8)             # ties between codes, normal and subnormal
    rows.append(r)
    for top in (1.75, 1.7578125, 1.0, 1.9921875):   # around 448 = 1.75 * 2^8
        r = np.linspace(-1, 1, cols) * top
        r[0] = top
        rows.append(r)
    return np.array(rows)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 64), (3, 128), (5, 192), (17, 2880), (64, 5120), (1000, 320), (4093, 1024)])
def test_quantize_rows(tre, rows, cols, dtype):
    torch = T()
    rng = np.random.default_rng(rows + cols)
    a = rng.standard_normal((rows, cols)) * np.exp(2 * rng.standard_normal((rows, 1)))
    e = edge_rows(cols, dtype)
    a[rows // 2:rows // 2 + len(e)] = e[:max(0, rows - rows // 2)]
    with np.errstate(over="ignore"):
        x = torch.from_numpy(a).to(torch.float32 if dtype == "f32" else torch.bfloat16).cuda()
    q, s = tre.moe_quantize_rows(x)
    sync()
    want_q, want_s = ref.quantize_rows(x.cpu().double().numpy())
    got_s = s.cpu().numpy().astype(np.float64)
    assert np.array_equal(got_s, want_s, equal_nan=True)
    assert np.array_equal(ref.codes(q), want_q, equal_nan=True)
    # zeros keep their sign, NaN codes are 0x7F
    raw = q.cpu().view(torch.uint8).numpy()
    assert np.all(raw[np.isnan(want_q)] == 0x7F)
    zero = want_q == 0
    assert np.array_equal(raw[zero] >> 7, np.signbit(x.cpu().double().numpy())[zero].astype(np.uint8))


def test_quantize_rows_edges(tre):
    torch = T()
    for dtype in ("bf16", "f32"):
        for cols in (64, 128, 192, 320):
            x = torch.from_numpy(edge_rows(cols, dtype)).to(torch.float32 if dtype == "f32" else torch.bfloat16).cuda()
            q, s = tre.moe_quantize_rows(x)
            sync()
            want_q, want_s = ref.quantize_rows(x.cpu().double().numpy())
            assert np.array_equal(s.cpu().numpy().astype(np.float64), want_s, equal_nan=True), (dtype, cols)
            assert np.array_equal(ref.codes(q), want_q, equal_nan=True), (dtype, cols)


def test_quantize_rows_leaves_the_rest(tre):
    torch = T()
    x, _ = rand((7, 192), "bf16", 3)
    q = torch.full((9, 192), 5, dtype=torch.uint8, device="cuda")
    s = torch.full((9, 2), -3.0, device="cuda")
    tre.moe_quantize_rows(x, q=q.view(torch.float8_e4m3fn)[:7], scale=s[:7])
    sync()
    assert torch.all(q[7:] == 5) and torch.all(s[7:] == -3.0) and torch.all(s[:7] > 0)
    q0, s0 = tre.moe_quantize_rows(x[:0])
    assert q0.shape == (0, 192) and s0.shape == (0, 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E,d,I", [(1, 64, 64), (2, 128, 256), (3, 192, 320), (2, 576, 64), (1, 64, 1088)])
def test_quantize_weights(tre, E, d, I, dtype):
    torch = T()
    wgu, vgu = rand((E, d, 2 * I), dtype, E + d)
    wd, vd = rand((E, I, d), dtype, E + I, std=0.02)
    wgu[0, 0, :I] = 0.0                      # and one non-finite block in the up half
    wgu[0, d - 1, 2 * I - 1] = float("inf")
    vgu = wgu.cpu().double().numpy()
    gq, gs, dq, ds = tre.moe_quantize_weights(wgu, wd)
    sync()
    for e in range(E):
        for half in (0, 1):
            q, s = ref.quantize_matrix(vgu[e, :, half * I:(half + 1) * I].T)
            assert np.array_equal(gs[e, half].cpu().numpy().astype(np.float64), s, equal_nan=True)
            assert np.array_equal(ref.codes(gq[e, half * I:(half + 1) * I]), q, equal_nan=True)
        q, s = ref.quantize_matrix(vd[e].T)
        assert np.array_equal(ds[e].cpu().numpy().astype(np.float64), s)
        assert np.array_equal(ref.codes(dq[e]), q)


# ---- grouped products -----------------------------------------------------------------------

def offsets_of(counts):
    return to_device(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))


GROUPS = [
    [1], [0, 3, 0], [16, 0, 17, 1], [33, 0, 64, 5, 31],           # low tiles
    [40, 65, 0, 50], [128, 70, 129, 1],                            # 64 and 128 rows
    [256, 257, 0, 200], [600, 3, 300], [2100, 0, 17, 900],         # 256 rows, several tiles of one expert
]


def product_tolerance(y, bound):
    return bound + ref.HALF_BF16 * (np.abs(y) + bound) + 1e-37


@pytest.mark.parametrize("counts", GROUPS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("K,N", [(64, 64), (128, 256), (320, 192), (1088, 576)])
def test_down_proj(tre, counts, K, N):
    torch = T()
    R, E = sum(counts), len(counts)
    spare = 5
    x_q, x_s = random_codes((R + spare, K), R + K), random_scales((R + spare, ref.blocks(K)), R, 0.01, 0.02)
    w_q, w_s = random_codes((E, N, K), N), random_scales((E, ref.blocks(N), ref.blocks(K)), N + 1)
    x_q.view(torch.uint8)[R:] = 0x7F          # what lies behind the last row is not read into any result
    x_s[R:] = float("nan")
    y = torch.full((R + spare, N), 7.0, dtype=torch.bfloat16, device="cuda")
    tre.moe_down_proj_fp8(x_q, x_s, offsets_of(counts), w_q, w_s, y_perm=y)
    sync()
    x, w = ref.row_values(x_q, x_s), ref.weight_values(w_q, w_s)
    at, worst = 0, 0.0
    for e, n in enumerate(counts):
        want, bound = ref.product(x[at:at + n], w[e].T, 3, codes8=True)
        got = as_f64(to_host(y[at:at + n]))
        tol = product_tolerance(want, bound)
        assert np.all(np.abs(got - want) <= tol), (e, np.max(np.abs(got - want) / tol))
        worst = max(worst, np.max(np.abs(got - want) / tol, initial=0))
        at += n
    assert torch.all(y[R:] == 7.0)             # rows behind the last expert are left alone
    say(f"down {counts} K={K} N={N}: worst error / bound {worst:.3f}")


def check_codes(h_q, h_s, h, eh, label):
    """Codes and scales of rows whose exact values lie within eh of h: the scale of some value in that range, and
    every code between those of the range's ends (rounding is monotone)."""
    got_s = h_s.cpu().numpy().astype(np.float64)
    cols = h.shape[1]
    pad = np.zeros((h.shape[0], ref.blocks(cols) * 128))
    pad[:, :cols] = np.abs(h)
    pe = np.zeros_like(pad)
    pe[:, :cols] = eh
    lo = ref.power_scale(np.maximum(pad - pe, 0).reshape(h.shape[0], -1, 128).max(-1))
    hi = ref.power_scale((pad + pe).reshape(h.shape[0], -1, 128).max(-1))
    assert np.all((got_s == lo) | (got_s == hi)), label
    s = ref.spread(got_s, cols, 1)
    q = ref.codes(h_q)
    assert np.all(np.isfinite(q)), label
    low, high = ref.round_e4m3(np.clip((h - eh) / s, -448, 448)), ref.round_e4m3(np.clip((h + eh) / s, -448, 448))
    assert np.all((q >= low) & (q <= high)), label
    return float(np.mean(low != high))


@pytest.mark.parametrize("counts", GROUPS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("d,I,gather", [(64, 64, False), (128, 256, True), (320, 192, True), (576, 320, False)])
def test_gate_up(tre, counts, d, I, gather):
    torch = T()
    R, E = sum(counts), len(counts)
    (wgu_q, wgu_s, _, _), wgu, _ = weights8(E, d, I, 10 + d)
    n_x = 50 if gather else R
    x_q, x_s = random_codes((n_x, d), R + d), random_scales((n_x, ref.blocks(d)), R, 0.002, 0.02)
    x = ref.row_values(x_q, x_s)
    row_token = None
    if gather:
        rt = np.random.default_rng(R).integers(0, n_x, R).astype(np.int32)
        row_token, x = to_device(rt), x[rt]
    h_q = torch.full((R, I), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    h_s = torch.full((R, ref.blocks(I)), float("nan"), device="cuda")
    tre.moe_gate_up_swiglu_fp8(x_q, x_s, offsets_of(counts), wgu_q, wgu_s, h_q=h_q, h_s=h_s, row_token=row_token)
    sync()
    at = 0
    for e, n in enumerate(counts):
        if n:
            gu, egu = ref.product(x[at:at + n], wgu[e], 3, codes8=True)
            h, eh = ref.swiglu(gu, egu)
            check_codes(h_q[at:at + n], h_s[at:at + n], h, eh, f"expert {e} of {counts}")
        at += n


@pytest.mark.parametrize("E,rows,d,I", [(13, 4, 64, 2560), (3, 1, 320, 192), (16, 30, 192, 2048), (4, 21, 1024, 64)])
def test_gate_up_few_rows_exact(tre, E, rows, d, I):
    """With up to 42 rows an expert the products are exact but for float32 sums: nothing of an 8-bit instruction's
    alignment may show in the codes."""
    counts = [rows] * E
    (wgu_q, wgu_s, _, _), wgu, _ = weights8(E, d, I, 30 + E)
    x_q, x_s = random_codes((E * rows, d), 31), random_scales((E * rows, ref.blocks(d)), 32, 0.002, 0.02)
    h_q, h_s = tre.moe_gate_up_swiglu_fp8(x_q, x_s, offsets_of(counts), wgu_q, wgu_s)
    sync()
    x = ref.row_values(x_q, x_s)
    for e in range(E):
        s = slice(e * rows, (e + 1) * rows)
        h, eh = ref.swiglu(*ref.product(x[s], wgu[e], 3))
        check_codes(h_q[s], h_s[s], h, eh, f"expert {e}")


def short_codes(shape, seed):
    """Codes +-0.5, +-1, +-2 and 0: every product is a multiple of 0.25 up to 4, so a matrix instruction loses
    nothing and every partial sum below 2^22 is exact in float32."""
    v = np.array([0.0, 0.5, 1.0, 2.0, -0.5, -1.0, -2.0], dtype=np.float32)
    return T().from_numpy(v[np.random.default_rng(seed).integers(0, 7, shape)]).to("cuda").to(T().float8_e4m3fn)


def power_scales(shape, seed):
    return to_device(np.exp2(np.random.default_rng(seed).integers(-4, 1, shape)).astype(np.float32))


@pytest.mark.parametrize("counts", GROUPS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("d,I", [(128, 64), (192, 320), (576, 256)])
def test_products_exact(tre, counts, d, I):
    """Codes and scales whose sums are exact in float32 in any order: the down projection gives the bf16 rounding of
    the exact sum bit for bit, and gate/up codes may differ only where silu's float32 error crosses a rounding."""
    torch = T()
    R, E = sum(counts), len(counts)
    offs, nb, db = offsets_of(counts), ref.blocks(I), ref.blocks(d)
    gq, gs = short_codes((E, 2 * I, d), 1), power_scales((E, 2, nb, db), 2)
    dq, ds = short_codes((E, d, I), 3), power_scales((E, db, nb), 4)
    xq, xs = short_codes((R, d), 5), power_scales((R, db), 6)
    xs *= 0.125
    hq, hs = tre.moe_gate_up_swiglu_fp8(xq, xs, offs, gq, gs)
    aq, as_ = short_codes((R, I), 7), power_scales((R, nb), 8)
    y = tre.moe_down_proj_fp8(aq, as_, offs, dq, ds)
    sync()
    x, wgu = ref.row_values(xq, xs), ref.weight_values(gq, gs)
    a, wd = ref.row_values(aq, as_), ref.weight_values(dq, ds)
    at = 0
    for e, n in enumerate(counts):
        rows = slice(at, at + n)
        exact = a[rows] @ wd[e].T
        assert np.array_equal(as_f64(to_host(y[rows])), as_f64(workloads.bf16_bits(exact.astype(np.float32)))), e
        if n:
            gu = x[rows] @ wgu[e].T
            h, eh = ref.swiglu(gu, np.zeros_like(gu))
            loose = check_codes(hq[rows], hs[rows], h, eh, f"expert {e} of {counts}")
            # an open code has a rounding border within 8 half steps of float32: about 2^-16 of them, few by chance
            assert loose * h.size <= 4 + 1e-3 * h.size, "the bound leaves too many codes open to check anything"
        at += n


def spread_groups(rows):
    """24 experts of about `rows` rows: enough tiles for every height, with an empty expert, one row, one row past a
    tile's edge, and one expert of several tiles."""
    counts = np.random.default_rng(rows).integers(rows // 2, rows + rows // 2, 24)
    counts[[0, 5, 7, 9]] = 0, 1, rows * 2 + 1, rows * 5
    return [int(c) for c in counts]


@pytest.mark.parametrize("rows", [30, 60, 96, 144, 250])           # tiles of 64, 128 and 288 rows, 160 in the last
@pytest.mark.parametrize("K", [64, 192, 320, 384, 512, 1088])      # 1 to 9 stages, with and without half a block
def test_products_exact_many_tiles(tre, rows, K):
    """As above with more tiles than compute units, so that a workgroup walks from one tile to the next; the exact
    sums in 64 bits on the GPU."""
    torch = T()
    counts, I, N = spread_groups(rows), 1408, 2880 if rows < 200 else 1408
    R, E, kb = sum(counts), len(counts), ref.blocks(K)
    offs = offsets_of(counts)

    def spread(codes, scales):   # [n, k] codes with scales [n / 128 or n, k / 128]
        s = scales.double().repeat_interleave(128, 1)[:, :codes.shape[1]]
        s = s if s.shape[0] == codes.shape[0] else s.repeat_interleave(128, 0)[:codes.shape[0]]
        return codes.float().double() * s

    xq, xs = short_codes((R, K), 5), power_scales((R, kb), 6)
    wq, ws = short_codes((E, N, K), 3), power_scales((E, ref.blocks(N), kb), 4)
    y = tre.moe_down_proj_fp8(xq, xs, offs, wq, ws)
    at = 0
    for e, n in enumerate(counts):
        exact = spread(xq[at:at + n], xs[at:at + n]) @ spread(wq[e], ws[e]).t().contiguous()
        assert torch.equal(y[at:at + n], exact.float().to(torch.bfloat16)), (e, n)
        at += n
    gq, gs = short_codes((E, 2 * I, K), 1), power_scales((E, 2, ref.blocks(I), kb), 2)
    xs *= 0.125
    token = to_device(np.random.default_rng(K).permutation(R).astype(np.int32))
    hq, hs = tre.moe_gate_up_swiglu_fp8(xq, xs, offs, gq, gs, row_token=token)
    at = 0
    for e, n in enumerate(counts):
        if n:
            r = token[at:at + n].long()
            x = spread(xq.view(torch.uint8)[r].view(torch.float8_e4m3fn), xs[r])
            gu = torch.cat([x @ spread(gq[e, i * I:(i + 1) * I], gs[e, i]).t().contiguous() for i in (0, 1)], 1)
            h, eh = ref.swiglu(gu.cpu().numpy(), np.zeros((n, 2 * I)))
            check_codes(hq[at:at + n], hs[at:at + n], h, eh, f"expert {e} of {counts}")
        at += n


def test_gate_up_rows_out_of_range(tre):
    """A row_token outside [0, x_rows) reads zeros: its h is zero, and no other row changes."""
    torch = T()
    E, d, I, R = 2, 128, 128, 40
    (wgu_q, wgu_s, _, _), _, _ = weights8(E, d, I, 1)
    x_q, x_s = random_codes((20, d), 2), random_scales((20, 1), 3)
    good = np.random.default_rng(4).integers(0, 20, R).astype(np.int32)
    bad = good.copy()
    bad[3], bad[30] = -1, 20
    offs = offsets_of([25, 15])
    a = tre.moe_gate_up_swiglu_fp8(x_q, x_s, offs, wgu_q, wgu_s, row_token=to_device(good))
    b = tre.moe_gate_up_swiglu_fp8(x_q, x_s, offs, wgu_q, wgu_s, row_token=to_device(bad))
    sync()
    qa, qb = (t[0].view(torch.uint8).cpu().numpy() for t in (a, b))
    keep = np.ones(R, bool)
    keep[[3, 30]] = False
    assert np.array_equal(qa[keep], qb[keep]) and np.all(ref.codes(b[0])[~keep] == 0)


def test_products_spread_nan_only_along_their_row(tre):
    """A row with a NaN scale gives a NaN row; the tile's other rows are those of the call without it."""
    torch = T()
    counts, K, N = [20, 300], 192, 320
    w_q, w_s = random_codes((2, N, K), 1), random_scales((2, 3, 2), 2)
    x_q, x_s = random_codes((320, K), 3), random_scales((320, 2), 4)
    y0 = tre.moe_down_proj_fp8(x_q, x_s, offsets_of(counts), w_q, w_s)
    x_s[7, 1], x_s[200, 0] = float("nan"), float("nan")
    y1 = tre.moe_down_proj_fp8(x_q, x_s, offsets_of(counts), w_q, w_s)
    sync()
    keep = torch.ones(320, dtype=torch.bool, device="cuda")
    keep[[7, 200]] = False
    assert torch.equal(y0[keep], y1[keep]) and torch.all(torch.isnan(y1[~keep]))


def test_product_signs_and_blocks(tre):
    """One-hot rows pick single weights: value, sign and scale of each come out exactly."""
    torch = T()
    K, N = 320, 192
    w_q, _ = random_codes((1, N, K), 5), None
    w_s = torch.from_numpy(np.exp2(np.random.default_rng(6).integers(-6, 6, (1, 2, 3))).astype(np.float32)).cuda()
    x = torch.eye(K, device="cuda") * 2.0
    x_q, x_s = tre.moe_quantize_rows(x)
    y = tre.moe_down_proj_fp8(x_q, x_s, offsets_of([K]), w_q, w_s)
    sync()
    want = 2.0 * ref.weight_values(w_q, w_s)[0].T
    assert np.array_equal(as_f64(to_host(y)), want)


def test_grouped_ffn_is_its_halves(tre):
    torch = T()
    counts, d, I = [100, 0, 37, 260], 192, 320
    w, _, _ = weights8(4, d, I, 20)
    x_q, x_s = tre.moe_quantize_rows(rand((sum(counts), d), "bf16", 21)[0])
    offs = offsets_of(counts)
    ws = torch.full((tre.load().moe_grouped_ffn_fp8_workspace_size(sum(counts), I),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    y = tre.moe_grouped_ffn_fp8(x_q, x_s, offs, *w, workspace=ws)
    h = tre.moe_gate_up_swiglu_fp8(x_q, x_s, offs, w[0], w[1])
    assert torch.equal(y, tre.moe_down_proj_fp8(*h, offs, w[2], w[3]))
    y0 = tre.moe_grouped_ffn_fp8(x_q[:0], x_s[:0], offsets_of([0, 0, 0, 0]), *w)
    assert y0.shape == (0, d)


# ---- the layer on 8-bit weights -----------------------------------------------------------------

def routed(T_, E, k, seed, ties=False):
    rng = np.random.default_rng(seed)
    lg = rng.integers(-2, 3, (T_, E)).astype(np.float32) if ties else rng.standard_normal((T_, E)).astype(np.float32)
    return to_device(lg), lg


@pytest.mark.parametrize("T_,d,E,k,I,given", [
    (1, 64, 1, 1, 64, False), (3, 128, 8, 2, 192, False), (40, 320, 5, 3, 256, True), (300, 192, 16, 4, 320, False),
    (1500, 256, 4, 2, 128, True), (2600, 128, 9, 1, 192, False)])
def test_forward_fp8_is_its_steps(tre, T_, d, E, k, I, given):
    """The layer equals its steps through their own entry points (each tested by itself) bit for bit."""
    torch = T()
    w, _, _ = weights8(E, d, I, 30)
    x, _ = rand((T_, d), "bf16", T_)
    if given:
        rng = np.random.default_rng(31)
        ids = rng.integers(-1, E, (T_, k)).astype(np.int32)
        ids[0] = -1                                   # a token without any pair
        idx, wt, lg = to_device(ids), to_device(rng.random((T_, k)).astype(np.float32)), None
    else:
        lg, _ = routed(T_, E, k, 32, ties=True)
        idx, wt = tre.moe_route_topk(lg, k)
    out = torch.full((T_, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = torch.full((tre.moe_forward_fp8_workspace_size(T_, d, E, k, I),), 0xFF, dtype=torch.uint8, device="cuda")
    kw = dict(topk_idx=idx, topk_w=wt) if given else dict(logits=lg)
    pr = torch.empty(T_ * k, dtype=torch.int32, device="cuda")
    _, i2, w2 = tre.moe_forward_fp8(x, *w, k, out=out, workspace=ws, pair_row=pr, **kw)
    _, rt, pair_row, offs = tre.moe_permute(x, idx, k, E, move_rows=False)
    h = tre.moe_gate_up_swiglu_fp8(*tre.moe_quantize_rows(x), offs, w[0], w[1], row_token=rt)
    y = tre.moe_down_proj_fp8(*h, offs, w[2], w[3])
    want = tre.moe_combine(y, pair_row, wt, T_, k)
    sync()
    assert torch.equal(i2, idx) and torch.equal(w2, wt) and torch.equal(pr, pair_row)
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    if given:
        assert torch.all(out[0] == 0)


def test_forward_fp8_empty(tre):
    torch = T()
    w, _, _ = weights8(2, 64, 64, 1)
    out, idx, _ = tre.moe_forward_fp8(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), *w, 1,
                                      logits=torch.empty((0, 2), device="cuda"))
    assert out.shape == (0, 64) and idx.shape == (0, 1)


# ---- the layer for a few tokens --------------------------------------------------------------------

def few_weights(form, E, d, I, seed):
    """(arguments of the call, [E, d, 2I] and [E, I, d] values)."""
    if form == "fp8":
        return weights8(E, d, I, seed)
    a, va = rand((E, d, 2 * I), form, seed, 0.05)
    b, vb = rand((E, I, d), form, seed + 1, 0.05)
    return (a, b), va, vb


def few_call(tre, form, x, w, k, **kw):
    return (tre.moe_forward_few_fp8 if form == "fp8" else tre.moe_forward_few)(x, *w, k, **kw)


def few_ws(tre, form, T_, d, E, k, I):
    torch = T()
    if form == "fp8":
        n = tre.moe_forward_few_fp8_workspace_size(T_, d, E, k, I)
    else:
        n = tre.moe_forward_few_workspace_size(T_, d, E, k, I, tre.MOE_F32 if form == "f32" else tre.MOE_BF16)
    assert n > 0
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")


def few_check(form, got, x, idx, wt, vgu, vd, label):
    half = ref.HALF_F32 if form == "f32" else ref.HALF_BF16
    want, tol = ref.layer(x, idx, wt, vgu, vd, half if form != "f32" else 0.0, half, 3 if form == "fp8" else 0)
    err = np.abs(as_f64(to_host(got)) - want)
    assert not np.any(np.isnan(err)), label
    assert np.all(err <= tol), (label, np.max(err / tol))
    say(f"{label}: worst error / bound {np.max(err / tol, initial=0):.3f}, "
        f"rel {np.linalg.norm(err) / max(np.linalg.norm(want), 1e-300):.1e}")


FEW = [
    (1, 64, 1, 1, 64), (1, 128, 8, 2, 256), (3, 192, 16, 4, 320), (2, 2880, 6, 4, 192), (15, 320, 7, 7, 64),
    (16, 128, 128, 4, 192), (17, 64, 5, 1, 1088), (33, 256, 40, 3, 128), (64, 192, 4, 2, 320), (64, 64, 256, 16, 64),
    (5, 1088, 200, 8, 64), (4, 64, 256, 256, 64), (64, 128, 2, 1, 576),
]


@pytest.mark.parametrize("form", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("T_,d,E,k,I", FEW)
def test_few_routed(tre, T_, d, E, k, I, form):
    torch = T()
    w, vgu, vd = few_weights(form, E, d, I, 40 + E)
    dtype = "f32" if form == "f32" else "bf16"
    x, vx = rand((T_, d), dtype, T_ + d)
    lg, lg_np = routed(T_, E, k, 41, ties=E > 20)
    out = torch.full((T_, d), float("nan"), dtype=x.dtype, device="cuda")
    idx = torch.full((T_, k), -9, dtype=torch.int32, device="cuda")
    wt = torch.full((T_, k), float("nan"), device="cuda")
    few_call(tre, form, x, w, k, logits=lg, topk_idx=idx, topk_w=wt, out=out, workspace=few_ws(tre, form, T_, d, E, k, I))
    want_idx, want_w = tre.moe_route_topk(lg, k)
    sync()
    assert np.array_equal(to_host(idx), oracle.route(lg_np, k)[0])
    assert torch.equal(idx, want_idx) and torch.equal(wt.view(torch.int32), want_w.view(torch.int32))
    few_check(form, out, vx, to_host(idx), to_host(wt).astype(np.float64), vgu, vd, f"few {form} {T_, d, E, k, I}")


@pytest.mark.parametrize("form", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("T_,d,E,k,I", [(1, 64, 4, 1, 64), (9, 192, 6, 3, 128), (20, 128, 3, 40, 192), (64, 320, 16, 2, 64),
                                        (40, 64, 8, 6, 320)])
def test_few_given_pairs(tre, T_, d, E, k, I, form):
    """Given pairs: masked ones, ids out of range, one expert several times in a token (k may pass E), a token
    without any pair, weights of zero."""
    torch = T()
    w, vgu, vd = few_weights(form, E, d, I, 50)
    x, vx = rand((T_, d), "f32" if form == "f32" else "bf16", T_)
    rng = np.random.default_rng(51)
    ids = rng.integers(-1, E, (T_, k)).astype(np.int32)
    if T_ > 4:
        ids[1], ids[2] = -1, E - 1
        ids[3, 0], ids[4, 0] = E, -2 ** 31
    wts = rng.random((T_, k)).astype(np.float32)
    wts[0, 0] = 0.0
    idx, wt = to_device(ids), to_device(wts)
    out = torch.full((T_, d), float("nan"), dtype=x.dtype, device="cuda")
    few_call(tre, form, x, w, k, topk_idx=idx, topk_w=wt, out=out, workspace=few_ws(tre, form, T_, d, E, k, I))
    sync()
    assert np.array_equal(to_host(idx), ids) and np.array_equal(to_host(wt), wts)
    few_check(form, out, vx, ids, wts.astype(np.float64), vgu, vd, f"few given {form} {T_, d, E, k, I}")
    if T_ > 4:
        assert torch.all(out[1] == 0)


@pytest.mark.parametrize("form", ["bf16", "f32", "fp8"])
def test_few_no_pairs_at_all(tre, form):
    torch = T()
    w, _, _ = few_weights(form, 3, 192, 64, 60)
    x, _ = rand((5, 192), "f32" if form == "f32" else "bf16", 61)
    out = torch.full((5, 192), float("nan"), dtype=x.dtype, device="cuda")
    few_call(tre, form, x, w, 2, topk_idx=torch.full((5, 2), -1, dtype=torch.int32, device="cuda"),
             topk_w=torch.full((5, 2), float("nan"), device="cuda"), out=out)
    sync()
    assert torch.all(out == 0)


@pytest.mark.parametrize("form", ["bf16", "f32", "fp8"])
def test_few_masked_tokens_touch_nobody(tre, form):
    """NaN and infinity in a token without pairs, and as the weight of a masked pair, reach no output."""
    torch = T()
    T_, d, E, k, I = 20, 128, 4, 2, 64
    w, vgu, vd = few_weights(form, E, d, I, 70)
    x, vx = rand((T_, d), "f32" if form == "f32" else "bf16", 71)
    ids = np.random.default_rng(72).integers(0, E, (T_, k)).astype(np.int32)
    ids[6], ids[7, 1] = -1, -1
    wts = np.random.default_rng(73).random((T_, k)).astype(np.float32)
    x[6, 5], x[6, 9], x[6, 127] = float("nan"), float("inf"), float("-inf")
    wts[6], wts[7, 1] = np.nan, np.inf
    out, _, _ = few_call(tre, form, x, w, k, topk_idx=to_device(ids), topk_w=to_device(wts))
    sync()
    assert torch.all(out[6] == 0)
    vx[6] = 0
    few_check(form, out, vx, ids, np.where(ids >= 0, wts, 0).astype(np.float64), vgu, vd, f"few masked {form}")


@pytest.mark.parametrize("form", ["bf16", "fp8"])
def test_few_nan_stays_in_its_token(tre, form):
    torch = T()
    T_, d, E, k, I = 18, 192, 2, 1, 128
    w, _, _ = few_weights(form, E, d, I, 80)
    x, _ = rand((T_, d), "bf16", 81)
    lg, _ = routed(T_, E, k, 82)
    a, _, _ = few_call(tre, form, x, w, k, logits=lg)
    x[4, 100] = float("nan")
    b, _, _ = few_call(tre, form, x, w, k, logits=lg)
    sync()
    keep = torch.arange(T_, device="cuda") != 4
    assert torch.equal(a[keep], b[keep]) and torch.all(torch.isnan(b[4]))


def test_few_near_the_full_layer(tre):
    """The same layer through moe_forward: both within the bound of the same formula (and the outputs' own rounding
    of the experts' rows there)."""
    T_, d, E, k, I = 30, 256, 8, 2, 320
    w, vgu, vd = few_weights("bf16", E, d, I, 90)
    x, vx = rand((T_, d), "bf16", 91)
    lg, _ = routed(T_, E, k, 92)
    a, ia, wa = tre.moe_forward_few(x, *w, k, logits=lg)
    b, ib, wb = tre.moe_forward(x, *w, k, logits=lg)
    sync()
    assert T().equal(ia, ib) and T().equal(wa, wb)
    rel = (a.double() - b.double()).norm() / b.double().norm()
    say(f"few against the full layer: rel {float(rel):.1e}")
    assert rel <= 2 * ref.HALF_BF16


# ---- the serving path together ------------------------------------------------------------------------

def test_prompt_then_decode(tre):
    """A model's life: weights quantised once, a prompt through the 8-bit layer, then decode steps through the
    few-token layer on the same weights -- each step near the bf16 layer by what 8 bits cost."""
    torch = T()
    d, E, k, I = 320, 16, 2, 192
    wgu, _ = rand((E, d, 2 * I), "bf16", 100, 0.05)
    wd, _ = rand((E, I, d), "bf16", 101, 0.05)
    w_router, _ = rand((E, d), "bf16", 102, 0.05)
    w8 = tre.moe_quantize_weights(wgu, wd)
    x, _ = rand((200, d), "bf16", 103)
    idx, wt = tre.moe_route_project(x, w_router, k)
    full, _, _ = tre.moe_forward(x, wgu, wd, k, topk_idx=idx, topk_w=wt)
    prompt, _, _ = tre.moe_forward_fp8(x, *w8, k, topk_idx=idx, topk_w=wt)
    steps = torch.cat([tre.moe_forward_few_fp8(x[t:t + n], *w8, k, topk_idx=idx[t:t + n].contiguous(),
                                               topk_w=wt[t:t + n].contiguous())[0]
                       for t, n in ((0, 1), (1, 1), (2, 14), (16, 64), (80, 64), (144, 56))])
    sync()
    # An e4m3 rounding is off by D = 2^-4 / sqrt(3) of the value at most in the root mean square (uniform over half
    # steps of 2^-4 2^e, |v| >= 2^e).  Independent errors add in quadrature: in h, silu multiplies g's by at most
    # 1 + max g (1 - s(g)) = 1.28 over the values with any weight.  Decode: Wg, Wu, Wd: sqrt(1.28^2 + 1 + 1) D =
    # 1.91 D.  Prompt: x reaches g and u together, 2.28 D; with Wg, Wu, h, Wd: sqrt(2.28^2 + 1.28^2 + 3) D = 3.13 D.
    D = 2.0 ** -4 / 3 ** 0.5
    size = full.double().norm()
    e_prompt, e_steps = (float((o.double() - full.double()).norm() / size) for o in (prompt, steps))
    say(f"prompt {e_prompt:.3f}, decode {e_steps:.3f} off the bf16 layer")
    assert e_prompt <= 3.13 * D and e_steps <= 1.91 * D and e_steps < e_prompt


def captured(torch, fn):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn()
    return g


@pytest.mark.parametrize("form", ["bf16", "f32", "fp8", "layer8"])
def test_graph_replays(tre, form):
    """Captured once, replayed on new inputs with eager calls (sharing nothing, then the workspace) in between:
    every replay gives the eager call's bits."""
    torch = T()
    T_, d, E, k, I = 12, 192, 8, 2, 320
    w, _, _ = few_weights("fp8" if form == "layer8" else form, E, d, I, 110)
    dtype = "f32" if form == "f32" else "bf16"
    x, _ = rand((T_, d), dtype, 111)
    lg, _ = routed(T_, E, k, 112)
    if form == "layer8":
        ws = torch.empty(tre.moe_forward_fp8_workspace_size(T_, d, E, k, I), dtype=torch.uint8, device="cuda")
        call = lambda x, lg, out, idx, wt, ws: tre.moe_forward_fp8(x, *w, k, logits=lg, topk_idx=idx, topk_w=wt,   # noqa: E731
                                                                   out=out, workspace=ws)
    else:
        ws = few_ws(tre, form, T_, d, E, k, I)
        call = lambda x, lg, out, idx, wt, ws: few_call(tre, form, x, w, k, logits=lg, topk_idx=idx, topk_w=wt,    # noqa: E731
                                                        out=out, workspace=ws)
    bufs = lambda: (torch.empty_like(x), torch.empty((T_, k), dtype=torch.int32, device="cuda"),                   # noqa: E731
                    torch.empty((T_, k), device="cuda"))
    got = bufs()
    g = captured(torch, lambda: call(x, lg, *got, ws))
    for r in range(5):
        nx, _ = rand((T_, d), dtype, 120 + r)
        nl, _ = routed(T_, E, k, 130 + r)
        want = bufs()
        call(nx, nl, *want, ws if r % 2 else torch.empty_like(ws))
        x.copy_(nx)
        lg.copy_(nl)
        for b in got:
            b.zero_()
        g.replay()
        sync()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (form, r)


@pytest.mark.parametrize("form", ["bf16", "f32", "fp8"])
def test_few_two_streams(tre, form):
    """Calls that overlap on two streams, each with a workspace of its own (the binding's): the bits of calls alone,
    over and over."""
    torch = T()
    T_, d, E, k, I = 8, 320, 16, 3, 256
    w, _, _ = few_weights(form, E, d, I, 140)
    dtype = "f32" if form == "f32" else "bf16"
    xs = [rand((T_, d), dtype, 141 + i)[0] for i in range(2)]
    lgs = [routed(T_, E, k, 143 + i)[0] for i in range(2)]
    want = [few_call(tre, form, x, w, k, logits=lg) for x, lg in zip(xs, lgs)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    sync()
    got = [few_call(tre, form, xs[i % 2], w, k, logits=lgs[i % 2], stream=streams[i % 2]) for i in range(20)]
    sync()
    for i, o in enumerate(got):
        for a, b in zip(o, want[i % 2]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i


def test_layer8_two_streams(tre):
    """The 8-bit layer on two streams at once, each call's workspace its own."""
    torch = T()
    T_, d, E, k, I = 300, 320, 8, 2, 256
    w, _, _ = weights8(E, d, I, 150)
    xs = [rand((T_, d), "bf16", 151 + i)[0] for i in range(2)]
    lgs = [routed(T_, E, k, 153 + i)[0] for i in range(2)]
    want = [tre.moe_forward_fp8(x, *w, k, logits=lg) for x, lg in zip(xs, lgs)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    sync()
    got = [tre.moe_forward_fp8(xs[i % 2], *w, k, logits=lgs[i % 2], stream=streams[i % 2]) for i in range(10)]
    sync()
    for i, o in enumerate(got):
        for a, b in zip(o, want[i % 2]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i


def test_two_graphs_share_a_workspace(tre):
    """Two captured steps of different sizes in one workspace, replayed in turn: each finds the other's leftovers."""
    torch = T()
    d, E, k, I = 192, 8, 2, 128
    w, _, _ = few_weights("bf16", E, d, I, 160)
    ws = torch.full((max(tre.moe_forward_few_workspace_size(t, d, E, k, I, tre.MOE_BF16) for t in (3, 40)),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    runs = []
    for t in (3, 40):
        x, lg = rand((t, d), "bf16", 161 + t)[0], routed(t, E, k, 162 + t)[0]
        want = tre.moe_forward_few(x, *w, k, logits=lg)[0]
        out = torch.empty_like(x)
        idx, wt = torch.empty((t, k), dtype=torch.int32, device="cuda"), torch.empty((t, k), device="cuda")
        call = lambda x=x, lg=lg, out=out, idx=idx, wt=wt: tre.moe_forward_few(   # noqa: E731
            x, *w, k, logits=lg, topk_idx=idx, topk_w=wt, out=out, workspace=ws)
        runs.append((captured(torch, call), out, want, call))   # call holds the tensors that the graph reads
    for r in range(6):
        g, out, want, _ = runs[r % 2]
        out.fill_(float("nan"))
        g.replay()
        sync()
        assert torch.equal(out, want), r


@pytest.mark.parametrize("T_,d,E,k,I", [(1, 128, 4, 2, 64), (40, 192, 16, 3, 320), (700, 256, 4, 2, 576)])
def test_device_checked_build_equals_release(tre, T_, d, E, k, I):
    """libmoe_debug.so (valid input only: a value outside its contract stops it) gives the same bits."""
    import os
    torch = T()
    assert os.path.exists(tre.DEBUG_LIB_PATH), "libmoe_debug.so is not built"
    dbg = tre.open_library(tre.DEBUG_LIB_PATH)
    w, _, _ = weights8(E, d, I, 170)
    wb, _, _ = few_weights("bf16", E, d, I, 171)
    x, _ = rand((T_, d), "bf16", 172)
    lg, _ = routed(T_, E, k, 173)
    calls = [lambda: tre.moe_quantize_rows(x), lambda: tre.moe_quantize_weights(*wb),
             lambda: tre.moe_forward_fp8(x, *w, k, logits=lg)]
    if T_ <= 64:
        calls += [lambda: tre.moe_forward_few(x, *wb, k, logits=lg),
                  lambda: tre.moe_forward_few_fp8(x, *w, k, logits=lg)]
    release = tre.load()
    for call in calls:
        a = call()
        try:
            tre._lib = dbg
            b = call()
        finally:
            tre._lib = release
        sync()
        for u, v in zip(a, b):
            assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))


def test_binding_checks(tre):
    torch = T()
    x, _ = rand((4, 128), "bf16", 1)
    w, _, _ = few_weights("bf16", 4, 128, 64, 2)
    w8, _, _ = few_weights("fp8", 4, 128, 64, 3)
    lg, _ = routed(4, 4, 2, 4)
    with pytest.raises(ValueError):
        tre.moe_forward_few(x.t(), *w, 2, logits=lg)
    with pytest.raises(ValueError):
        tre.moe_forward_few(x, *w, 2)                                         # neither logits nor pairs
    with pytest.raises(ValueError):
        tre.moe_forward_few(x, *w, 2, logits=lg, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        tre.moe_forward_few_fp8(x.float(), *w8, 2, logits=lg)                 # activations are bf16
    with pytest.raises(ValueError):
        tre.moe_forward_few(x, *w, 2, logits=lg.cpu())
    with pytest.raises(ValueError):
        tre.moe_quantize_rows(x[:, ::2])                                      # strided
    with pytest.raises(tre.MoeError) as e:
        tre.moe_forward_few(x, *w, 5, logits=lg)
    assert e.value.status == 1
    big, _ = rand((65, 128), "bf16", 5)
    with pytest.raises(tre.MoeError) as e:
        tre.moe_forward_few(big, *w, 2, logits=routed(65, 4, 2, 6)[0])
    assert e.value.status == 2
    flat = torch.empty(4 * 128 + 1, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(tre.MoeError) as e:                                    # rows off a 16-byte boundary
        tre.moe_forward_few(flat[1:].view(4, 128), *w, 2, logits=lg)
    assert e.value.status == 1
