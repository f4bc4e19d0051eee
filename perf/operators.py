"""The layer's 8-bit and few-token operators as measured work: their plain forms in elementary torch operations, the
framework's calls, and the definition in 64 bits.

Kinds of cases:
  rows     moe_quantize_rows: activation rows to e4m3 with one scale for each block of 128 columns
  weights  moe_quantize_weights: expert weights to e4m3, transposed to [N, K], one scale for each block of 128 x 128
  product  moe_down_proj_fp8: the grouped product of 8-bit rows with 8-bit expert weights
  layer8   moe_forward_fp8: the whole layer on 8-bit expert weights
  few      moe_forward_few / moe_forward_few_fp8: the whole layer for a few tokens, in two kernels

`own` selects the framework's calls; the plain forms need torch only.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 128
F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ------------------------------------------------------------------------

def listed():
    return [
        # one decode step's activations before an 8-bit product: 64 rows, latency counts
        dict(name="rows_decode", kind="rows", rows=64, cols=5120, dtype="bf16"),
        # a prompt batch's activations, width with a half block at its end
        dict(name="rows_batch", kind="rows", rows=8192, cols=2880, dtype="bf16"),
        # float32 activations, an odd number of rows
        dict(name="rows_f32", kind="rows", rows=4093, cols=1024, dtype="f32"),
        # a layer's weights when a model is loaded: 16 experts
        dict(name="weights_small", kind="weights", E=16, d=1024, I=2816, dtype="bf16"),
        # a decode step's down projection: four rows an expert, the weights' bytes are the work
        dict(name="product_decode", kind="product", rows=64, E=16, K=8192, N=5120, skew=False),
        # the rows one expert-parallel rank received, skewed, three experts without rows
        dict(name="product_rank", kind="product", rows=32768, E=16, K=2880, N=2880, skew=True),
        # a prompt batch through a 16-expert layer
        dict(name="layer8_small", kind="layer8", T=4096, d=1024, E=16, k=2, I=2816),
        # a prompt batch through a 128-expert layer
        dict(name="layer8_large", kind="layer8", T=8192, d=2880, E=128, k=4, I=2880),
        # three tokens of a tiny float32 layer: launches are all that counts
        dict(name="few_tiny_f32", kind="few", T=3, d=128, E=8, k=2, I=256, weights="f32", given=False),
        # one token of one sequence: four of 128 experts
        dict(name="few_one_bf16", kind="few", T=1, d=2880, E=128, k=4, I=2880, weights="bf16", given=False),
        # a batch of 64 sequences, one step each, one expert a token, already routed
        dict(name="few_batch_bf16", kind="few", T=64, d=5120, E=16, k=1, I=8192, weights="bf16", given=True),
        # eight sequences on 8-bit weights
        dict(name="few_eight_fp8", kind="few", T=8, d=2880, E=128, k=4, I=2880, weights="fp8", given=False),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, even over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _width(rng, lo, hi):
    return 64 * _spread(rng, lo // 64, hi // 64)


def draw(rng):
    kind = rng.choice(["rows", "weights", "product", "product", "layer8", "layer8", "few", "few", "few"])
    if kind == "rows":
        rows = _spread(rng, 1, 8192)
        return dict(kind=kind, rows=rows, cols=_width(rng, 64, 2880 if rows > 4096 else 5120),
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
    if kind == "weights":
        return dict(kind=kind, E=_spread(rng, 1, 16), d=_width(rng, 64, 1024), I=_width(rng, 64, 2816),
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
    if kind == "product":
        return dict(kind=kind, rows=_spread(rng, 1, 32768), E=_spread(rng, 1, 16), K=_width(rng, 64, 2880),
                    N=_width(rng, 64, 2880), skew=rng.random() < 0.5)
    if kind == "layer8":
        E = _spread(rng, 2, 128)
        return dict(kind=kind, T=_spread(rng, 1, 8192), d=_width(rng, 64, 2880), E=E, k=rng.randint(1, min(4, E)),
                    I=_width(rng, 64, 2880))
    E = _spread(rng, 2, 128)
    k = rng.randint(1, min(8, E))
    return dict(kind=kind, T=rng.choice([1, 1, _spread(rng, 2, 64)]), d=_width(rng, 64, 2880), E=E, k=k,
                I=_width(rng, 64, 2880), weights=rng.choice(["bf16", "bf16", "f32", "fp8", "fp8"]),
                given=rng.random() < 0.3)


# ---- inputs -------------------------------------------------------------------------

def _blocks(n):
    return -(-n // BLOCK)


def _weights8(shape, scales, g):
    """8-bit weights as a checkpoint holds them: e4m3 codes using most of their range, and float32 scales that are no
    powers of two; the values they stand for are about N(0, 0.02)."""
    q = torch.empty(shape, dtype=F8, device=DEV)
    for e in range(shape[0]):
        q[e] = torch.randn(shape[1:], generator=g, device=DEV).mul_(110.0).clamp_(-448.0, 448.0).to(F8)
    s = torch.rand(scales, generator=g, device=DEV).mul_(0.2).add_(0.9).mul_(0.02 / 110.0)
    return q, s


def _weights(shape, dtype, g):
    w = torch.empty(shape, dtype=dtype, device=DEV)
    for e in range(shape[0]):
        w[e] = torch.randn(shape[1:], generator=g, device=DEV).mul_(0.02).to(dtype)
    return w


def _rows(rows, cols, dtype, g):
    """Activations: N(0, 1), each row with a size of its own, a few columns much larger than the others."""
    x = torch.randn((rows, cols), generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn((rows, 1), generator=g, device=DEV))
    x[:, torch.randint(0, cols, (max(1, cols // 200),), generator=g, device=DEV)] *= 20.0
    return x.to(dtype)


def _quantized_rows(rows, cols, g):
    """8-bit rows as a quantizer leaves them: e4m3 codes up to 448 and a power-of-two scale for each block."""
    q = torch.randn((rows, cols), generator=g, device=DEV).mul_(100.0).clamp_(-448.0, 448.0).to(F8)
    s = torch.exp2(torch.randint(-9, -5, (rows, _blocks(cols)), generator=g, device=DEV).float())
    return q, s


def _counts(case, rng):
    """Rows for each expert: even shares with chance, or shares that fall as rank^-1.1 with every fifth expert empty."""
    E, rows = case["E"], case["rows"]
    if case["skew"]:
        rank = rng.permutation(E) + 1.0
        share = rank ** -1.1
        share[rank > E - E // 5] = 0.0
    else:
        share = np.ones(E)
    return rng.multinomial(rows, share / share.sum()).tolist()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    kind = case["kind"]
    s = dict(case)
    if kind == "rows":
        s["x"] = _rows(case["rows"], case["cols"], TYPES[case["dtype"]], g)
    elif kind == "weights":
        E, d, I = case["E"], case["d"], case["I"]
        s["w_gate_up"] = _weights((E, d, 2 * I), TYPES[case["dtype"]], g)
        s["w_down"] = _weights((E, I, d), TYPES[case["dtype"]], g)
    elif kind == "product":
        E, K, N, rows = case["E"], case["K"], case["N"], case["rows"]
        s["x_q"], s["x_s"] = _quantized_rows(rows, K, g)
        s["w_q"], s["w_s"] = _weights8((E, N, K), (E, _blocks(N), _blocks(K)), g)
        s["counts"] = _counts(case, np.random.default_rng(seed))
        s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(s["counts"])]), dtype=torch.int32, device=DEV)
        s["y"] = torch.empty((rows, N), dtype=torch.bfloat16, device=DEV)
    else:
        T, d, E, k, I = case["T"], case["d"], case["E"], case["k"], case["I"]
        form = case.get("weights", "fp8")
        dtype = torch.float32 if form == "f32" else torch.bfloat16
        s["x"] = _rows(T, d, dtype, g)
        if form == "fp8":
            s["w_gate_up"] = _weights8((E, 2 * I, d), (E, 2, _blocks(I), _blocks(d)), g)
            s["w_down"] = _weights8((E, d, I), (E, _blocks(d), _blocks(I)), g)
        else:
            s["w_gate_up"] = _weights((E, d, 2 * I), dtype, g)
            s["w_down"] = _weights((E, I, d), dtype, g)
        logits = torch.randn((T, E), generator=g, device=DEV)
        if case.get("given"):
            # pairs routed elsewhere, one in ten of them another rank's (-1)
            s["logits"] = None
            s["idx"] = torch.topk(logits, k).indices.to(torch.int32)
            s["idx"][torch.rand((T, k), generator=g, device=DEV) < 0.1] = -1
            s["w"] = 1.0 - torch.rand((T, k), generator=g, device=DEV)
        else:
            s["logits"] = logits
            s["idx"] = torch.empty((T, k), dtype=torch.int32, device=DEV)
            s["w"] = torch.empty((T, k), dtype=torch.float32, device=DEV)
        s["out"] = torch.empty((T, d), dtype=dtype, device=DEV)
    return s


# ---- the framework's calls --------------------------------------------------------------

def _workspace(s, size, *sizes):
    """The workspace that a program keeps between calls, as large as `size` says for these sizes."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(size(*sizes), dtype=torch.uint8, device=DEV)
    return s["workspace"]


def _run_own(s):
    import token_routing_expert_amd as tre
    kind = s["kind"]
    if kind == "rows":
        return tre.moe_quantize_rows(s["x"])
    if kind == "weights":
        return tre.moe_quantize_weights(s["w_gate_up"], s["w_down"])
    if kind == "product":
        return tre.moe_down_proj_fp8(s["x_q"], s["x_s"], s["offsets"], s["w_q"], s["w_s"], y_perm=s["y"])
    T, d, E, k, I = (s[n] for n in ("T", "d", "E", "k", "I"))
    if kind == "layer8":
        ws = _workspace(s, tre.moe_forward_fp8_workspace_size, T, d, E, k, I)
        return tre.moe_forward_fp8(s["x"], *s["w_gate_up"], *s["w_down"], k, logits=s["logits"], topk_idx=s["idx"],
                                   topk_w=s["w"], out=s["out"], workspace=ws)
    if s["weights"] == "fp8":
        ws = _workspace(s, tre.moe_forward_few_fp8_workspace_size, T, d, E, k, I)
        return tre.moe_forward_few_fp8(s["x"], *s["w_gate_up"], *s["w_down"], k, logits=s["logits"],
                                       topk_idx=s["idx"], topk_w=s["w"], out=s["out"], workspace=ws)
    dt = tre.MOE_F32 if s["weights"] == "f32" else tre.MOE_BF16
    ws = _workspace(s, tre.moe_forward_few_workspace_size, T, d, E, k, I, dt)
    return tre.moe_forward_few(s["x"], s["w_gate_up"], s["w_down"], k, logits=s["logits"], topk_idx=s["idx"],
                               topk_w=s["w"], out=s["out"], workspace=ws)


# ---- the plain forms ------------------------------------------------------------------------

def _power_scale(amax):
    """The smallest power of two, 2^-126 at least, that brings amax to 448 or less; NaN where amax is not finite."""
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126)
    return torch.where(torch.isfinite(amax), torch.ldexp(torch.ones_like(amax), e), math.nan)


def _quantize(x, real=torch.float32):
    """Codes and scales of the last dimension's blocks of 128."""
    cols = x.shape[-1]
    nb = _blocks(cols)
    x = torch.nn.functional.pad(x.to(real), (0, nb * BLOCK - cols)).unflatten(-1, (nb, BLOCK))
    s = _power_scale(x.abs().amax(-1))
    q = (x / s[..., None]).flatten(-2)[..., :cols].to(torch.float32).to(F8)
    return q, s.to(torch.float32)


def _quantize_weight(w):
    """Codes and scales of the blocks of 128 x 128 of the last two dimensions."""
    n, k = w.shape[-2:]
    nb, kb = _blocks(n), _blocks(k)
    x = torch.nn.functional.pad(w.float(), (0, kb * BLOCK - k, 0, nb * BLOCK - n))
    x = x.unflatten(-1, (kb, BLOCK)).unflatten(-3, (nb, BLOCK))
    s = _power_scale(x.abs().amax((-3, -1)))
    q = (x / s[..., :, None, :, None]).flatten(-4, -3).flatten(-2)[..., :n, :k].to(F8)
    return q, s


def _spell(scales, n, dim):
    """A scale for each element from a scale for each block, along dim."""
    return scales.repeat_interleave(BLOCK, dim).narrow(dim, 0, n)


def _values(q, s):
    """The rows that codes and scales stand for."""
    return q.float() * _spell(s, q.shape[-1], -1)


def _weight_values(q, s):
    """The [N, K] weights that codes and scales stand for; packed gate/up weights have their halves' scales apart."""
    if s.dim() == q.dim() + 1:
        return torch.cat([_weight_values(h, t) for h, t in zip(q.chunk(2, -2), s.unbind(-3))], -2)
    return q.float() * _spell(_spell(s, q.shape[-2], -2), q.shape[-1], -1)


def _route(s):
    """Selected experts and weights: the k largest logits, equal ones by the lower index."""
    if s["logits"] is None:
        return s["idx"], s["w"]
    top, idx = torch.sort(s["logits"], dim=-1, descending=True, stable=True)
    top, idx = top[:, :s["k"]], idx[:, :s["k"]]
    p = torch.exp(top - top[:, :1])
    return idx.to(torch.int32), p / p.sum(-1, keepdim=True)


def _swiglu(gu):
    g, u = gu.chunk(2, -1)
    return g / (1.0 + torch.exp(-g)) * u


def _plain_product(s):
    # the groups are ragged: one product for each expert that has rows
    parts = [x @ _weight_values(s["w_q"][e], s["w_s"][e]).t()
             for e, x in enumerate(torch.split(_values(s["x_q"], s["x_s"]), s["counts"])) if x.shape[0]]
    return torch.cat(parts).to(torch.bfloat16)


def _plain_layer8(s):
    E, k = s["E"], s["k"]
    idx, w = _route(s)
    x = _values(*_quantize(s["x"]))
    flat = idx.flatten()
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=E).tolist()
    y = torch.empty((flat.shape[0], s["d"]), dtype=torch.float32, device=DEV)
    for e, pairs in enumerate(torch.split(order, counts)):   # ragged groups, as in the product
        if pairs.shape[0]:
            h = _swiglu(x[pairs // k] @ _weight_values(s["w_gate_up"][0][e], s["w_gate_up"][1][e]).t())
            y[pairs] = _values(*_quantize(h)) @ _weight_values(s["w_down"][0][e], s["w_down"][1][e]).t()
    out = (y.unflatten(0, (-1, k)) * w[:, :, None]).sum(1)
    return out.to(torch.bfloat16), idx, w


def _plain_few(s):
    T, E, k = s["T"], s["E"], s["k"]
    idx, w = _route(s)
    x = s["x"].float()
    live = torch.where(idx >= 0, w, 0.0)
    gather = T * k < E

    def matrices(name):
        """The pairs' own weights where they are fewer than the experts, or every expert's, as [.., K, N]."""
        pick = idx.clamp(min=0).flatten().long()
        if s["weights"] == "fp8":
            q, sc = s[name]
            return _weight_values(q[pick], sc[pick]).mT if gather else _weight_values(q, sc).mT
        return s[name][pick].float() if gather else s[name].float()

    if gather:
        h = _swiglu(torch.bmm(x.repeat_interleave(k, 0)[:, None], matrices("w_gate_up").contiguous()))
        y = torch.bmm(h, matrices("w_down").contiguous())[:, 0]
        out = (y.unflatten(0, (T, k)) * live[:, :, None]).sum(1)
    else:
        h = _swiglu(torch.bmm(x.expand(E, -1, -1).contiguous(), matrices("w_gate_up").contiguous()))
        y = torch.bmm(h, matrices("w_down").contiguous())
        share = torch.zeros((T, E), device=DEV).scatter_add_(1, idx.clamp(min=0).long(), live)
        out = (y * share.t()[:, :, None]).sum(0)
    return out.to(s["x"].dtype), idx, w


def _run_plain(s):
    kind = s["kind"]
    if kind == "rows":
        return _quantize(s["x"])
    if kind == "weights":
        gate, up = s["w_gate_up"].mT.chunk(2, -2)
        (gq, gs), (uq, us) = _quantize_weight(gate), _quantize_weight(up)
        return (torch.cat([gq, uq], 1), torch.stack([gs, us], 1), *_quantize_weight(s["w_down"].mT))
    if kind == "product":
        return _plain_product(s)
    return _plain_layer8(s) if kind == "layer8" else _plain_few(s)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- the work of one pass -------------------------------------------------------------------

def _live_experts(E, draws):
    """Experts with at least one row, on average, of `draws` rows over equal experts."""
    return E * (1.0 - (1.0 - 1.0 / E) ** draws)


def work(case):
    kind = case["kind"]
    size = {"bf16": 2, "f32": 4, "fp8": 1}
    if kind == "rows":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (size[case["dtype"]] + 1) + 4 * case["rows"] * _blocks(case["cols"]), "flops": 2 * n}
    if kind == "weights":
        n = 3 * case["E"] * case["d"] * case["I"]
        return {"bytes": n * (size[case["dtype"]] + 1) + 4 * n // BLOCK ** 2, "flops": 2 * n}
    if kind == "product":
        E, K, N, rows = case["E"], case["K"], case["N"], case["rows"]
        live = _live_experts(E - E // 5 if case["skew"] else E, rows)
        return {"bytes": live * N * K + rows * (K + 4 * _blocks(K) + 2 * N), "flops": 2 * rows * K * N}
    T, d, E, k, I = (case[n] for n in ("T", "d", "E", "k", "I"))
    form = case.get("weights", "fp8")
    live = E * (1.0 - (1.0 - k / E) ** T)
    rows = T * k
    if case.get("given"):
        rows *= 0.9
        live = E * (1.0 - (1.0 - 0.9 * k / E) ** T)
    bytes_ = 3 * live * d * I * size[form] + 2 * T * d * (4 if form == "f32" else 2) + 8 * T * k
    return {"bytes": bytes_ + (0 if case.get("given") else 4 * T * E), "flops": 6 * rows * d * I}


# ---- the definitions in 64 bits ---------------------------------------------------------------

_CODES = np.array([(-1.0 if c & 128 else 1.0) * (math.nan if c & 127 == 127 else (c & 7) * 2.0 ** -9 if c & 120 == 0
                   else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3 & 15) - 7)) for c in range(256)])


def _codes64(q):
    """e4m3 codes by their bits: sign, four bits of exponent with bias 7, three of mantissa, no infinities."""
    return torch.from_numpy(_CODES).to(DEV)[q.view(torch.uint8).long()]


def _round_e4m3(v):
    """The nearest e4m3 value of |v| <= 448, ties to the even code: steps of 2^(e-3) in [2^e, 2^(e+1)), 2^-9 below 2^-6."""
    _, e = torch.frexp(v.abs())
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return torch.round(v / step) * step


def _rows64(x):
    """(values before the scale, scales) of rows in 64 bits."""
    cols = x.shape[1]
    v, sc = torch.empty_like(x), torch.empty((x.shape[0], _blocks(cols)), dtype=torch.float64, device=DEV)
    for b in range(_blocks(cols)):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        top = part.abs().max(1, keepdim=True).values
        power = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448.0)).clamp(min=-126)
        # log2 may be off by a step next to a power of two
        power = torch.where(torch.exp2(power) * 448.0 < top, power + 1, power)
        power = torch.where((torch.exp2(power - 1) * 448.0 >= top) & (power > -126), power - 1, power)
        v[:, b * BLOCK:(b + 1) * BLOCK] = _round_e4m3(part / torch.exp2(power))
        sc[:, b] = torch.exp2(power)[:, 0]
    return v, sc


def _weights64(w, kind):
    """The [K, N] matrix of one expert in 64 bits; 8-bit ones come as (codes, scales)."""
    if kind != "fp8":
        return w.double()
    q, s = w
    v = _codes64(q)
    halves = s if s.dim() == 3 else s[None]
    n = v.shape[0] // halves.shape[0]
    for i in range(halves.shape[0]):
        for b in range(halves.shape[1]):
            rows = v[i * n + b * BLOCK:min(i * n + (b + 1) * BLOCK, (i + 1) * n)]
            for c in range(halves.shape[2]):
                rows[:, c * BLOCK:(c + 1) * BLOCK] *= halves[i, b, c].double()
    return v.t()


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "rows":
        return _rows64(s["x"].double())
    if kind == "weights":
        E, d, I = case["E"], case["d"], case["I"]

        def blocks64(w, n, k):   # w [K, N] of one expert -> codes' values [N, K], scales
            v, sc = torch.empty((n, k), dtype=torch.float64, device=DEV), []
            for a in range(0, n, BLOCK):
                strip = w[:, a:a + BLOCK].double().t()
                for b in range(0, k, BLOCK):
                    part = strip[:, b:b + BLOCK]
                    top = float(part.abs().max())
                    p = max(-126, math.ceil(math.log2(max(top, 1e-300) / 448.0)))
                    p += 2.0 ** p * 448.0 < top
                    p -= 2.0 ** (p - 1) * 448.0 >= top and p > -126
                    v[a:a + BLOCK, b:b + BLOCK] = _round_e4m3(part / 2.0 ** p)
                    sc.append(2.0 ** p)
            return v, torch.tensor(sc, dtype=torch.float64, device=DEV).reshape(_blocks(n), _blocks(k))

        gu = [[blocks64(s["w_gate_up"][e][:, h * I:(h + 1) * I], I, d) for h in (0, 1)] for e in range(E)]
        dn = [blocks64(s["w_down"][e], d, I) for e in range(E)]
        return (torch.stack([torch.cat([v for v, _ in p]) for p in gu]),
                torch.stack([torch.stack([sc for _, sc in p]) for p in gu]),
                torch.stack([v for v, _ in dn]), torch.stack([sc for _, sc in dn]))
    if kind == "product":
        x, y, at = _codes64(s["x_q"]), [], 0
        for b in range(_blocks(case["K"])):
            x[:, b * BLOCK:(b + 1) * BLOCK] *= s["x_s"][:, b:b + 1].double()
        for e, n in enumerate(s["counts"]):
            if n:
                y.append(x[at:at + n] @ _weights64((s["w_q"][e], s["w_s"][e]), "fp8"))
                at += n
        return torch.cat(y)
    form = case.get("weights", "fp8")
    T, k = case["T"], case["k"]
    if s["logits"] is None:
        idx, w = s["idx"].cpu().numpy(), s["w"].cpu().numpy().astype(np.float64)
    else:
        lg = s["logits"].cpu().numpy().astype(np.float64)
        idx = np.argsort(-lg, axis=1, kind="stable")[:, :k]
        w = np.exp(np.take_along_axis(lg, idx, 1))
        w /= w.sum(1, keepdims=True)
    x = s["x"].double()
    if kind == "layer8":
        v, sc = _rows64(x)
        for b in range(sc.shape[1]):
            v[:, b * BLOCK:(b + 1) * BLOCK] *= sc[:, b:b + 1]
        x = v
    out = torch.zeros((T, case["d"]), dtype=torch.float64, device=DEV)
    for e in range(case["E"]):
        t, j = np.nonzero(idx == e)
        if not len(t):
            continue
        wgu = (s["w_gate_up"][0][e], s["w_gate_up"][1][e]) if form == "fp8" else s["w_gate_up"][e]
        wd = (s["w_down"][0][e], s["w_down"][1][e]) if form == "fp8" else s["w_down"][e]
        gu = x[torch.from_numpy(t).to(DEV)] @ _weights64(wgu, form)
        g, u = gu[:, :case["I"]], gu[:, case["I"]:]
        h = g * torch.sigmoid(g) * u
        if kind == "layer8":
            v, sc = _rows64(h)
            for b in range(sc.shape[1]):
                v[:, b * BLOCK:(b + 1) * BLOCK] *= sc[:, b:b + 1]
            h = v
        y = (h @ _weights64(wd, form)) * torch.from_numpy(w[t, j]).to(DEV)[:, None]
        out.index_add_(0, torch.from_numpy(t).to(DEV), y)
    return out, None, torch.from_numpy(w)
