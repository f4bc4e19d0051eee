"""The expert feed-forward's gradients and its 8-bit activation checkpoints as measured work: their plain forms in
elementary torch operations, the framework's calls, and the definition in 64 bits.

Kinds of cases:
  block    moe_grouped_ffn_backward: gradients of the grouped gated feed-forward, gate and up computed again
  step8    moe_grouped_ffn_train + moe_grouped_ffn_backward: a training step of the same rows, with the
           pre-activations kept in 8 bits between the two
  keep8    moe_forward_train_q8: the layer's forward that keeps the 8-bit checkpoint, and moe_checkpoint_values,
           which reads it back
  grad8    moe_backward_q8: the layer's gradients from such a checkpoint

`own` selects the framework's calls; the plain forms need torch only.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 64          # columns that share a scale in a checkpoint
FLOOR = 2.0 ** -100  # the least magnitude that a scale stands for
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ------------------------------------------------------------------------

def listed():
    return [
        # a tiny float32 layer's experts: launches are all that counts
        dict(name="block_tiny_f32", kind="block", rows=128, E=8, d=128, I=256, dtype="f32", skew=False),
        # a prompt batch's rows at a 16-expert layer
        dict(name="block_small", kind="block", rows=8192, E=16, d=1024, I=2816, dtype="bf16", skew=False),
        # the rows one expert-parallel rank received, skewed, three experts without rows
        dict(name="block_rank", kind="block", rows=32768, E=16, d=2880, I=2880, dtype="bf16", skew=True),
        # a short batch, ragged: some experts have a few rows, some hundreds
        dict(name="step8_odd", kind="step8", rows=1537, E=16, d=1024, I=2816, dtype="bf16", skew=True),
        # a training step's rows at a 16-expert layer
        dict(name="step8_small", kind="step8", rows=8192, E=16, d=1024, I=2816, dtype="bf16", skew=False),
        # a training step of one expert-parallel rank's rows
        dict(name="step8_rank", kind="step8", rows=32768, E=16, d=2880, I=2880, dtype="bf16", skew=True),
        # the forward of a tiny float32 layer
        dict(name="keep8_tiny_f32", kind="keep8", T=64, d=128, E=8, k=2, I=256, dtype="f32", given=False),
        # the forward of a 16-expert layer on a batch
        dict(name="keep8_small", kind="keep8", T=4096, d=1024, E=16, k=2, I=2816, dtype="bf16", given=False),
        # the forward of a 128-expert layer
        dict(name="keep8_large", kind="keep8", T=8192, d=2880, E=128, k=4, I=2880, dtype="bf16", given=False),
        # the gradients of the tiny float32 layer
        dict(name="grad8_tiny_f32", kind="grad8", T=64, d=128, E=8, k=2, I=256, dtype="f32", given=False),
        # the gradients of a 16-expert layer, pairs routed elsewhere, a tenth of them another rank's
        dict(name="grad8_small", kind="grad8", T=4095, d=1024, E=16, k=2, I=2816, dtype="bf16", given=True),
        # the gradients of a 128-expert layer
        dict(name="grad8_large", kind="grad8", T=8192, d=2880, E=128, k=4, I=2880, dtype="bf16", given=False),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, even over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _width(rng, lo, hi):
    return 64 * _spread(rng, lo // 64, hi // 64)


def draw(rng):
    kind = rng.choice(["block", "step8", "keep8", "grad8"])
    # (float32 gradients behind an 8-bit rounding are no float32 results: step8 is drawn in bf16 only)
    dtype = "bf16" if kind == "step8" else rng.choice(["bf16", "bf16", "f32"])
    widths = (64, 1024) if dtype == "f32" else (64, 2880)
    d, I = _width(rng, *widths), _width(rng, *widths)
    if kind in ("block", "step8"):
        return dict(kind=kind, rows=_spread(rng, 1, 4096 if dtype == "f32" else 32768), E=_spread(rng, 1, 16), d=d,
                    I=I, dtype=dtype, skew=rng.random() < 0.5)
    E = _spread(rng, 2, 128)
    return dict(kind=kind, T=_spread(rng, 1, 2048 if dtype == "f32" else 8192), d=d, E=E, k=rng.randint(1, min(4, E)),
                I=I, dtype=dtype, given=rng.random() < 0.3)


# ---- inputs -------------------------------------------------------------------------

def _weights(shape, dtype, g):
    w = torch.empty(shape, dtype=dtype, device=DEV)
    for e in range(shape[0]):
        w[e] = torch.randn(shape[1:], generator=g, device=DEV).mul_(0.02).to(dtype)
    return w


def _rows(rows, cols, dtype, g):
    """Activations: N(0, 1), each row with a size of its own, a few columns larger than the others."""
    x = torch.randn((rows, cols), generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn((rows, 1), generator=g, device=DEV))
    x[:, torch.randint(0, cols, (max(1, cols // 200),), generator=g, device=DEV)] *= 5.0
    return x.to(dtype)


def _grad(rows, cols, dtype, g):
    """What reaches a block from the loss: small, each row with a size of its own."""
    x = torch.randn((rows, cols), generator=g, device=DEV)
    x *= 1e-3 * torch.exp(0.5 * torch.randn((rows, 1), generator=g, device=DEV))
    return x.to(dtype)


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


def _group(idx, k, E):
    """Pairs grouped by expert, in order: (row_token, pair_row, expert_offsets), as int32; -1 for pairs of no expert."""
    flat = idx.flatten().long()
    order = torch.argsort(torch.where(flat >= 0, flat, E), stable=True)
    row_of = torch.empty_like(order)
    row_of[order] = torch.arange(order.shape[0], device=DEV)
    counts = torch.bincount(flat[flat >= 0], minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return ((order // k).to(torch.int32), torch.where(flat >= 0, row_of, -1).to(torch.int32),
            offsets.to(torch.int32), counts.tolist())


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    kind, E, d, I, dtype = case["kind"], case["E"], case["d"], case["I"], TYPES[case["dtype"]]
    s = dict(case)
    s["w_gate_up"] = _weights((E, d, 2 * I), dtype, g)
    s["w_down"] = _weights((E, I, d), dtype, g)
    if kind in ("block", "step8"):
        s["counts"] = _counts(case, np.random.default_rng(seed))
        s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(s["counts"])]), dtype=torch.int32, device=DEV)
        s["x"] = _rows(case["rows"], d, dtype, g)
        s["dy"] = _grad(case["rows"], d, dtype, g)
        return s
    T, k = case["T"], case["k"]
    s["x"] = _rows(T, d, dtype, g)
    s["logits"] = torch.randn((T, E), generator=g, device=DEV)
    if kind == "keep8" and not case["given"]:
        return s
    s["idx"] = torch.topk(s["logits"], k).indices.to(torch.int32)
    s["w"] = torch.softmax(torch.gather(s["logits"], 1, s["idx"].long()), -1)
    s["logits"] = None
    if kind == "keep8":
        return s
    if case["given"]:
        s["idx"][torch.rand((T, k), generator=g, device=DEV) < 0.1] = -1
        s["w"] = 1.0 - torch.rand((T, k), generator=g, device=DEV)
    s["dout"] = _grad(T, d, dtype, g)
    s["row_token"], s["pair_row"], s["offsets"], s["counts"] = _group(s["idx"], k, E)
    # the checkpoint that a forward left: gate and up N(0, 1.5), each row with a size of its own
    s["gu_q"] = torch.empty((T * k, 2 * I), dtype=torch.int8, device=DEV)
    s["gu_s"] = torch.empty((T * k, 2, I // BLOCK), dtype=torch.float32, device=DEV)
    for a in range(0, T * k, 4096):
        gu = torch.randn((min(4096, T * k - a), 2 * I // BLOCK, BLOCK), generator=g, device=DEV).mul_(1.5)
        gu *= torch.exp(0.3 * torch.randn((gu.shape[0], 1, 1), generator=g, device=DEV))
        sc = gu.abs().amax(-1) / 127.0
        s["gu_q"][a:a + 4096] = torch.round(gu / sc[..., None]).flatten(1).to(torch.int8)
        s["gu_s"][a:a + 4096] = sc.unflatten(1, (2, I // BLOCK))
    return s


# ---- the framework's calls --------------------------------------------------------------

def _workspace(s, name, size, *sizes):
    """The workspace that a program keeps between calls, as large as `size` says for these sizes."""
    if name not in s:
        s[name] = torch.empty(size(*sizes), dtype=torch.uint8, device=DEV)
    return s[name]


def _run_own(s):
    import token_routing_expert_amd as tre
    kind, E, d, I = s["kind"], s["E"], s["d"], s["I"]
    dt = tre.MOE_F32 if s["dtype"] == "f32" else tre.MOE_BF16
    if kind in ("block", "step8"):
        R = s["rows"]
        bws = _workspace(s, "backward_ws", tre.moe_grouped_ffn_backward_workspace_size, R, E, d, I, dt)
        if kind == "block":
            return tre.moe_grouped_ffn_backward(s["x"], s["offsets"], s["w_gate_up"], s["w_down"], s["dy"],
                                                workspace=bws)
        fws = _workspace(s, "forward_ws", tre.moe_grouped_ffn_train_workspace_size, R, E, d, I, dt)
        y, gu_q, gu_s = tre.moe_grouped_ffn_train(s["x"], s["offsets"], s["w_gate_up"], s["w_down"], workspace=fws)
        return (y, *tre.moe_grouped_ffn_backward(s["x"], s["offsets"], s["w_gate_up"], s["w_down"], s["dy"],
                                                 gu_q=gu_q, gu_s=gu_s, workspace=bws))
    T, k = s["T"], s["k"]
    if kind == "keep8":
        ws = _workspace(s, "forward_ws", tre.moe_forward_train_q8_workspace_size, T, d, E, k, I, dt)
        out, idx, w, kept = tre.moe_forward_train_q8(s["x"], s["w_gate_up"], s["w_down"], k, logits=s["logits"],
                                                     topk_idx=s.get("idx"), topk_w=s.get("w"), workspace=ws)
        return out, idx, w, kept.expert_offsets, tre.moe_checkpoint_values(kept.gu_q, kept.gu_s, torch.bfloat16)
    kept = tre.Checkpoint(s["offsets"], s["row_token"], s["pair_row"], s["gu_q"], s["gu_s"])
    ws = _workspace(s, "backward_ws", tre.moe_backward_q8_workspace_size, T, d, E, k, I, dt)
    r = tre.moe_backward_q8(s["x"], s["w_gate_up"], s["w_down"], k, s["dout"], s["idx"], s["w"], kept,
                            want_dlogits=not s["given"], workspace=ws)
    return {n: r[n] for n in ("dx", "dw_gate_up", "dw_down", "dtopk_w", "dlogits") if n in r}


# ---- the plain forms ------------------------------------------------------------------------

def _route(s):
    """Selected experts and weights: the k largest logits, equal ones by the lower index."""
    if s["logits"] is None:
        return s["idx"], s["w"]
    top, idx = torch.sort(s["logits"], dim=-1, descending=True, stable=True)
    top, idx = top[:, :s["k"]], idx[:, :s["k"]]
    p = torch.exp(top - top[:, :1])
    return idx.to(torch.int32), p / p.sum(-1, keepdim=True)


def _kept(gu):
    """The values that an 8-bit checkpoint of gu stands for: whole multiples of a block's largest magnitude / 127."""
    b = gu.unflatten(-1, (-1, BLOCK))
    sc = b.abs().amax(-1, keepdim=True).clamp(min=FLOOR) / 127.0
    return (torch.round(b / sc) * sc).flatten(-2)


def _forward_block(s, x, e):
    """(gate | up of expert e's rows x, their output), in float32."""
    gu = x @ s["w_gate_up"][e].float()
    g, u = gu.chunk(2, -1)
    return gu, (g / (1.0 + torch.exp(-g)) * u) @ s["w_down"][e].float()


def _backward_block(s, x, gu, dy, w, e):
    """Gradients of expert e on its rows: (dx, dw_gate_up, dw_down, <dy, y>), for dy times the rows' weights w."""
    g, u = gu.chunk(2, -1)
    sg = 1.0 / (1.0 + torch.exp(-g))
    h = g * sg * u
    dh = dy @ s["w_down"][e].float().t()
    dot = (dh * h).sum(-1)
    dh, dy = (dh, dy) if w is None else (dh * w[:, None], dy * w[:, None])
    dgu = torch.cat([dh * u * sg * (1.0 + g * (1.0 - sg)), dh * g * sg], -1)
    return dgu @ s["w_gate_up"][e].float().t(), x.t() @ dgu, h.t() @ dy, dot


def _plain_block(s):
    dx = torch.empty_like(s["x"])
    y, dwgu, dwd = torch.empty_like(s["x"]), torch.zeros_like(s["w_gate_up"]), torch.zeros_like(s["w_down"])
    at = 0
    for e, n in enumerate(s["counts"]):   # the groups are ragged: products for each expert that has rows
        if n:
            rows = slice(at, at + n)
            x, dy = s["x"][rows].float(), s["dy"][rows].float()
            if s["kind"] == "block":
                gu = x @ s["w_gate_up"][e].float()
            else:
                gu, out = _forward_block(s, x, e)
                y[rows] = out.to(y.dtype)
                gu = _kept(gu)
            a, b, c, _ = _backward_block(s, x, gu, dy, None, e)
            dx[rows], dwgu[e], dwd[e] = a.to(dx.dtype), b.to(dx.dtype), c.to(dx.dtype)
            at += n
    return (dx, dwgu, dwd) if s["kind"] == "block" else (y, dx, dwgu, dwd)


def _plain_keep(s):
    k, E = s["k"], s["E"]
    idx, w = _route(s)
    row_token, pair_row, offsets, counts = _group(idx, k, E)
    x = s["x"].float()
    y = torch.empty((row_token.shape[0], s["d"]), dtype=torch.float32, device=DEV)
    gu = torch.empty((row_token.shape[0], 2 * s["I"]), dtype=torch.bfloat16, device=DEV)
    at = 0
    for e, n in enumerate(counts):   # ragged groups, as in the block
        if n:
            a, y[at:at + n] = _forward_block(s, x[row_token[at:at + n].long()], e)
            gu[at:at + n] = _kept(a).to(gu.dtype)
            at += n
    out = (y[pair_row.long()].unflatten(0, (-1, k)) * w[:, :, None]).sum(1)
    return out.to(s["x"].dtype), idx, w, offsets, gu


def _plain_grad(s):
    T, k, dtype = s["T"], s["k"], s["x"].dtype
    x, dout = s["x"].float(), s["dout"].float()
    live = s["pair_row"] >= 0
    row = s["pair_row"].clamp(min=0).long()
    row_w = torch.zeros(T * k, device=DEV)
    row_w[row[live]] = s["w"].flatten()[live]
    dxp = torch.zeros((T * k, s["d"]), device=DEV)
    dot = torch.zeros(T * k, device=DEV)
    dwgu, dwd = torch.zeros_like(s["w_gate_up"]), torch.zeros_like(s["w_down"])
    at = 0
    for e, n in enumerate(s["counts"]):   # ragged groups, as in the block
        if n:
            rows, tok = slice(at, at + n), s["row_token"][at:at + n].long()
            gu = (s["gu_q"][rows].float().unflatten(-1, (-1, BLOCK)) * s["gu_s"][rows].flatten(1)[..., None]).flatten(1)
            dxp[rows], b, c, dot[rows] = _backward_block(s, x[tok], gu, dout[tok], row_w[rows], e)
            dwgu[e], dwd[e] = b.to(dtype), c.to(dtype)
            at += n
    dx = torch.where(live[:, None], dxp[row], 0.0).unflatten(0, (T, k)).sum(1)
    dw = torch.where(live, dot[row], 0.0).unflatten(0, (T, k))
    r = dict(dx=dx.to(dtype), dw_gate_up=dwgu, dw_down=dwd, dtopk_w=dw)
    if not s["given"]:
        inner = (s["w"] * dw).sum(-1, keepdim=True)
        r["dlogits"] = torch.zeros((T, s["E"]), device=DEV).scatter_(1, s["idx"].long(), s["w"] * (dw - inner))
    return r


def run(state):
    if own:
        return _run_own(state)
    if state["kind"] == "keep8":
        return _plain_keep(state)
    return _plain_grad(state) if state["kind"] == "grad8" else _plain_block(state)


# ---- the work of one pass -------------------------------------------------------------------

def _live_experts(E, draws):
    """Experts with at least one row, on average, of `draws` rows over equal experts."""
    return E * (1.0 - (1.0 - 1.0 / E) ** draws)


def work(case):
    kind, E, d, I = case["kind"], case["E"], case["d"], case["I"]
    size = 4 if case["dtype"] == "f32" else 2
    kept = 2 * I + 4 * 2 * I // BLOCK   # bytes of a row's checkpoint
    if kind in ("block", "step8"):
        rows = case["rows"]
        live = _live_experts(E - E // 5 if case["skew"] else E, rows)
        # weights once, their gradients once (of experts without rows too), x and dy in, dx (and y) out
        n = 3 * d * I * size * (live + E) + rows * d * size * (3 if kind == "block" else 4)
        return {"bytes": n + (0 if kind == "block" else 2 * rows * kept),
                "flops": (16 if kind == "block" else 18) * rows * d * I}
    T, k = case["T"], case["k"]
    live = E * (1.0 - (1.0 - k / E) ** T)
    if kind == "keep8":
        # the checkpoint is written, read back and returned as bf16 values
        return {"bytes": 3 * d * I * size * live + 2 * T * d * size + 4 * T * (2 * k if case["given"] else E + 2 * k) +
                T * k * (2 * kept + 4 * I), "flops": 6 * T * k * d * I}
    rows = T * k * (0.9 if case["given"] else 1.0)
    return {"bytes": 3 * d * I * size * (live + E) + 3 * T * d * size + rows * kept + 24 * T * k +
            (0 if case["given"] else 4 * T * E), "flops": 12 * rows * d * I}


# ---- the definitions in 64 bits ---------------------------------------------------------------

def _kept64(v):
    """A checkpoint's values of v, block by block."""
    out = torch.empty_like(v)
    for c in range(0, v.shape[1], BLOCK):
        part = v[:, c:c + BLOCK]
        step = torch.clamp(part.abs().max(1, keepdim=True).values, min=FLOOR) / 127.0
        out[:, c:c + BLOCK] = step * torch.round(part / step)
    return out


def _silu64(g):
    """silu(g) and its derivative."""
    p = torch.sigmoid(g)
    return g * p, p + g * p * (1.0 - p)


def exact(case, seed):
    s = prepare(case, seed)
    kind, E, d, I = case["kind"], case["E"], case["d"], case["I"]
    F = torch.float64

    def matrices(e):
        w = s["w_gate_up"][e].to(F)
        return w[:, :I], w[:, I:], s["w_down"][e].to(F)

    if kind in ("block", "step8"):
        R = case["rows"]
        y = torch.zeros((R, d), dtype=F, device=DEV)
        dx = torch.zeros_like(y)
        dwgu, dwd = torch.zeros((E, d, 2 * I), dtype=F, device=DEV), torch.zeros((E, I, d), dtype=F, device=DEV)
        ends = np.cumsum(s["counts"])
        for e in np.nonzero(s["counts"])[0]:
            lo, hi = ends[e] - s["counts"][e], ends[e]
            wg, wu, wd = matrices(e)
            x, dy = s["x"][lo:hi].to(F), s["dy"][lo:hi].to(F)
            g, u = x @ wg, x @ wu
            y[lo:hi] = (_silu64(g)[0] * u) @ wd
            if kind == "step8":
                g, u = _kept64(g), _kept64(u)
            f, df = _silu64(g)
            dh = dy @ wd.T
            dg, du = dh * u * df, dh * f
            dx[lo:hi] = dg @ wg.T + du @ wu.T
            dwgu[e, :, :I], dwgu[e, :, I:], dwd[e] = x.T @ dg, x.T @ du, (f * u).T @ dy
        return (dx, dwgu, dwd) if kind == "block" else (y, dx, dwgu, dwd)

    T, k = case["T"], case["k"]
    x = s["x"].to(F)
    if kind == "keep8":
        if s["logits"] is None:
            idx, w = s["idx"].cpu().numpy(), s["w"].to(F)
        else:
            lg = s["logits"].cpu().numpy().astype(np.float64)
            idx = np.argsort(-lg, axis=1, kind="stable")[:, :k]
            w = np.exp(np.take_along_axis(lg, idx, 1))
            w = torch.from_numpy(w / w.sum(1, keepdims=True)).to(DEV)
        out = torch.zeros((T, d), dtype=F, device=DEV)
        gu = []
        for e in range(E):
            t, j = (torch.from_numpy(v).to(DEV) for v in np.nonzero(idx == e))
            if t.shape[0]:
                wg, wu, wd = matrices(e)
                g, u = x[t] @ wg, x[t] @ wu
                out.index_add_(0, t, (_silu64(g)[0] * u) @ wd * w[t, j][:, None])
                gu.append(torch.cat([_kept64(g), _kept64(u)], 1))
        return out, None, w, None, torch.cat(gu)

    idx, w, dout = s["idx"].cpu().numpy(), s["w"].to(F), s["dout"].to(F)
    dx, dw = torch.zeros((T, d), dtype=F, device=DEV), torch.zeros((T, k), dtype=F, device=DEV)
    dwgu, dwd = torch.zeros((E, d, 2 * I), dtype=F, device=DEV), torch.zeros((E, I, d), dtype=F, device=DEV)
    for e in range(E):
        t, j = (torch.from_numpy(v).to(DEV) for v in np.nonzero(idx == e))
        if not t.shape[0]:
            continue
        r = s["pair_row"].view(T, k)[t, j].long()
        values = s["gu_q"][r].to(F) * s["gu_s"][r].to(F).reshape(r.shape[0], -1).repeat_interleave(BLOCK, 1)
        g, u = values[:, :I], values[:, I:]
        wg, wu, wd = matrices(e)
        f, df = _silu64(g)
        y = (f * u) @ wd
        dw[t, j] = (y * dout[t]).sum(1)
        dy = dout[t] * w[t, j][:, None]
        dh = dy @ wd.T
        dg, du = dh * u * df, dh * f
        dx.index_add_(0, t, dg @ wg.T + du @ wu.T)
        dwgu[e, :, :I], dwgu[e, :, I:], dwd[e] = x[t].T @ dg, x[t].T @ du, (f * u).T @ dy
    res = dict(dx=dx, dw_gate_up=dwgu, dw_down=dwd, dtopk_w=dw)
    if not case["given"]:
        dl = torch.zeros((T, E), dtype=F, device=DEV)
        mean = (w * dw).sum(1)
        for j in range(k):
            dl[torch.arange(T, device=DEV), s["idx"][:, j].long()] = w[:, j] * (dw[:, j] - mean)
        res["dlogits"] = dl
    return res
