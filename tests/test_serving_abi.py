"""include/moe_serving.h: every declared function is exported (by both builds),
and the host-side checks refuse bad arguments before anything is enqueued.
No kernel is launched: every call fails a check or has nothing to do."""
import ctypes
import os

import pytest

import token_routing_expert_amd as tre

P = ctypes.c_void_p
FAKE = P(4096)
ODD = P(4096 + 8)   # not a multiple of 16

NAMES = {
    "moe_quantize_rows", "moe_quantize_weights", "moe_gate_up_swiglu_fp8", "moe_down_proj_fp8",
    "moe_grouped_ffn_fp8_workspace_size", "moe_grouped_ffn_fp8", "moe_forward_fp8_workspace_size", "moe_forward_fp8",
    "moe_forward_few_workspace_size", "moe_forward_few", "moe_forward_few_fp8_workspace_size", "moe_forward_few_fp8",
}
OK, ARG, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    return tre.load()


def test_exports_every_declared_symbol(lib):
    assert set(tre.exported_symbols(tre.SERVING_HEADER_PATH)) == NAMES
    if not os.path.exists(tre.DEBUG_LIB_PATH):
        from token_routing_expert_amd import build as tre_build
        tre_build.build(debug=True)
    dbg = tre.open_library(tre.DEBUG_LIB_PATH)
    for n in NAMES:
        assert hasattr(lib, n) and hasattr(dbg, n), n


def call(fn, **kw):
    """fn's defaults (a dict of its arguments in order) with some replaced."""
    f, defaults = fn
    args = dict(defaults)
    for k in kw:
        assert k in args, k
    args.update(kw)
    return f(*args.values())


def test_quantize_rows(lib):
    fn = lib.moe_quantize_rows, dict(x=FAKE, dt=1, rows=10, cols=192, q=FAKE, scale=FAKE, stream=None)
    assert call(fn, dt=2) == ARG
    assert call(fn, rows=-1) == ARG
    assert call(fn, cols=0) == ARG
    assert call(fn, cols=100) == UNSUPPORTED
    assert call(fn, rows=1 << 25) == UNSUPPORTED           # 2^25 * 192 elements
    for name in ("x", "q", "scale"):
        assert call(fn, **{name: None}) == ARG
    assert call(fn, x=ODD) == ARG and call(fn, q=ODD) == ARG
    assert call(fn, rows=0, x=None, q=None, scale=None) == OK


def test_quantize_weights(lib):
    fn = lib.moe_quantize_weights, dict(wgu=FAKE, wd=FAKE, dt=0, E=4, d=128, I=64, gq=FAKE, gs=FAKE, dq=FAKE, ds=FAKE,
                                        stream=None)
    assert call(fn, dt=9) == ARG
    assert call(fn, E=0) == ARG and call(fn, E=257) == UNSUPPORTED
    assert call(fn, d=96) == UNSUPPORTED and call(fn, I=100) == UNSUPPORTED and call(fn, I=0) == ARG
    assert call(fn, d=32768, I=16384) == UNSUPPORTED       # one expert's weights
    for name in ("wgu", "wd", "gq", "gs", "dq", "ds"):
        assert call(fn, **{name: None}) == ARG
    for name in ("wgu", "wd", "gq", "dq"):
        assert call(fn, **{name: ODD}) == ARG


def test_halves(lib):
    gu = lib.moe_gate_up_swiglu_fp8, dict(xq=FAKE, xs=FAKE, offs=FAKE, max_rows=10, E=4, d=128, I=64, wq=FAKE,
                                          ws=FAKE, row_token=None, x_rows=0, hq=FAKE, hs=FAKE, stream=None)
    dn = lib.moe_down_proj_fp8, dict(hq=FAKE, hs=FAKE, offs=FAKE, max_rows=10, E=4, d=128, I=64, wq=FAKE, ws=FAKE,
                                     y=FAKE, stream=None)
    for fn, ptrs, aligned in ((gu, ("xq", "xs", "offs", "wq", "ws", "hq", "hs"), ("xq", "wq", "hq")),
                              (dn, ("hq", "hs", "offs", "wq", "ws", "y"), ("hq", "wq", "y"))):
        assert call(fn, max_rows=-1) == ARG
        assert call(fn, E=0) == ARG and call(fn, E=300) == UNSUPPORTED
        assert call(fn, d=72) == UNSUPPORTED and call(fn, I=72) == UNSUPPORTED
        assert call(fn, max_rows=1 << 25) == UNSUPPORTED
        for name in ptrs:
            assert call(fn, **{name: None}) == ARG, name
        for name in aligned:
            assert call(fn, **{name: ODD}) == ARG, name
        assert call(fn, max_rows=0, **{n: None for n in ptrs}) == OK
    assert call(gu, row_token=FAKE, x_rows=-1) == ARG
    assert call(gu, row_token=FAKE, x_rows=1 << 25) == UNSUPPORTED


def test_grouped_ffn(lib):
    n = lib.moe_grouped_ffn_fp8_workspace_size(10, 192)
    assert n >= 10 * 192 + 10 * 2 * 4
    assert lib.moe_grouped_ffn_fp8_workspace_size(-1, 192) == 0 and lib.moe_grouped_ffn_fp8_workspace_size(1, 0) == 0
    fn = lib.moe_grouped_ffn_fp8, dict(xq=FAKE, xs=FAKE, offs=FAKE, max_rows=10, E=4, d=128, I=192, gq=FAKE, gs=FAKE,
                                       dq=FAKE, ds=FAKE, y=FAKE, ws=FAKE, ws_bytes=n, stream=None)
    assert call(fn, ws_bytes=n - 1) == WORKSPACE and call(fn, ws=None) == WORKSPACE
    assert call(fn, d=100) == UNSUPPORTED and call(fn, max_rows=-3) == ARG
    for name in ("xq", "xs", "offs", "gq", "gs", "dq", "ds", "y"):
        assert call(fn, **{name: None}) == ARG
    for name in ("xq", "gq", "dq", "y", "ws"):
        assert call(fn, **{name: ODD}) == ARG
    assert call(fn, max_rows=0, ws=None, ws_bytes=0) == OK


def test_forward(lib):
    n = lib.moe_forward_fp8_workspace_size(10, 128, 4, 2, 192)
    assert n > 0 and lib.moe_forward_fp8_workspace_size(20, 128, 4, 2, 192) > n
    assert lib.moe_forward_fp8_workspace_size(-1, 128, 4, 2, 192) == 0
    fn = lib.moe_forward_fp8, dict(x=FAKE, logits=FAKE, T=10, d=128, E=4, k=2, I=192, gq=FAKE, gs=FAKE, dq=FAKE,
                                   ds=FAKE, idx=FAKE, w=FAKE, offs=None, rt=None, pr=None, out=FAKE, ws=FAKE,
                                   ws_bytes=n, stream=None)
    assert call(fn, T=-1) == ARG and call(fn, k=0) == ARG and call(fn, k=5) == ARG
    assert call(fn, E=257) == UNSUPPORTED and call(fn, d=32) == UNSUPPORTED and call(fn, T=1 << 24) == UNSUPPORTED
    for name in ("x", "gq", "gs", "dq", "ds", "idx", "w", "out"):
        assert call(fn, **{name: None}) == ARG
    for name in ("x", "gq", "dq", "out", "ws"):
        assert call(fn, **{name: ODD}) == ARG
    assert call(fn, ws_bytes=n - 1) == WORKSPACE and call(fn, ws=None) == WORKSPACE
    assert call(fn, T=0, x=None, out=None, ws=None, ws_bytes=0) == OK


@pytest.mark.parametrize("fp8", [False, True])
def test_few(lib, fp8):
    sizes = dict(T=8, d=128, E=16, k=2, I=192)
    if fp8:
        size = lambda **kw: lib.moe_forward_few_fp8_workspace_size(*{**sizes, **kw}.values())   # noqa: E731
        weights, names = dict(gq=FAKE, gs=FAKE, dq=FAKE, ds=FAKE), ("gq", "dq")
    else:
        size = lambda **kw: lib.moe_forward_few_workspace_size(*{**sizes, **kw}.values(), 1)    # noqa: E731
        weights, names = dict(wgu=FAKE, wd=FAKE, dt=1), ("wgu", "wd")
    n = size()
    assert n >= 16 * 192 * 2 + 16 * 128 * 4
    assert size(T=65) == 0 and size(T=64, k=17) == 0 and size(T=-1) == 0 and size(k=0) == 0
    fn = (lib.moe_forward_few_fp8 if fp8 else lib.moe_forward_few,
          dict(x=FAKE, logits=FAKE, **sizes, **weights, idx=FAKE, w=FAKE, out=FAKE, ws=FAKE, ws_bytes=n, stream=None))
    assert call(fn, T=-1) == ARG and call(fn, k=0) == ARG and call(fn, k=17) == ARG
    assert call(fn, T=65) == UNSUPPORTED                                 # more than 64 tokens
    assert call(fn, T=64, k=17, logits=None) == UNSUPPORTED              # more than 1024 pairs
    assert call(fn, E=257) == UNSUPPORTED and call(fn, E=0) == ARG
    assert call(fn, d=100) == UNSUPPORTED and call(fn, I=32) == UNSUPPORTED
    for name in ("x", "idx", "w", "out") + tuple(k for k in weights if k != "dt"):
        assert call(fn, **{name: None}) == ARG
    for name in ("x", "out", "ws") + names:
        assert call(fn, **{name: ODD}) == ARG
    assert call(fn, ws_bytes=n - 1) == WORKSPACE and call(fn, ws=None) == WORKSPACE
    assert call(fn, T=0, x=None, out=None, ws=None, ws_bytes=0) == OK
    if not fp8:
        assert call(fn, dt=3) == ARG
        assert lib.moe_forward_few_workspace_size(*sizes.values(), 3) == 0


def test_widths_below_2_22(lib):
    """A tile's rows of codes are addressed with 31 bits: wider layers are refused by every call that takes one."""
    big = 1 << 22
    assert lib.moe_quantize_weights(FAKE, FAKE, 1, 1, big, 64, FAKE, FAKE, FAKE, FAKE, None) == UNSUPPORTED
    assert lib.moe_down_proj_fp8(FAKE, FAKE, FAKE, 4, 1, 64, big, FAKE, FAKE, FAKE, None) == UNSUPPORTED
    assert lib.moe_gate_up_swiglu_fp8(FAKE, FAKE, FAKE, 4, 1, big, 64, FAKE, FAKE, None, 0, FAKE, FAKE,
                                      None) == UNSUPPORTED
    assert lib.moe_grouped_ffn_fp8(FAKE, FAKE, FAKE, 4, 1, 64, big, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 40,
                                   None) == UNSUPPORTED
    assert lib.moe_forward_fp8(FAKE, FAKE, 1, big, 1, 1, 64, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, None, None, FAKE,
                               FAKE, 1 << 40, None) == UNSUPPORTED
    assert lib.moe_forward_few(FAKE, FAKE, 1, 64, 1, 1, big, FAKE, FAKE, 1, FAKE, FAKE, FAKE, FAKE, 1 << 40,
                               None) == UNSUPPORTED
    assert lib.moe_forward_few_fp8(FAKE, FAKE, 1, big, 1, 1, 64, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                                   1 << 40, None) == UNSUPPORTED


def test_binding_refuses(lib):
    """What the binding itself checks, with host tensors: nothing reaches the library."""
    import torch
    with pytest.raises(ValueError):
        tre.moe_quantize_rows(torch.zeros(4, 128, dtype=torch.bfloat16))         # not on the GPU
    with pytest.raises(ValueError):
        tre.moe_forward_few(torch.zeros(4, 128), torch.zeros(2, 64, 128), torch.zeros(2, 64, 128), 1)   # d differs


def test_reference_blocks():
    """The tests' own e4m3 arithmetic against torch's conversion, over every code and every midpoint."""
    import numpy as np
    import torch

    import serving_ref as ref
    v = ref.E4M3[np.isfinite(ref.E4M3)]
    v = np.unique(v)
    between = np.concatenate([v, (v[1:] + v[:-1]) / 2, (v[1:] * 0.75 + v[:-1] * 0.25)])
    want = torch.from_numpy(between).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.round_e4m3(between), want)
    assert ref.power_scale(np.array([448.0]))[0] == 1.0 and ref.power_scale(np.array([448.0001]))[0] == 2.0
    assert ref.power_scale(np.array([0.0]))[0] == 2.0 ** -126 and np.isnan(ref.power_scale(np.array([np.inf]))[0])
