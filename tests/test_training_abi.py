"""include/moe_training.h: every declared function is exported (by both
builds), and the host-side checks refuse bad arguments before anything is
enqueued.  No kernel is launched: every call fails a check or has nothing to do."""
import ctypes
import os

import pytest

import token_routing_expert_amd as tre

P = ctypes.c_void_p
FAKE = P(4096)
ODD = P(4096 + 8)   # not a multiple of 16

NAMES = {
    "moe_grouped_ffn_train_workspace_size", "moe_grouped_ffn_train", "moe_grouped_ffn_backward_workspace_size",
    "moe_grouped_ffn_backward", "moe_forward_train_q8_workspace_size", "moe_forward_train_q8",
    "moe_backward_q8_workspace_size", "moe_backward_q8", "moe_checkpoint_values",
}
OK, ARG, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return tre.load()


def test_exports_every_declared_symbol(lib):
    assert set(tre.exported_symbols(tre.TRAINING_HEADER_PATH)) == NAMES
    if not os.path.exists(tre.DEBUG_LIB_PATH):
        from token_routing_expert_amd import build as tre_build
        tre_build.build(debug=True)
    dbg = tre.open_library(tre.DEBUG_LIB_PATH)
    for n in NAMES:
        assert hasattr(lib, n) and hasattr(dbg, n), n


def calls(lib):
    """(function, its arguments in order, those that must be given, those of 16-byte alignment) by name."""
    train = dict(x=FAKE, offs=FAKE, max_rows=10, E=4, d=128, I=64, wgu=FAKE, wd=FAKE, dt=1, y=FAKE, q=FAKE, s=FAKE,
                 ws=FAKE, nbytes=BIG, stream=None)
    back = dict(x=FAKE, offs=FAKE, max_rows=10, E=4, d=128, I=64, wgu=FAKE, wd=FAKE, dt=1, q=FAKE, s=FAKE, dy=FAKE,
                dx=FAKE, dwgu=FAKE, dwd=FAKE, ws=FAKE, nbytes=BIG, stream=None)
    fwd = dict(x=FAKE, logits=FAKE, T=10, d=128, E=4, k=2, I=64, wgu=FAKE, wd=FAKE, dt=1, idx=FAKE, w=FAKE, offs=FAKE,
               tok=FAKE, row=FAKE, q=FAKE, s=FAKE, out=FAKE, ws=FAKE, nbytes=BIG, stream=None)
    bwd = dict(x=FAKE, T=10, d=128, E=4, k=2, I=64, wgu=FAKE, wd=FAKE, dt=1, idx=FAKE, w=FAKE, offs=FAKE, tok=FAKE,
               row=FAKE, q=FAKE, s=FAKE, dout=FAKE, dx=FAKE, dwgu=FAKE, dwd=FAKE, dw=FAKE, dlogits=None, ws=FAKE,
               nbytes=BIG, stream=None)
    return {
        "train": (lib.moe_grouped_ffn_train, train, "x offs wgu wd y q s", "x wgu wd y q ws"),
        "back": (lib.moe_grouped_ffn_backward, back, "x offs wgu wd dy dx dwgu dwd", "x wgu wd dy dx dwgu dwd q ws"),
        "fwd": (lib.moe_forward_train_q8, fwd, "x wgu wd idx w offs tok row q s out", "x wgu wd q out ws"),
        "bwd": (lib.moe_backward_q8, bwd, "x wgu wd idx w offs tok row q s dout dx dwgu dwd dw",
                "x wgu wd q dout dx dwgu dwd ws"),
    }


def call(fn, **kw):
    f, args = fn[0], dict(fn[1])
    for k in kw:
        assert k in args, k
    args.update(kw)
    return f(*args.values())


@pytest.mark.parametrize("name", ["train", "back", "fwd", "bwd"])
def test_refusals(lib, name):
    fn = calls(lib)[name]
    rows = "T" if "T" in fn[1] else "max_rows"
    assert call(fn, dt=2) == ARG and call(fn, dt=-1) == ARG
    assert call(fn, **{rows: -1}) == ARG
    assert call(fn, E=0) == ARG and call(fn, E=257) == UNSUPPORTED
    assert call(fn, d=0) == ARG and call(fn, d=100) == UNSUPPORTED and call(fn, I=-64) == ARG
    assert call(fn, I=96) == UNSUPPORTED
    assert call(fn, d=1 << 21, I=64) == UNSUPPORTED and call(fn, d=64, I=1 << 21) == UNSUPPORTED
    assert call(fn, d=32768, I=16384) == UNSUPPORTED              # one expert's weights
    assert call(fn, **{rows: 1 << 23}, I=128, d=64) == UNSUPPORTED   # 2^23 * 2 * 128 elements
    for p in fn[2].split():
        if p == "s" and name == "back":
            continue
        assert call(fn, **{p: None}) == ARG, p
    for p in fn[3].split():
        assert call(fn, **{p: ODD}) == ARG, p
    assert call(fn, ws=None) == WORKSPACE and call(fn, nbytes=0) == WORKSPACE


def test_checkpoint_comes_whole(lib):
    fn = calls(lib)["back"]
    assert call(fn, q=None) == ARG and call(fn, s=None) == ARG
    assert call(fn, q=None, s=None, nbytes=0) == WORKSPACE        # without one: g | u are computed again


def test_layer_arguments(lib):
    c = calls(lib)
    assert call(c["fwd"], k=0) == ARG and call(c["bwd"], k=0) == ARG
    assert call(c["fwd"], k=5) == ARG                              # routes, k > E
    assert call(c["fwd"], k=5, logits=None, nbytes=0) == WORKSPACE   # given pairs may be more
    assert call(c["bwd"], k=5, dlogits=FAKE) == ARG and call(c["bwd"], k=5, nbytes=0) == WORKSPACE
    assert call(c["fwd"], T=1 << 24, k=1, I=64, d=64) == UNSUPPORTED   # token rows past 32-bit byte offsets


def test_nothing_to_do(lib):
    c = calls(lib)
    assert call(c["train"], max_rows=0, x=None, y=None, ws=None, nbytes=0) == OK
    assert call(c["fwd"], T=0, x=None, out=None, ws=None, nbytes=0) == OK
    # no rows: the weight gradients are still written
    assert call(c["back"], max_rows=0, dwgu=None) == ARG and call(c["bwd"], T=0, dwd=None) == ARG
    assert call(c["back"], max_rows=0, dwd=ODD) == ARG


def test_checkpoint_values(lib):
    args = dict(q=FAKE, s=FAKE, rows=4, I=64, dt=0, gu=FAKE, stream=None)
    fn = (lib.moe_checkpoint_values, args)
    assert call(fn, dt=3) == ARG and call(fn, rows=-1) == ARG and call(fn, I=0) == ARG
    assert call(fn, I=100) == UNSUPPORTED and call(fn, rows=1 << 24) == UNSUPPORTED
    for p in ("q", "s", "gu"):
        assert call(fn, **{p: None}) == ARG
    assert call(fn, q=ODD) == ARG and call(fn, gu=ODD) == ARG
    assert call(fn, rows=0, q=None, s=None, gu=None) == OK


def test_workspace_sizes(lib):
    for dt in (0, 1):
        for f, bad in ((lib.moe_grouped_ffn_train_workspace_size, (-1, 4, 128, 64)),
                       (lib.moe_grouped_ffn_backward_workspace_size, (10, 0, 128, 64))):
            assert f(*bad, dt) == 0 and f(10, 4, 128, 64, 2) == 0
            assert 0 < f(10, 4, 128, 64, dt) <= f(1000, 4, 128, 64, dt) <= f(1000, 4, 128, 640, dt)
        for f in (lib.moe_forward_train_q8_workspace_size, lib.moe_backward_q8_workspace_size):
            assert f(-1, 128, 4, 2, 64, dt) == 0 and f(10, 128, 4, 0, 64, dt) == 0 and f(10, 128, 4, 2, 64, 7) == 0
            assert 0 < f(10, 128, 4, 2, 64, dt) <= f(1000, 128, 4, 2, 64, dt)
            assert f(0, 128, 4, 2, 64, dt) >= 0


def test_a_checkpoint_is_smaller_than_the_kept_state(lib):
    """2.125 I bytes a grouped row and three indices a pair, against the workspace that moe_forward_train keeps."""
    T, d, E, k, I = 8192, 2880, 128, 4, 2880
    kept = T * k * (2 * I + 8 * I // 64 + 8) + 4 * (E + 1)
    assert 4 * kept < lib.moe_backward_workspace_size(T, d, E, k, I, 1)
