"""The sizes that include/moe_serving.h promises, on both sides of each limit.
No kernel is launched: a call inside its limits has no rows to work on, or
stops at a missing workspace."""
import ctypes

import pytest

import token_routing_expert_amd as tre

FAKE = ctypes.c_void_p(4096)
OK, UNSUPPORTED, WORKSPACE = 0, 2, 3


def answers(lib, E, d, I):
    """What each call says to a layer of these sizes, by name."""
    F = FAKE
    codes = {
        "gate_up": lib.moe_gate_up_swiglu_fp8(F, F, F, 0, E, d, I, F, F, None, 0, F, F, None),
        "down": lib.moe_down_proj_fp8(F, F, F, 0, E, d, I, F, F, F, None),
        "ffn": lib.moe_grouped_ffn_fp8(F, F, F, 0, E, d, I, F, F, F, F, F, F, 0, None),
        "forward": lib.moe_forward_fp8(F, F, 1, d, E, 1, I, F, F, F, F, F, F, None, None, None, F, None, 0, None),
        "few": lib.moe_forward_few_fp8(F, F, 1, d, E, 1, I, F, F, F, F, F, F, F, None, 0, None),
    }
    return codes, lib.moe_forward_few(F, F, 1, d, E, 1, I, F, F, 1, F, F, F, None, 0, None)


@pytest.mark.parametrize("E,d,I", [
    (1, 16384, 40960),                  # 2 d I = 1.34e9
    (3, 16384, 40960),                  # three of them: 4.0e9 codes
    (1, 16384, 65536 - 64),             # the last width below 2^31
    (8, 16384, 65536 - 64),             # and of all experts together below 2^34
    (1, 256, (1 << 22) - 64),           # the widest layer
])
def test_eight_bit_layers_inside(E, d, I):
    codes, _ = answers(tre.load(), E, d, I)
    assert codes == {"gate_up": OK, "down": OK, "ffn": OK, "forward": WORKSPACE, "few": WORKSPACE}


@pytest.mark.parametrize("E,d,I", [
    (1, 16384, 65536),                  # one expert's 2 d I = 2^31
    (9, 16384, 65536 - 64),             # all experts past 2^34
    (1, 64, 1 << 22),                   # a width of 2^22
])
def test_eight_bit_layers_outside(E, d, I):
    codes, _ = answers(tre.load(), E, d, I)
    assert set(codes.values()) == {UNSUPPORTED}


def test_weights_in_sixteen_bits():
    """Weights in moe.h's layouts keep its limit of 2 GiB an expert, here and in moe_quantize_weights."""
    lib, F = tre.load(), FAKE
    assert answers(lib, 1, 16384, 32768 - 64)[1] == WORKSPACE
    assert answers(lib, 1, 16384, 32768)[1] == UNSUPPORTED
    assert lib.moe_quantize_weights(F, F, 1, 1, 16384, 32768, F, F, F, F, None) == UNSUPPORTED


@pytest.mark.parametrize("E,k", [(1, 1), (16, 2), (256, 1), (4, 256)])
def test_no_tokens(E, k):
    """Zero tokens are valid: every workspace has a size, and every call nothing to do."""
    lib, d, I = tre.load(), 128, 192
    sizes = [lib.moe_forward_fp8_workspace_size(0, d, E, k, I), lib.moe_forward_few_fp8_workspace_size(0, d, E, k, I)]
    sizes += [lib.moe_forward_few_workspace_size(0, d, E, k, I, dt) for dt in (0, 1)]
    assert all(0 < n <= lib.moe_forward_fp8_workspace_size(1, d, E, k, I) for n in sizes)
    assert lib.moe_grouped_ffn_fp8_workspace_size(0, I) == 0
    for dt in (0, 1):
        assert lib.moe_forward_few(None, None, 0, d, E, k, I, FAKE, FAKE, dt, None, None, None, None, 0, None) == OK
    assert lib.moe_forward_few_fp8(None, None, 0, d, E, k, I, FAKE, FAKE, FAKE, FAKE, None, None, None, None, 0,
                                   None) == OK
    assert lib.moe_forward_fp8(None, None, 0, d, E, k, I, FAKE, FAKE, FAKE, FAKE, None, None, None, None, None, None,
                               None, 0, None) == OK
