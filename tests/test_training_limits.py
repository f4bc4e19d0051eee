"""Rules on sizes of the training operators that the host can be asked for, without a GPU."""
import token_routing_expert_amd as tre

WIDEST = (1 << 21) - 64


def test_the_widest_rows_take_no_tall_tiles():
    """288 rows of 4 I bytes pass 2^31 from I = 1864128 on.  Tall tiles of gate/up need 256 I bytes of workspace more
    than the 576 I of h: without them a wider call needs less."""
    size = tre.load().moe_grouped_ffn_train_workspace_size
    tall, widest = size(288, 1, 128, 1864064, 1), size(288, 1, 128, WIDEST, 1)
    assert tall > (576 + 256) * 1864064 and 576 * WIDEST < widest < tall


def test_the_least_calls_go_to_the_kernels_of_few_tiles_unless_a_sum_is_long():
    """Those kernels' forward of d <= 768 has h in float32 for its workspace, and nothing else.  A workgroup there walks d
    or 2 I terms by itself, which long sums are too slow for, unless experts without rows cost more elsewhere."""
    size = tre.load().moe_grouped_ffn_train_workspace_size

    def few(rows, E, d, I):
        return size(rows, E, d, I, 1) == -(-4 * rows * I // 256) * 256

    assert few(1, 1, 64, 64) and few(64, 1, 64, 2880) and few(16, 8, 512, 512) and few(8, 8, 64, 1024)
    assert not few(64, 1, 64, 8192) and not few(1, 1, 512, 16384) and not few(128, 8, 64, 65536)
    assert few(1, 64, 512, 8192)


def test_the_forward_takes_tall_tiles_up_to_288_rows_an_expert():
    """Above, a tall tile's 32 rows more no longer hold what 256 leave, and cost 5 to 14% of the forward.  Tall tiles show as
    64 I floats of workspace for each expert."""
    size, E, I = tre.load().moe_grouped_ffn_train_workspace_size, 8, 1024
    at, above = size(288 * E, E, 1024, I, 1), size(289 * E, E, 1024, I, 1)
    assert at - above == 4 * E * 64 * I - 2 * E * I
