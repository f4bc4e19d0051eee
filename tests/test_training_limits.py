"""Rules on sizes of the training operators that the host can be asked for, without a GPU."""
import token_routing_expert_amd as tre

WIDEST = (1 << 21) - 64


def test_the_widest_rows_take_no_tall_tiles():
    """288 rows of 4 I bytes pass 2^31 from I = 1864128 on.  Tall tiles of gate/up need 256 I bytes of workspace more
    than the 576 I of h: without them a wider call needs less."""
    size = tre.load().moe_grouped_ffn_train_workspace_size
    tall, widest = size(288, 1, 128, 1864064, 1), size(288, 1, 128, WIDEST, 1)
    assert tall > (576 + 256) * 1864064 and 576 * WIDEST < widest < tall
