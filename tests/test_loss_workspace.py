"""What the vocabulary loss asks for as workspace (no GPU): what it uses, not a
copy that no call of that dtype makes."""
import pytest
import torch

import collective_communication_primitives_amd as dt

SHARDS = [16384] * 8


@pytest.mark.parametrize("cols", [4096, 4097, 16384])
def test_fp32_weights_are_never_copied(cols):
    """fp32 rows lie on 4-byte boundaries, which the kernels read as they are: beside a padded copy of hidden there is a
    maximum and a sum per 64 rows and token, with a margin for the ends of shards and pieces, and the target's logit."""
    tokens, rows = 2, sum(SHARDS)
    hidden = tokens * ((cols + 3) // 4 * 16)
    entries = rows // 64 + 2 * (rows // 16384)
    forward = dt.dt_vocab_loss_workspace(SHARDS, tokens, cols, torch.float32)
    assert forward <= hidden + entries * tokens * 8 + tokens * 4 + 4 * 256
    # the piece's d (each rank's part on whole steps of 16 rows) and up to 32 sums of the hidden state's gradient
    piece = 1000
    backward = dt.dt_vocab_loss_backward_workspace(SHARDS, tokens, cols, torch.float32, piece)
    assert backward <= hidden + tokens * (piece + 9 * 16) * 4 + 32 * hidden + 64 * 4 + 4 * 256


def test_bf16_keeps_room_for_a_copied_piece():
    """Rows of odd width, or weights that start at an odd element, are copied a piece at a time."""
    assert dt.dt_vocab_loss_workspace(SHARDS, 2, 4096, torch.bfloat16) >= 16384 * 4096 * 2
