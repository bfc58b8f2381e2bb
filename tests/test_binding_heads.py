"""Host-side checks of the head norm's arguments in the binding (no GPU)."""
import pytest
import torch

from kda_recurrent_state_gb300 import binding

Q, TABLE, AT = torch.zeros(3, 2, 8), torch.zeros(5, 2), torch.zeros(3, dtype=torch.int64)


def heads(cos, sin, positions):
    return binding._head_args(Q, None, None, None, cos, sin, positions, -1)  # -1: the CPU's number


def test_half_a_rotation_is_refused():
    """cos without sin or positions, and sin without cos: nothing would be turned, or half of it."""
    for cos, sin, positions in ((TABLE, None, AT), (TABLE, TABLE, None), (None, TABLE, AT), (None, TABLE, None)):
        with pytest.raises(ValueError, match="the rotation wants cos and sin"):
            heads(cos, sin, positions)


def test_positions_alone_turn_nothing():
    """A layer without a rotation may pass its positions all the same."""
    assert heads(None, None, AT)[0][-1] == 0 and heads(None, None, None)[0][-1] == 0
    assert heads(TABLE, TABLE, AT)[0][-1] == 4
