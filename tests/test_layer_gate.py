"""What a gate's shape means, on the host."""
import pytest
import torch

import zero_partitioned_mixed_step_gb300 as zs
from zero_partitioned_mixed_step_gb300.layer import GATE_COLS, GATE_NONE, GATE_ONE, GATE_ROWS


@pytest.mark.parametrize("rows", [1, 2, 5])
def test_a_gates_kind_is_its_own(rows):
    kind = zs.layer._gate_kind
    assert kind(None, rows, 8) == GATE_NONE
    assert kind(torch.ones(()), rows, 8) == GATE_ONE and kind(torch.ones(1), rows, 8) == GATE_ONE
    assert kind(torch.ones(8), rows, 8) == GATE_COLS and kind(torch.ones(rows, 1), rows, 8) == GATE_ROWS
    for other in ((rows + 1, 1), (1, 8), (rows, 8), (rows + 8,)):
        with pytest.raises(ValueError):
            kind(torch.ones(other), rows, 8)


def test_one_number_in_two_dimensions_is_refused():
    """It would be a token's gate where a call has one row, whose gradient is written, and not one number's, whose
    gradient is added."""
    with pytest.raises(ValueError):
        zs.layer._gate_kind(torch.ones(1, 1), 4, 8)
