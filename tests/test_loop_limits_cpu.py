"""What the operators around the loop take and refuse at their limits, before anything touches a device."""
import pytest
import torch


@pytest.mark.parametrize("shape", [(0, 100), (4, 0, 100), (0, 3, 100), (2, 0, 5, 7), (3, 0, 0)])
def test_rows_of_an_empty_tensor(shape):
    """No rows have any layout, whichever extent is 0."""
    from draft_block_candidate_gb300.logits import _logit_rows
    assert _logit_rows(torch.zeros(shape), "logits") == (0, shape[-1], shape[-1])
