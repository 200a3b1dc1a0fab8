"""Sizes of the training-step operators' scratch, without a GPU."""

import pytest

from gradient_aggregation_gb300 import fc


@pytest.mark.parametrize("rows,cols,most", [
    (1024, 1 << 20, 1),       # one set of the two sums
    (1 << 20, 1 << 20, 1),
    (2048, 40000, 13),
    (1 << 20, 16385, 31),
    (1024, 16384, 80),
    (1 << 20, 8192, 160),
    (1 << 20, 257, 160),
    (1 << 20, 256, 1024),
    (3, 8192, 3),
])
def test_backward_scratch_is_what_the_blocks_leave(fc_lib, rows, cols, most):
    """A set is two rows of fp32 sums, and there are no more sets than blocks that
    leave one."""
    padded = (cols + 7) // 8 * 8
    assert fc.fc_layernorm_backward_workspace_size(rows, cols) <= most * padded * 8
