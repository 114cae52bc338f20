"""Sizes that do not fit their C types: the workspace calls answer -1, as for any size that is
refused, the plan raises ValueError (no GPU needed)."""
import pytest

import block_sparse_attention_lva_b200 as lva


@pytest.mark.parametrize("sizes", [(1 << 31, 4, 2, 64, 10, 10), (1, 1 << 40, 2, 64, 10, 10), (1, 4, 2, 64, 1 << 63, 10), (1, 4, 2, 64, 10, -(1 << 70))])
def test_packed_workspace(sizes):
    assert lva.lva_packed_workspace_bytes(*sizes) == -1


@pytest.mark.parametrize("at,value", [(0, 1 << 31), (1, 1 << 31), (2, -(1 << 31) - 1), (5, 1 << 63), (6, 1 << 64)])
def test_shared_prefix_workspace_and_plan(at, value):
    sizes = [2, 1, 4, 2, 64, 100, 50]
    sizes[at] = value
    assert lva.lva_shared_prefix_workspace_bytes(*sizes) == -1
    with pytest.raises(ValueError, match="out of range"):
        lva.lva_shared_prefix_plan(*sizes)
