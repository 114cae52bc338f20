"""Values that are not finite: a visible NaN key reaches every row that sees it."""
import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.test_gpu_packed import cu, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("place", list(range(16)))
@pytest.mark.parametrize("keys", [384, 3000])
def test_a_visible_nan_key_reaches_the_rows_of_packed_attention(keys, place, d):
    # one NaN key in a block that every row sees and that is not its first; 3,000 keys: in parts
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    q, k, v = make(torch.Generator().manual_seed(place), 40, keys, 2, 1, d, dev)
    k[256 + 32 + place] = float("nan")
    assert (lva.lva_packed_workspace_bytes(1, 2, 1, d, 40, keys) > 0) == (keys == 3000)
    o, lse = run(lva, q, k, v, cu([40]), cu([keys]), d ** -0.5, False)
    assert torch.isnan(o).all() and torch.isnan(lse).all()
