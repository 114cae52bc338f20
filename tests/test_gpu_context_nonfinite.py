"""Values that are not finite: a visible NaN key reaches every row that sees it, and nothing at a
key that a row does not see reaches that row, whatever it is."""
import numpy as np
import pytest
import torch

from tests.context_forms import FORMS
from tests.gpu_helpers import bits, require_gpu
from tests.test_gpu_context_cache import Case
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


@pytest.mark.parametrize("place", [0, 14, 15])
@pytest.mark.parametrize("where", ["prefix", "cache"])
@pytest.mark.parametrize("form", [("turn", 128, 8), ("beside", 64, 32), ("list", 64, 16)], ids=str)
def test_a_visible_nan_key_reaches_the_rows_of_a_shared_prefix(form, where, place):
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    sizes, _ = FORMS[form]
    B, T, cap = sizes[0], sizes[1], sizes[6]
    c = Case(dev, place, *sizes, [cap] * B, False)
    clean = c.run(lva)
    (c.pk if where == "prefix" else c.kc[0, 0])[16 + place] = float("nan")
    o, lse, _ = c.run(lva)
    if where == "prefix":
        assert torch.isnan(o).all() and torch.isnan(lse).all()
    else:
        g = sizes[2] // sizes[3]
        assert torch.isnan(o[0, :, :g]).all() and torch.isnan(lse[0, :g]).all()
        assert np.array_equal(bits(o[0, :, g:]), bits(clean[0][0, :, g:])) and np.array_equal(bits(o[1:]), bits(clean[0][1:]))


# (B, steps, q_heads, kv_heads, d, prefix, capacity), lens: 8, 16, 32 and 64 rows, a batch in the
# list, the step's tokens across a tile's edge, at one, and more tokens than entries
STEPS = {
    "rows_8": ((2, 4, 4, 2, 128, 70, 90), [90, 66]),
    "rows_8_alone": ((2, 8, 2, 2, 64, 0, 300), [300, 132]),
    "rows_16": ((3, 4, 12, 3, 128, 300, 200), [200, 67, 3]),
    "rows_32": ((3, 4, 8, 1, 128, 0, 200), [129, 66, 200]),
    "rows_40": ((2, 5, 8, 1, 64, 70, 190), [190, 67]),
    "rows_64": ((2, 32, 4, 2, 128, 70, 190), [190, 80]),
    "rows_64_tokens": ((2, 64, 1, 1, 64, 0, 190), [190, 60]),
    "list": ((2, 3, 4, 2, 64, 165, 169), [130, 2]),
}


@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("name", list(STEPS))
def test_a_later_tokens_value_does_not_reach_the_earlier_ones(name, value):
    # token t sees the entries up to n - T + t: what V holds at the later ones is nothing to it
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    sizes, lens = STEPS[name]
    B, T, hq, hk, d, lp, cap = sizes
    x = float(value)
    for back in {1, 2, T - 1}:                        # the entry that many before the end
        if back >= T:
            continue
        c = Case(dev, 7 + back, *sizes, lens, True)
        clean, v0 = c.run(lva), c.vc.clone()
        dims = [0, 9, 17, d // 2 + 8, d - 1]
        for b, n in enumerate(lens):
            c.vc[b, :, max(n - back, 0), dims] = x
        o, lse, w = c.run(lva)
        c.vc.copy_(v0)
        assert lva.lva_device_error() == (0, 0)
        assert np.array_equal(bits(lse), bits(clean[1])) and np.array_equal(bits(w), bits(clean[2]))
        patched = o.clone()
        for b, n in enumerate(lens):
            first = max(max(n - back, 0) - (n - T), 0)     # the first token that sees the entry
            got = o[b, first:, :, dims].float()
            assert torch.isnan(got).all() if np.isnan(x) else (got == x).all()
            patched[b, first:, :, dims] = clean[0][b, first:, :, dims]
        # other columns bit for bit; these, whose sums are taken another way, as near the oracle
        rest = [e for e in range(d) if e not in dims]
        assert np.array_equal(bits(patched[..., rest]), bits(clean[0][..., rest]))
        c.compare(patched, lse, w)


def test_opposite_infinities_meet_only_where_both_are_seen():
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    B, T, hq, hk, d, lp, cap = sizes = (2, 4, 4, 1, 128, 40, 150)
    lens = [150, 66]
    c = Case(dev, 3, *sizes, lens, False)
    (clean, lse, _), v0 = c.run(lva), c.vc.clone()
    for b, n in enumerate(lens):
        c.vc[b, 0, n - 3, 5] = float("inf")            # token 1 sees it first
        c.vc[b, 0, n - 1, 5] = float("-inf")           # the last token alone
    o = c.run(lva)[0]
    c.vc.copy_(v0)
    assert torch.isposinf(o[:, 1:3, :, 5]).all() and torch.isnan(o[:, 3, :, 5]).all()
    rest = [e for e in range(d) if e != 5]
    assert np.array_equal(bits(o[..., rest]), bits(clean[..., rest]))
    o[:, 1:, :, 5] = clean[:, 1:, :, 5]
    c.compare(o, lse, None)


def test_a_value_seen_by_all_rows_reaches_them():
    # not finite in the prefix, or at a cache entry that every token sees: nothing is summed up again
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    sizes, lens = STEPS["rows_16"]
    for where, x in (("prefix", "nan"), ("prefix", "inf"), ("cache", "-inf")):
        c = Case(dev, 4, *sizes, lens, False)
        clean = c.run(lva)[0]
        if where == "prefix":
            c.pv[3, :, 7] = float(x)
        else:
            c.vc[0, :, 5, 7] = float(x)
        o = c.run(lva)[0]
        hit = o[:, :, :, 7].float() if where == "prefix" else o[0, :, :, 7].float()
        assert torch.isnan(hit).all() if x == "nan" else (hit == float(x)).all()
        hit_clean = clean[:, :, :, 7] if where == "prefix" else clean[0, :, :, 7]
        (o[:, :, :, 7] if where == "prefix" else o[0, :, :, 7]).copy_(hit_clean)
        assert np.array_equal(bits(o), bits(clean))
