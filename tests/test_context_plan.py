"""How the shared-prefix call is cut (``lva_shared_prefix_plan``): every form that the kernels
have is reached by a shape of ``tests.context_forms``, and a plan keeps to the kernels' limits
and to the workspace's size (no GPU needed)."""
import ctypes
import random

import pytest

import block_sparse_attention_lva_b200 as lva
from block_sparse_attention_lva_b200 import _binding as lb
from tests.context_forms import FORMS


@pytest.mark.parametrize("form", list(FORMS), ids=str)
def test_forms(form):
    (B, steps, hq, hk, d, lp, cap), plan = FORMS[form]
    kind, dim, most = form
    assert lva.lva_shared_prefix_plan(B, steps, hq, hk, d, lp, cap) == plan and d == dim
    rows = steps * hq // hk * (B if kind == "list" else 1)         # the list's rows are the whole batch's
    assert {8: 0, 16: 8, 32: 16, 64: 32}[most] < rows <= most
    parts, workers, in_list = plan
    assert {"list": in_list and parts == 0, "turn": parts > 1 and workers == 148, "beside": parts > 1 and workers < 148}[kind]


@pytest.mark.parametrize("seed", range(50))
def test_plans_stay_within_the_kernels_limits(seed):
    rng = random.Random(seed)
    log = lambda lo, hi: int(lo * (hi / lo) ** rng.random())
    for _ in range(20):
        hk, group, steps = rng.choice([1, 2, 3, 8, 12]), rng.choice([1, 2, 3, 4, 5, 8, 16]), rng.choice([1, 1, 2, 4])
        B, d, lp, cap = log(1, 300), rng.choice([64, 128]), rng.choice([0, log(1, 70000)]), rng.choice([0, log(1, 9000)])
        parts, workers, in_list = lva.lva_shared_prefix_plan(B, steps, hk * group, hk, d, lp, cap)
        tok = 128 // group
        items = (B * steps + tok - 1) // tok * hk
        assert 52 <= workers <= 148
        assert (parts == 0) == (lp == 0 or in_list) and parts <= min(32, (lp + 127) // 128)
        assert workers == 148 or workers + items * parts == 148
        if in_list:
            assert cap > 0 and B * steps * group <= 32 and workers == 148
        # the workspace: the prefix's parts, a segment per (sequence, head) and worker, the scores
        up = lambda x: (x + 255) // 256 * 256
        rows = steps * group
        shared = (hk + 148) * B * rows if in_list else parts * B * hk * rows
        own = (B * hk + 148) * rows if cap else 0
        want = up(shared * d * 4) + up(shared * 4) + up(own * d * 4) + up(own * 4)
        size = lva.lva_shared_prefix_workspace_bytes
        assert size(B, steps, hk * group, hk, d, lp, cap) == want
        assert size(B, steps, hk * group, hk, d, lp, cap, True) == want + up(B * hk * rows * ((cap + 63) // 64 * 64) * 4)


def test_refusals():
    good = (2, 1, 4, 2, 64, 100, 50)
    for at, bad, status in ((4, 96, 2), (2, 3, 1), (0, -1, 1), (1, 0, 1), (1, 33, 2), (5, -1, 1), (6, 1 << 31, 2)):
        sizes = list(good)
        sizes[at] = bad
        with pytest.raises(lva.LvaError) as e:
            lva.lva_shared_prefix_plan(*sizes)
        assert e.value.status == status
    ints = [ctypes.byref(ctypes.c_int()) for _ in range(3)]
    params = lb._PREFIX.pack(*good[:5], 1.0, *good[5:], *[0] * 8)
    assert lb.lib.lva_shared_prefix_plan(None, *ints) == 1
    for missing in range(3):
        assert lb.lib.lva_shared_prefix_plan(params, *[None if i == missing else x for i, x in enumerate(ints)]) == 1
