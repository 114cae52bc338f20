"""Every form of the shared-prefix call (``tests.context_forms``) against the float64 oracle,
on two streams and over one workspace; a sequence alone and in a batch."""
import numpy as np
import pytest
import torch

from tests.context_forms import FORMS, lens_of
from tests.gpu_helpers import bits, require_gpu
from tests.test_gpu_context_cache import Case

pytestmark = pytest.mark.gpu


def case_of(dev, form, weights, seed=0):
    sizes, _ = FORMS[form]
    return Case(dev, sum(repr(form).encode()) + seed, *sizes, lens_of(form), weights)


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("form", list(FORMS), ids=str)
def test_form_matches_oracle(form, weights):
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    sizes, plan = FORMS[form]
    assert lva.lva_shared_prefix_plan(*sizes) == plan
    c = case_of(dev, form, weights)
    out = c.run(lva)
    assert lva.lva_device_error() == (0, 0)
    c.compare(*out)


def same(a, b):
    return all(np.array_equal(bits(x), bits(y)) for x, y in zip(a, b) if x is not None)


TURNS = [("beside", 128, 8), ("list", 64, 32), ("beside", 64, 64), ("turn", 128, 16), ("beside", 128, 32)]


def test_forms_on_two_streams():
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    cases = [case_of(dev, f, True) for f in TURNS[:2]]
    refs = [c.run(lva) for c in cases]
    spaces = [c.workspace(lva) for c in cases]
    outs = [[c.outputs() for _ in range(12)] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for i in range(12):
        for c, ws, out, st in zip(cases, spaces, outs, streams):
            o, lse, w = out[i]
            with torch.cuda.stream(st):
                lva.lva_shared_prefix_attn(c.q, c.pk, c.pv, c.kc, c.vc, c.lens_t, o, lse, ws, c.scale, weight=w)
    torch.cuda.synchronize()
    assert lva.lva_device_error() == (0, 0)
    assert all(same(ref, got) for ref, out in zip(refs, outs) for got in out)


def test_forms_in_turn_over_one_workspace():
    # parts beside the caches' workers, in the list and behind them: none writes the workspace
    # while the call before still reads it
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    cases = [case_of(dev, f, i % 2 == 0, seed=1) for i, f in enumerate(TURNS)]
    refs = [c.run(lva) for c in cases]
    ws = max((c.workspace(lva) for c in cases), key=lambda x: x.numel())
    outs = [[c.outputs() for _ in range(6)] for c in cases]
    torch.cuda.synchronize()
    for i in range(6):
        for c, out in zip(cases, outs):
            o, lse, w = out[i]
            lva.lva_shared_prefix_attn(c.q, c.pk, c.pv, c.kc, c.vc, c.lens_t, o, lse, ws, c.scale, weight=w)
    torch.cuda.synchronize()
    assert lva.lva_device_error() == (0, 0)
    assert all(same(ref, got) for ref, out in zip(refs, outs) for got in out)


def test_a_sequence_alone_and_in_a_batch():
    # its parts are cut elsewhere, its results agree within twice their distance from the oracle
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    B, T, hq, hk, d, lp, cap = sizes = (7, 2, 8, 2, 128, 400, 900)
    lens = [900, 5, 0, 333, 64, 800, 700]
    c = Case(dev, 3, *sizes, lens, True)
    o, lse, w = c.run(lva)
    for b in (0, 3, 6):
        one = Case(dev, 3, 1, T, hq, hk, d, lp, cap, [lens[b]], True)
        one.q, one.pk, one.pv, one.kc, one.vc, one.w0 = (c.q[b:b + 1], c.pk, c.pv, c.kc[b:b + 1].contiguous(),
                                                         c.vc[b:b + 1].contiguous(), c.w0[b:b + 1].contiguous())
        o1, lse1, w1 = one.run(lva)
        one.compare(o1, lse1, w1)
        one.compare(o[b:b + 1], lse[b:b + 1], w[b:b + 1])
