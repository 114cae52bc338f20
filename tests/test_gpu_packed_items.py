"""Packed attention where a thread block takes several items of many key blocks each (cluster
launch control, the double Q buffer, ring phases from one item to the next), on sampled rows;
long key ranges without a workspace; the same call again."""
import ctypes

import numpy as np
import pytest
import torch

from oracle.packed import _rows
from tests.context_helpers import tolerances
from tests.gpu_helpers import bits, require_gpu
from tests.test_gpu_packed import LONG, compare, cu, run

pytestmark = pytest.mark.gpu

# query and key lengths; with 8 key/value heads 500 to 1,300 items of 1 to 20 blocks, none
# of them cut into parts
PROMPTS = [100, 2500, 0, 1281, 700, 1, 1900, 128, 0, 2300, 517, 1024]


def sample(rng, n, tok):
    """Rows of a sequence: its ends, both sides of tile edges, some between."""
    edges = [x for t in (1, 2, 5, 9) for x in (t * tok - 1, t * tok)]
    rows = {0, n - 1, *[x for x in edges if x < n], *[int(x) for x in rng.integers(0, n, 24)]} if n else set()
    return sorted(rows)


def check_rows(q, k, v, o, lse, ql, kl, scale, causal, seed):
    qh, kh, vh, oh = (x.double().cpu().numpy() for x in (q, k, v, o))
    lh = lse.double().cpu().numpy()
    assert not np.isnan(oh).any() and not np.isnan(lh).any()
    hq, hk = q.shape[1], k.shape[1]
    rng = np.random.default_rng(seed)
    at_q = at_k = 0
    for n, m in zip(ql, kl):
        rows = np.array(sample(rng, n, 128 // (hq // hk)), dtype=int)
        for h in range(hq if len(rows) else 0):
            g = h // (hq // hk)
            c = np.arange(m)[None, :]
            seen = (c <= rows[:, None] + m - n) if causal else np.ones((len(rows), m), dtype=bool)
            keys, values = kh[at_k:at_k + m, g], vh[at_k:at_k + m, g]
            qr = qh[at_q + rows, h]
            o_ref, lse_ref, _, mag = _rows(qr, keys, values, seen, scale)
            tol_o, tol_l = tolerances(torch.from_numpy(qr), torch.from_numpy(keys), scale, mag, o_ref)
            got, got_l = oh[at_q + rows, h], lh[h, at_q + rows]
            bad = np.abs(got - o_ref) > tol_o
            assert not bad.any(), (h, n, m, bad.sum(), np.abs(got - o_ref).max(), rows[np.argwhere(bad)[:4, 0]])
            empty = np.isneginf(lse_ref)
            assert np.array_equal(np.isneginf(got_l), empty)
            if not empty.all():
                assert np.abs(got_l[~empty] - lse_ref[~empty]).max() <= tol_l
        at_q, at_k = at_q + n, at_k + m


def inputs(dev, seed, tq, tk, hq, hk, d):
    g = torch.Generator(device=dev).manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device=dev).to(torch.bfloat16)
    return n(tq, hq, d), n(tk, hk, d), n(tk, hk, d)


@pytest.mark.parametrize("kind", ["prompts", "reversed", "growing", "continued"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hk,d", [(16, 8, 64), (16, 8, 128), (24, 8, 64), (24, 8, 128)])
def test_many_items_of_many_blocks(hq, hk, d, causal, kind):
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    kl = PROMPTS[::-1] if kind == "reversed" else PROMPTS
    ql = [min(n, 900) if i % 3 else n // 2 for i, n in enumerate(kl)] if kind == "continued" else kl
    assert lva.lva_packed_workspace_bytes(len(ql), hq, hk, d, sum(ql), sum(kl)) == 0       # no parts
    q, k, v = inputs(dev, hq + d, sum(ql), sum(kl), hq, hk, d)
    if kind == "growing":
        # scores that outgrow the reference by far more than 2^8, again and again in an item
        for i in range(1, 8):
            k[i * 128::1024] *= 1 + i
        for start in np.cumsum([0] + kl)[:-1]:
            k[start + 900:start + 950] *= 8
    o, lse = run(lva, q, k, v, cu(ql), cu(kl), d ** -0.5, causal)
    assert lva.lva_device_error() == (0, 0)
    check_rows(q, k, v, o, lse, ql, kl, float(np.float32(d ** -0.5)), causal, hq + d)
    # bit for bit the same again, whichever thread block takes which item
    o2, lse2 = run(lva, q, k, v, cu(ql), cu(kl), d ** -0.5, causal)
    assert np.array_equal(bits(o), bits(o2)) and np.array_equal(bits(lse), bits(lse2))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hk,d", [(1, 1, 128), (10, 2, 64), (8, 2, 128)])
@pytest.mark.parametrize("name", list(LONG))
def test_long_key_ranges_without_a_workspace(name, hq, hk, d, causal):
    # the C call with a null workspace: every tile whole
    import block_sparse_attention_lva_b200 as lva
    from block_sparse_attention_lva_b200 import _binding as lb
    dev = require_gpu()
    ql, kl = LONG[name]
    q, k, v = inputs(dev, sum(name.encode()) + hq + d, sum(ql), sum(kl), hq, hk, d)
    o = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=dev)
    lse = torch.full((hq, sum(ql)), float("nan"), device=dev)
    cq, ck = (torch.tensor(cu(x), dtype=torch.int32, device=dev) for x in (ql, kl))
    p = lb._PACKED.pack(len(ql), hq, hk, d, int(causal), d ** -0.5, sum(ql), sum(kl), hq * d, d, hk * d, d, hk * d, d, hq * d, d)
    vp = lambda t: ctypes.c_void_p(t.data_ptr())
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert lb.lib.lva_packed_attn(p, vp(q), vp(k), vp(v), vp(o), vp(lse), vp(cq), vp(ck), None, 0, stream) == 0
    torch.cuda.synchronize()
    assert lva.lva_device_error() == (0, 0)
    compare(q, k, v, o, lse, cu(ql), cu(kl), float(np.float32(d ** -0.5)), causal)
