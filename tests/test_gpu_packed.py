"""Packed-sequence attention (``lva_packed_attn``) against the float64 oracle: ragged lengths
from none to several key blocks, grouped heads, strided views, buffers with anything between
the sequences, bad length lists, streams and graphs."""
import numpy as np
import pytest
import torch

from oracle.packed import packed_attention
from tests.context_helpers import tolerances
from tests.gpu_helpers import bits, require_gpu

pytestmark = pytest.mark.gpu


def run(lva, q, k, v, cu_q, cu_k, scale, causal, fill=float("nan")):
    dev = q.device
    o = torch.full(q.shape, fill, dtype=torch.bfloat16, device=dev)
    lse = torch.full((q.shape[1], q.shape[0]), fill, dtype=torch.float32, device=dev)
    cq, ck = (torch.tensor(x, dtype=torch.int32, device=dev) for x in (cu_q, cu_k))
    lva.lva_packed_attn(q, k, v, o, lse, cq, ck, scale, causal=causal)
    torch.cuda.synchronize()
    return o, lse


def compare(q, k, v, o, lse, cu_q, cu_k, scale, causal):
    o_ref, lse_ref, mag = packed_attention(q.cpu(), k.cpu(), v.cpu(), cu_q, cu_k, scale, causal)
    og, lg = o.double().cpu().numpy(), lse.double().cpu().numpy()
    inside = ~np.isnan(lse_ref[0])
    # tokens in no sequence are left as they were (NaN from `run`)
    assert np.isnan(og[~inside]).all() and np.isnan(lg[:, ~inside]).all()
    fin = lambda x: x[torch.from_numpy(np.isfinite(x.double().cpu().numpy()).all(axis=(1, 2)))]
    tol_o, tol_l = tolerances(fin(q.cpu()), fin(k.cpu()), scale, mag[inside], o_ref[inside])
    bad = np.abs(og[inside] - o_ref[inside]) > tol_o
    assert not np.isnan(og[inside]).any()
    assert not bad.any(), (bad.sum(), np.abs(og[inside] - o_ref[inside]).max(), np.argwhere(bad)[:4])
    empty = np.isneginf(lse_ref[:, inside])
    assert np.array_equal(np.isneginf(lg[:, inside]), empty)
    diff = np.abs(lg[:, inside] - lse_ref[:, inside])[~empty]
    assert diff.size == 0 or diff.max() <= tol_l, (diff.max(), tol_l)


def make(g, tq, tk, hq, hk, d, dev):
    n = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to(dev)
    return n(tq, hq, d), n(tk, hk, d), n(tk, hk, d)


def cu(lens, start=0):
    return [start + sum(lens[:i]) for i in range(len(lens) + 1)]


# (query lengths, key lengths): one token; tile edges; empty sequences and empty sides; more
# queries than keys (rows without keys); one past and one short of a key block
LENGTHS = {
    "one_token": ([1], [1]),
    "short": ([17, 1, 40, 5], [17, 1, 40, 5]),
    "edges": ([127, 128, 129, 1, 0, 2], [127, 128, 129, 1, 0, 2]),
    "blocks": ([300, 257], [300, 257]),
    "continued": ([1, 7, 0, 33, 130], [300, 129, 20, 33, 256]),
    "more_queries": ([200, 50, 3], [70, 0, 2]),
    "no_queries": ([0, 4, 0], [9, 128, 0]),
    "no_keys": ([5, 129], [0, 0]),
}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hk,d", [(4, 2, 64), (3, 3, 128), (5, 1, 64), (6, 2, 128), (8, 1, 128)])
@pytest.mark.parametrize("name", list(LENGTHS))
def test_matches_oracle(name, hq, hk, d, causal):
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    ql, kl = LENGTHS[name]
    g = torch.Generator().manual_seed(sum(name.encode()) + hq + d)
    q, k, v = make(g, sum(ql), sum(kl), hq, hk, d, dev)
    o, lse = run(lva, q, k, v, cu(ql), cu(kl), d ** -0.5, causal)
    assert lva.lva_device_error() == (0, 0)
    compare(q, k, v, o, lse, cu(ql), cu(kl), float(np.float32(d ** -0.5)), causal)


@pytest.mark.parametrize("hq,hk", [(7, 1), (12, 1), (48, 1), (100, 1), (128, 1)])
def test_group_sizes(hq, hk):
    # groups that do not divide the 128-row tile, up to the whole tile
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    ql, kl = [19, 2, 40], [150, 2, 40]
    q, k, v = make(torch.Generator().manual_seed(hq), sum(ql), sum(kl), hq, hk, 64, dev)
    o, lse = run(lva, q, k, v, cu(ql), cu(kl), 0.125, True)
    compare(q, k, v, o, lse, cu(ql), cu(kl), 0.125, True)


# Few tokens against long key ranges: the tiles are cut into parts along the keys
LONG = {
    "one_token": ([1], [8000]),
    "tokens": ([64, 1, 3], [5000, 900, 131]),
    "short_and_long": ([130, 0, 300, 1], [130, 700, 3333, 6]),
    "continued_prompt": ([700], [2700]),
    "one_long_of_many": ([1] * 30, [50] * 29 + [9000]),
    "uneven": ([40, 1, 0, 3], [2000, 9001, 700, 5]),
    "more_queries": ([700, 20], [600, 2000]),
}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hk,d", [(1, 1, 128), (10, 2, 64), (8, 2, 128)])
@pytest.mark.parametrize("name", list(LONG))
def test_parts_along_the_keys(name, hq, hk, d, causal):
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    ql, kl = LONG[name]
    assert lva.lva_packed_workspace_bytes(len(ql), hq, hk, d, sum(ql), sum(kl) + 70) > 0
    g = torch.Generator().manual_seed(sum(name.encode()) + hq + d)
    q, k, v = make(g, sum(ql), sum(kl) + 70, hq, hk, d, dev)
    k[sum(kl):] = float("nan")
    v[sum(kl):] = float("nan")
    o, lse = run(lva, q, k, v, cu(ql), cu(kl), d ** -0.5, causal)
    assert lva.lva_device_error() == (0, 0)
    compare(q, k, v, o, lse, cu(ql), cu(kl), float(np.float32(d ** -0.5)), causal)
    # the caller's own workspace (its contents do not matter), and none at all through the C call
    ws = torch.full((lva.lva_packed_workspace_bytes(len(ql), hq, hk, d, *[x.shape[0] for x in (q, k)]),), 0xff, dtype=torch.uint8, device=dev)
    o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
    cq, ck = (torch.tensor(x, dtype=torch.int32, device=dev) for x in (cu(ql), cu(kl)))
    lva.lva_packed_attn(q, k, v, o2, lse2, cq, ck, d ** -0.5, causal=causal, workspace=ws)
    torch.cuda.synchronize()
    assert np.array_equal(bits(o2), bits(o)) and np.array_equal(bits(lse2), bits(lse))


def test_parts_with_refused_lengths():
    # a list that falls may count more tiles than the totals allow: nothing is written past the
    # workspace (its end is checked), the sequences are reported
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    q, k, v = make(torch.Generator().manual_seed(3), 128, 4000, 1, 1, 64, dev)
    cq = torch.tensor([0, 128] * 20, dtype=torch.int32, device=dev)
    ck = torch.tensor([0, 4000] * 20, dtype=torch.int32, device=dev)
    n = lva.lva_packed_workspace_bytes(39, 1, 1, 64, 128, 4000)
    assert n > 0
    ws = torch.full((n + 4096,), 7, dtype=torch.uint8, device=dev)
    o, lse = torch.zeros_like(q), torch.zeros((1, 128), device=dev)
    lva.lva_packed_attn(q, k, v, o, lse, cq, ck, 0.1, workspace=ws)
    torch.cuda.synchronize()
    assert lva.lva_device_error()[0] == 1
    assert (ws[n:] == 7).all()


def test_many_sequences():
    # more sequences than one round of the warp's search covers, many of them empty
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    rng = np.random.default_rng(5)
    ql = [int(x) for x in rng.integers(0, 4, 1500)]
    kl = [a + int(x) for a, x in zip(ql, rng.integers(0, 5, 1500))]
    q, k, v = make(torch.Generator().manual_seed(8), sum(ql), sum(kl), 4, 2, 64, dev)
    o, lse = run(lva, q, k, v, cu(ql), cu(kl), 0.125, True)
    assert lva.lva_device_error() == (0, 0)
    compare(q, k, v, o, lse, cu(ql), cu(kl), 0.125, True)


@pytest.mark.parametrize("causal", [True, False])
def test_anything_between_and_behind_the_sequences(causal):
    # tokens in no sequence hold NaN and infinity: before the first, behind the last
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    ql, kl = [30, 1, 129], [30, 200, 140]
    q, k, v = make(torch.Generator().manual_seed(9), 9 + sum(ql) + 140, 5 + sum(kl) + 140, 4, 2, 128, dev)
    cq, ck = cu(ql, 9), cu(kl, 5)
    for t, c in ((q, cq), (k, ck), (v, ck)):
        t[:c[0]] = float("nan")
        t[c[-1]:] = float("nan")
        t[c[-1] + 3:] = float("inf")
    o, lse = run(lva, q, k, v, cq, ck, 0.09, causal)
    compare(q, k, v, o, lse, cq, ck, float(np.float32(0.09)), causal)


def test_masked_keys_of_a_sequence_may_be_nan():
    # K of a causally unseen key never matters (its V has to be finite)
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    q, k, v = make(torch.Generator().manual_seed(10), 64, 64, 2, 1, 64, dev)
    k2 = k.clone()
    k2[40:] = float("nan")
    a, la = run(lva, q, k, v, [0, 64], [0, 64], 0.125, True)
    b, lb = run(lva, q, k2, v, [0, 64], [0, 64], 0.125, True)
    assert np.array_equal(bits(a[:40]), bits(b[:40])) and np.array_equal(bits(la[:, :40]), bits(lb[:, :40]))
    assert torch.isnan(b[40:]).all() and torch.isnan(lb[:, 40:]).all()


def test_growing_scores():
    # later key blocks outgrow the earlier ones by far more than 2^8: the reference moves
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    q, k, v = make(torch.Generator().manual_seed(11), 520, 520, 2, 2, 128, dev)
    k[128:256] *= 8
    k[384:] *= 16
    o, lse = run(lva, q, k, v, [0, 520], [0, 520], 128 ** -0.5, True)
    compare(q, k, v, o, lse, [0, 520], [0, 520], float(np.float32(128 ** -0.5)), True)


def test_strided_views_of_a_fused_projection():
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    hq, hk, d, ql = 6, 2, 64, [33, 140]
    g = torch.Generator().manual_seed(12)
    qkv = torch.randn((sum(ql), hq + 2 * hk, d), generator=g).to(torch.bfloat16).to(dev)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    kh = k.transpose(0, 1).contiguous().transpose(0, 1)          # heads outermost in memory
    ref, lref = run(lva, q.contiguous(), k.contiguous(), v.contiguous(), cu(ql), cu(ql), 0.125, True)
    o8 = torch.full((sum(ql), hq, d + 8), 7.0, dtype=torch.bfloat16, device=dev)   # rows on 16-byte boundaries only
    lse = torch.empty((hq, sum(ql)), dtype=torch.float32, device=dev)
    c = torch.tensor(cu(ql), dtype=torch.int32, device=dev)
    lva.lva_packed_attn(q, kh, v, o8[:, :, 8:], lse, c, c, 0.125)
    torch.cuda.synchronize()
    assert np.array_equal(bits(o8[:, :, 8:]), bits(ref)) and np.array_equal(bits(lse), bits(lref))
    assert (o8[:, :, :8] == 7.0).all()


def test_keys_past_32_bit_offsets():
    # the second sequence's keys start past 2^31 elements of the buffer
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    hk, d, tk = 8, 128, 2_200_000
    k = torch.zeros((tk, hk, d), dtype=torch.bfloat16, device=dev)
    g = torch.Generator().manual_seed(13)
    q, ks, vs = make(g, 40, 300, 8, hk, d, dev)
    k[tk - 300:] = ks
    v = k.clone()
    v[tk - 300:] = vs
    cq, ck = [0, 40], [tk - 300, tk]
    o, lse = run(lva, q, k, v, cq, ck, 0.09, True)
    small, lsmall = run(lva, q, ks, vs, [0, 40], [0, 300], 0.09, True)
    assert np.array_equal(bits(o), bits(small)) and np.array_equal(bits(lse), bits(lsmall))


@pytest.mark.parametrize("bad", ["falls", "past_end", "negative", "keys_fall"])
def test_bad_lengths_are_reported_and_skipped(bad):
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    q, k, v = make(torch.Generator().manual_seed(14), 100, 100, 2, 1, 64, dev)
    cq, ck = [0, 30, 60, 100], [0, 30, 60, 100]
    if bad == "falls":
        cq = [0, 30, 20, 100]
    elif bad == "past_end":
        cq = [0, 30, 60, 1 << 30]
    elif bad == "negative":
        ck = [0, -5, 60, 100]
    else:
        ck = [0, 30, 90, 80]
    o, lse = run(lva, q, k, v, cq, ck, 0.125, True)
    status, detail = lva.lva_device_error()
    assert status == 1 and 0 <= detail < 3
    assert lva.lva_device_error() == (0, 0)
    if bad == "past_end":                                     # the sequences before it are whole
        compare(q[:60], k[:60], v[:60], o[:60], lse[:, :60], [0, 30, 60], [0, 30, 60], 0.125, True)
        assert torch.isnan(o[60:]).all()


def test_streams_and_graph():
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    ql = [70, 300, 9]
    q, k, v = make(torch.Generator().manual_seed(15), sum(ql), sum(ql), 4, 2, 128, dev)
    ref, lref = run(lva, q, k, v, cu(ql), cu(ql), 0.09, True)
    c = torch.tensor(cu(ql), dtype=torch.int32, device=dev)
    outs = [(torch.zeros_like(q), torch.zeros_like(lref)) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for st, (o, lse) in zip(streams, outs):
            with torch.cuda.stream(st):
                lva.lva_packed_attn(q, k, v, o, lse, c, c, 0.09)
    torch.cuda.synchronize()
    for o, lse in outs:
        assert np.array_equal(bits(o), bits(ref)) and np.array_equal(bits(lse), bits(lref))
    # captured once, replayed on new inputs and lengths
    o, lse = outs[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lva.lva_packed_attn(q, k, v, o, lse, c, c, 0.09)
    new = [100, 1, sum(ql) - 101]
    c.copy_(torch.tensor(cu(new), dtype=torch.int32))
    q.copy_(q.flip(0))
    o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    compare(q, k, v, o, lse, cu(new), cu(new), float(np.float32(0.09)), True)
