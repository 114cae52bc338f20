"""The packed / shared-prefix / eviction oracle is pinned by the dense oracle, by torch's own
softmax attention and by hand-worked examples."""
import numpy as np
import pytest
import torch

from oracle.attention import attention_blocked
from oracle.packed import evict_kept, packed_attention, shared_prefix_attention


def _rand(g, *shape):
    return torch.randn(shape, generator=g, dtype=torch.float64)


def test_one_sequence_is_dense_attention():
    g = torch.Generator().manual_seed(1)
    q, k, v = (_rand(g, 128, 2, 64) for _ in range(3))
    o, lse, _ = packed_attention(q, k, v, [0, 128], [0, 128], 0.125, causal=False)
    plane = lambda x: x.permute(1, 0, 2)[None]
    od, ld = attention_blocked(plane(q), plane(k), plane(v), np.ones((1, 2, 2), dtype=bool), 64, 128, 0.125)
    np.testing.assert_allclose(o.transpose(1, 0, 2), od[0], rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(lse, ld[0], rtol=1e-12)


@pytest.mark.parametrize("n,m", [(5, 5), (3, 9), (9, 3), (1, 7), (4, 0)])
def test_causal_rows_against_torch(n, m):
    g = torch.Generator().manual_seed(n * 16 + m)
    q, k, v = _rand(g, n, 4, 8), _rand(g, m, 2, 8), _rand(g, m, 2, 8)
    scale = float(np.float32(0.3))
    o, lse, mag = packed_attention(q, k, v, [0, n], [0, m], scale, causal=True)
    for h in range(4):
        for i in range(n):
            end = min(m, i + m - n + 1)
            if end <= 0:
                assert (o[i, h] == 0).all() and np.isneginf(lse[h, i]) and (mag[i, h] == 0).all()
                continue
            s = scale * (k[:end, h // 2] @ q[i, h])
            np.testing.assert_allclose(o[i, h], (torch.softmax(s, 0) @ v[:end, h // 2]).numpy(), rtol=1e-11, atol=1e-13)
            np.testing.assert_allclose(lse[h, i], torch.logsumexp(s, 0).item(), rtol=1e-12)


def test_sequences_do_not_meet():
    g = torch.Generator().manual_seed(3)
    q, k, v = _rand(g, 12, 2, 8), _rand(g, 14, 1, 8), _rand(g, 14, 1, 8)
    o, lse, _ = packed_attention(q, k, v, [1, 4, 4, 11], [0, 5, 7, 14], 0.3, causal=True)
    assert np.isnan(o[0]).all() and np.isnan(o[11]).all() and np.isnan(lse[:, [0, 11]]).all()
    one, lone, _ = packed_attention(q[4:11], k[7:14], v[7:14], [0, 7], [0, 7], 0.3, causal=True)
    np.testing.assert_allclose(o[4:11], one, rtol=1e-13)
    np.testing.assert_allclose(lse[:, 4:11], lone, rtol=1e-13)


def test_shared_prefix_is_attention_over_the_joined_keys():
    g = torch.Generator().manual_seed(4)
    B, T, hq, hk, d, lp, cap = 3, 2, 4, 2, 8, 6, 5
    q, pk, pv = _rand(g, B, T, hq, d), _rand(g, lp, hk, d), _rand(g, lp, hk, d)
    kc, vc = _rand(g, B, hk, cap, d), _rand(g, B, hk, cap, d)
    lens = [5, 2, 1]
    o, lse, _, w = shared_prefix_attention(q, pk, pv, kc, vc, lens, 0.4)
    for b, n in enumerate(lens):
        k = torch.cat([pk, kc[b, :, :n].transpose(0, 1)])
        v = torch.cat([pv, vc[b, :, :n].transpose(0, 1)])
        if n >= T:   # then it is the causal continuation of one sequence
            o1, l1, _ = packed_attention(q[b], k, v, [0, T], [0, lp + n], 0.4, causal=True)
            np.testing.assert_allclose(o[b], o1, rtol=1e-12, atol=1e-14)
            np.testing.assert_allclose(lse[b], l1, rtol=1e-12)
        assert (w[b, :, n:] == 0).all()
    # sample 2 holds one entry: its first token sees the prefix alone
    o1, l1, _ = packed_attention(q[2, :1], pk, pv, [0, 1], [0, lp], 0.4, causal=False)
    np.testing.assert_allclose(o[2, :1], o1, rtol=1e-12)
    # probabilities of prefix and cache add up to one per row
    total = w.sum(axis=(1, 2))
    assert (total < B * hq).all() and (total[0] > 0)


def test_evict_by_hand():
    w = np.array([9.0, 1.0, 5.0, 3.0, 5.0, 0.0, np.nan, 2.0, 8.0, 7.0])
    # budget 6: sinks 0, recent 8 9; of 1..7 the three largest: 5 (index 2), 5 (index 4), 3 (index 3)
    assert evict_kept(w, 10, 6, 1, 2).tolist() == [0, 2, 3, 4, 8, 9]
    assert evict_kept(w, 10, 4, 1, 2).tolist() == [0, 2, 8, 9]        # the tie goes to the lower index
    assert evict_kept(w, 10, 9, 1, 2).tolist() == [0, 1, 2, 3, 4, 5, 7, 8, 9]   # NaN leaves first
    assert evict_kept(w, 4, 6, 1, 2).tolist() == [0, 1, 2, 3]
    assert evict_kept(w, 10, 3, 0, 3).tolist() == [7, 8, 9]
