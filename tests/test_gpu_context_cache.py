"""Shared-prefix attention, the append and the eviction (``lva_shared_prefix_attn``,
``lva_append_cache``, ``lva_evict_cache``) against the float64 oracle, alone and in a run as a
rollout uses them."""
import numpy as np
import pytest
import torch

from oracle.packed import evict_kept, packed_attention, shared_prefix_attention
from tests.context_helpers import tolerances
from tests.gpu_helpers import bits, require_gpu

pytestmark = pytest.mark.gpu


def normal(g, dev, *shape):
    return torch.randn(shape, generator=g).to(torch.bfloat16).to(dev)


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


class Case:
    """Inputs of one shared-prefix call; dead cache entries hold NaN."""

    def __init__(self, dev, seed, B, T, hq, hk, d, lp, cap, lens, weights):
        g = torch.Generator().manual_seed(seed)
        self.dims = (B, T, hq, hk, d, lp, cap)
        self.lens, self.lens_t = lens, i32(lens, dev)
        self.q = normal(g, dev, B, T, hq, d)
        self.pk, self.pv = (normal(g, dev, lp, hk, d), normal(g, dev, lp, hk, d)) if lp else (None, None)
        self.kc, self.vc = normal(g, dev, B, hk, cap, d), normal(g, dev, B, hk, cap, d)
        for b, n in enumerate(lens):
            if 0 <= n <= cap:
                self.kc[b, :, n:] = float("nan")
                self.vc[b, :, n:] = float("nan")
        self.w0 = torch.rand((B, hk, cap), generator=g).to(dev) if weights else None
        self.scale = float(np.float32(d ** -0.5))

    def outputs(self):
        B, T, hq, hk, d, lp, cap = self.dims
        dev = self.q.device
        return (torch.full((B, T, hq, d), float("nan"), dtype=torch.bfloat16, device=dev),
                torch.full((B, hq, T), float("nan"), device=dev), self.w0.clone() if self.w0 is not None else None)

    def workspace(self, lva):
        B, T, hq, hk, d, lp, cap = self.dims
        n = lva.lva_shared_prefix_workspace_bytes(B, T, hq, hk, d, lp, cap, self.w0 is not None)
        assert n >= 0
        # what a workspace holds between calls has no meaning
        return torch.full((max(n, 16),), 0xff, dtype=torch.uint8, device=self.q.device)

    def run(self, lva, ws=None):
        o, lse, w = self.outputs()
        ws = self.workspace(lva) if ws is None else ws
        lva.lva_shared_prefix_attn(self.q, self.pk, self.pv, self.kc, self.vc, self.lens_t, o, lse, ws, self.scale, weight=w)
        torch.cuda.synchronize()
        return o, lse, w

    def compare(self, o, lse, w, lens=None):
        B, T, hq, hk, d, lp, cap = self.dims
        lens = self.lens if lens is None else lens
        none = torch.zeros((0, hk, d))
        pk, pv = (self.pk.cpu(), self.pv.cpu()) if lp else (none, none)
        o_ref, lse_ref, mag, w_ref = shared_prefix_attention(self.q.cpu(), pk, pv, self.kc.cpu(), self.vc.cpu(), lens, self.scale)
        live = torch.cat([pk.reshape(-1, d)] + [self.kc[b, :, :n].reshape(-1, d).cpu() for b, n in enumerate(lens)])
        tol_o, tol_l = tolerances(self.q.cpu(), live, self.scale, mag, o_ref)
        og, lg = o.double().cpu().numpy(), lse.double().cpu().numpy()
        assert not np.isnan(og).any()
        bad = np.abs(og - o_ref) > tol_o
        assert not bad.any(), (bad.sum(), np.abs(og - o_ref).max(), np.argwhere(bad)[:4])
        empty = np.isneginf(lse_ref)
        assert np.array_equal(np.isneginf(lg), empty)
        diff = np.abs(lg[~empty] - lse_ref[~empty])
        assert diff.size == 0 or diff.max() <= 2 * tol_l, (diff.max(), tol_l)       # a part's LSE and the join
        if w is not None:
            # a weight is exp of a score less a row's LSE, both within their bounds; added in fp32
            wg, base = w.double().cpu().numpy(), self.w0.double().cpu().numpy()
            tol_w = 4 * tol_l * w_ref + 2.0 ** -22 * (base + w_ref)
            bad = np.abs(wg - base - w_ref) > tol_w
            assert not bad.any(), (bad.sum(), np.abs(wg - base - w_ref).max(), np.argwhere(bad)[:4])
            for b, n in enumerate(lens):
                assert np.array_equal(wg[b, :, n:], base[b, :, n:])


# (B, T, Hq, Hkv, d, prefix, capacity, lens)
SHAPES = {
    "one": (1, 1, 1, 1, 64, 1, 1, [1]),
    "pair": (2, 1, 4, 2, 64, 100, 64, [3, 40]),
    "no_prefix": (3, 1, 4, 1, 128, 0, 200, [1, 64, 200]),
    "no_cache": (3, 1, 4, 4, 128, 129, 0, [0, 0, 0]),
    "empty_caches": (3, 1, 2, 2, 64, 65, 70, [0, 70, 0]),
    "nothing_seen": (2, 2, 2, 1, 128, 0, 9, [0, 1]),
    "edges": (6, 1, 8, 2, 128, 128, 257, [63, 64, 65, 128, 129, 257]),
    "steps": (4, 4, 12, 12, 128, 300, 150, [2, 4, 65, 150]),
    "steps_over_tiles": (3, 3, 5, 1, 64, 31, 300, [65, 66, 130]),
    "rows_16": (2, 2, 8, 1, 128, 70, 90, [90, 33]),
    "rows_17": (2, 1, 17, 1, 64, 70, 90, [90, 33]),
    "rows_32": (2, 4, 8, 1, 128, 70, 190, [190, 133]),
    "rows_40": (2, 5, 8, 1, 128, 70, 190, [190, 133]),
    "rows_64": (2, 64, 2, 2, 64, 70, 190, [190, 63]),
    "long_prefix": (5, 1, 10, 2, 128, 5000, 70, [1, 2, 3, 70, 9]),
    "long_cache": (2, 1, 4, 1, 128, 3, 30000, [29999, 17]),
    # batches of at most 32 rows: the prefix in the caches' list
    "list_rows_20": (2, 5, 16, 8, 64, 1097, 518, [219, 500]),
    "list_one_head": (3, 2, 1, 1, 128, 500, 700, [2, 700, 65]),
    "list_empty_caches": (2, 1, 4, 4, 64, 300, 50, [0, 0]),
    "list_rows_32": (4, 1, 32, 4, 128, 90, 130, [64, 0, 129, 130]),
    "list_many_heads": (1, 4, 16, 16, 128, 65, 64, [4]),
    "many_planes": (83, 1, 60, 12, 64, 462, 24, [(5 * i) % 25 for i in range(83)]),
    "many_sequences": (150, 1, 2, 1, 64, 20, 80, [(7 * i) % 81 for i in range(150)]),
}


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("name", list(SHAPES))
def test_shared_prefix_matches_oracle(name, weights):
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    *dims, lens = SHAPES[name]
    c = Case(dev, sum(name.encode()), *dims, lens, weights)
    out = c.run(lva)
    assert lva.lva_device_error() == (0, 0)
    c.compare(*out)


def test_shared_prefix_is_repeatable_and_split_independent():
    # the same call twice, bit for bit; and a sequence's result does not depend on the others
    # in the batch beyond rounding (its parts are cut elsewhere)
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    c = Case(dev, 3, 7, 1, 8, 2, 128, 400, 900, [900, 5, 0, 333, 64, 800, 700], True)
    a, b = c.run(lva), c.run(lva)
    assert all(np.array_equal(bits(x), bits(y)) for x, y in zip(a, b))


def test_growing_scores_move_the_reference():
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    c = Case(dev, 5, 2, 1, 8, 2, 128, 300, 400, [400, 390], True)
    c.kc[:, :, 100:] *= 6
    c.kc[:, :, 300:] *= 3
    c.pk[128:] *= 5
    c.compare(*c.run(lva))


def test_strided_queries_and_prefix():
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    B, T, hq, hk, d, lp, cap = 3, 2, 4, 2, 64, 90, 80
    c = Case(dev, 6, B, T, hq, hk, d, lp, cap, [80, 2, 33], False)
    ref = c.run(lva)
    fused = torch.full((B, T, hq + 2 * hk, d), float("nan"), dtype=torch.bfloat16, device=dev)
    fused[:, :, :hq] = c.q
    c.q = fused[:, :, :hq]
    kv = torch.stack([c.pk, c.pv], dim=1)                    # [Lp, 2, Hkv, d]
    c.pk, c.pv = kv[:, 0], kv[:, 1]
    o = torch.full((B, T, hq, 2 * d), 3.0, dtype=torch.bfloat16, device=dev)
    lse = torch.empty_like(ref[1])
    lva.lva_shared_prefix_attn(c.q, c.pk, c.pv, c.kc, c.vc, c.lens_t, o[..., d:], lse, c.workspace(lva), c.scale)
    torch.cuda.synchronize()
    assert np.array_equal(bits(o[..., d:]), bits(ref[0])) and np.array_equal(bits(lse), bits(ref[1]))
    assert (o[..., :d] == 3.0).all()


@pytest.mark.parametrize("bad", [-1, 81, 1 << 30])
def test_bad_cache_length_is_reported_and_counts_as_none(bad):
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    c = Case(dev, 7, 3, 1, 4, 2, 64, 50, 80, [80, bad, 20], True)
    out = c.run(lva)
    assert lva.lva_device_error() == (1, 1)
    c.compare(*out, lens=[80, 0, 20])


def test_cache_past_32_bit_offsets():
    # the last sequence's cache starts past 2^31 elements
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    B, hk, d, cap = 9, 8, 128, 260_000
    g = torch.Generator().manual_seed(8)
    kc = torch.empty((B, hk, cap, d), dtype=torch.bfloat16, device=dev)
    vc = torch.empty_like(kc)
    lens = [0] * (B - 1) + [1000]
    ks, vs = normal(g, dev, hk, 1000, d), normal(g, dev, hk, 1000, d)
    lva.lva_append_cache(ks.transpose(0, 1).expand(B, -1, -1, -1)[-1:], vs.transpose(0, 1)[None], kc[-1:], vc[-1:], None,
                         i32([0], dev), i32([0], dev))
    assert np.array_equal(bits(kc[-1, :, :1000]), bits(ks)) and np.array_equal(bits(vc[-1, :, :1000]), bits(vs))
    q = normal(g, dev, B, 1, hk, d)
    o, lse = torch.empty_like(q), torch.empty((B, hk, 1), device=dev)
    ws = torch.empty(lva.lva_shared_prefix_workspace_bytes(B, 1, hk, hk, d, 0, cap), dtype=torch.uint8, device=dev)
    lva.lva_shared_prefix_attn(q, None, None, kc, vc, i32(lens, dev), o, lse, ws, 0.09)
    torch.cuda.synchronize()
    assert lva.lva_device_error() == (0, 0)
    assert (o[:-1] == 0).all() and torch.isneginf(lse[:-1]).all()
    o_ref, lse_ref, mag = packed_attention(q[-1].cpu(), ks.transpose(0, 1).cpu(), vs.transpose(0, 1).cpu(), [0, 1], [0, 1000],
                                           float(np.float32(0.09)), True)
    tol_o, tol_l = tolerances(q[-1].cpu(), ks.cpu(), 0.09, mag, o_ref)
    assert (np.abs(o[-1].double().cpu().numpy() - o_ref) <= tol_o).all()
    assert np.abs(lse[-1].cpu().numpy() - lse_ref).max() <= 2 * tol_l


# ---------------------------------------------------------------- append


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,T,hk,d,cap,lens", [
    (3, 1, 2, 64, 9, [0, 8, 4]), (2, 5, 3, 128, 40, [0, 35]), (2, 200, 4, 128, 500, [7, 300]), (1, 0, 1, 64, 4, [3]),
    (70, 1, 8, 128, 5, [i % 5 for i in range(70)]), (2, 7, 12, 64, 60, [50, 3]), (2, 33, 5, 64, 90, [1, 57]),
    (3, 17, 8, 128, 40, [23, 0, 5]), (1, 31, 3, 64, 100, [9]), (2, 1560, 3, 128, 1700, [100, 0]),
])
def test_append(B, T, hk, d, cap, lens, in_place):
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    g = torch.Generator().manual_seed(B + T)
    fused = normal(g, dev, B, T, 2 * hk, d)
    kn, vn = fused[:, :, :hk], fused[:, :, hk:]
    kc, vc = normal(g, dev, B, hk, cap, d), normal(g, dev, B, hk, cap, d)
    w = torch.rand((B, hk, cap), generator=g).to(dev)
    want_k, want_v, want_w = kc.clone(), vc.clone(), w.clone()
    for b, n in enumerate(lens):
        want_k[b, :, n:n + T] = kn[b].transpose(0, 1)
        want_v[b, :, n:n + T] = vn[b].transpose(0, 1)
        want_w[b, :, n:n + T] = 0
    lt = i32(lens, dev)
    out = lt if in_place else torch.full_like(lt, -7)
    lva.lva_append_cache(kn, vn, kc, vc, w, lt, out)
    torch.cuda.synchronize()
    assert lva.lva_device_error() == (0, 0)
    assert out.tolist() == [n + T for n in lens]
    assert in_place or lt.tolist() == lens
    assert np.array_equal(bits(kc), bits(want_k)) and np.array_equal(bits(vc), bits(want_v))
    assert np.array_equal(bits(w), bits(want_w))


@pytest.mark.parametrize("T", [3, 300])
def test_append_to_a_full_cache_is_reported_and_skipped(T):
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    g = torch.Generator().manual_seed(4)
    B, hk, d, cap = 3, 2, 64, T + 5
    lens = [2, 6, 5]
    kn, vn, kc, vc = normal(g, dev, B, T, hk, d), normal(g, dev, B, T, hk, d), normal(g, dev, B, hk, cap, d), normal(g, dev, B, hk, cap, d)
    before = kc.clone()
    lt = i32(lens, dev)
    lva.lva_append_cache(kn, vn, kc, vc, None, lt, lt)
    torch.cuda.synchronize()
    assert lva.lva_device_error() == (3, 1)
    assert lt.tolist() == [2 + T, 6, 5 + T]
    assert np.array_equal(bits(kc[1]), bits(before[1])) and np.array_equal(bits(kc[2, :, 5:]), bits(kn[2].transpose(0, 1)))


# ---------------------------------------------------------------- evict


def weights_like(g, kind, *shape):
    w = torch.exp(2 * torch.randn(shape, generator=g))
    if kind == "ties":
        w = torch.round(w)
    elif kind == "equal":
        w = torch.full(shape, 0.25)
    elif kind == "special":
        r = torch.rand(shape, generator=g)
        for i, x in enumerate([float("nan"), float("inf"), float("-inf"), 0.0, -0.0, -3.0, 1e-42, -1e-42]):
            w[(r > i * 0.08) & (r < (i + 1) * 0.08)] = x
    return w


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "special"])
@pytest.mark.parametrize("B,hk,d,cap,lens,budget,sinks,recent", [
    (3, 2, 64, 160, [150, 90, 101], 100, 4, 16),
    (2, 1, 128, 30, [30, 29], 29, 0, 0),
    (2, 2, 128, 50, [50, 9], 8, 3, 5),
    (1, 3, 64, 40, [40], 1, 0, 0),
    (2, 2, 64, 40, [0, 40], 40, 2, 2),
    (2, 2, 128, 9000, [9000, 5001], 5000, 4, 500),
    (4, 5, 128, 700, [700, 699, 300, 650], 301, 1, 0),
    (1, 2, 64, 640, [640], 400, 3, 100),
    (2, 1, 64, 641, [641, 500], 400, 0, 0),
    (2, 2, 128, 609, [609, 608], 300, 1, 33),
    (1, 2, 64, 1024, [1024], 700, 3, 100),
    (2, 1, 64, 1025, [1025, 701], 700, 0, 0),
    (2, 1, 64, 16384, [16384, 4097], 4096, 1, 1),
    (2, 1, 64, 16385, [16385, 8200], 8199, 7, 0),
    (1, 2, 64, 40000, [39999], 1, 0, 0),
])
def test_evict_matches_oracle(B, hk, d, cap, lens, budget, sinks, recent, kind, in_place):
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    g = torch.Generator().manual_seed(cap + budget + len(kind))
    kc, vc = normal(g, dev, B, hk, cap, d), normal(g, dev, B, hk, cap, d)
    w = weights_like(g, kind, B, hk, cap).to(dev)
    lt = i32(lens, dev)
    if in_place:
        ko, vo, wo, lo = kc, vc, w, lt
    else:
        ko, vo, wo, lo = normal(g, dev, B, hk, cap, d), normal(g, dev, B, hk, cap, d), torch.rand(w.shape).to(dev), torch.full_like(lt, -9)
    kept = torch.full((B, hk, budget), -5, dtype=torch.int32, device=dev)
    k0, v0, w0 = kc.clone(), vc.clone(), w.clone()
    want = [ko.clone(), vo.clone(), wo.clone()]
    want_kept = np.full((B, hk, budget), -1)
    for b, n in enumerate(lens):
        for h in range(hk):
            idx = evict_kept(w0[b, h].cpu().numpy(), n, budget, sinks, recent)
            want_kept[b, h, :len(idx)] = idx
            for dst, src in zip(want, (k0, v0, w0)):
                dst[b, h, :len(idx)] = src[b, h, torch.from_numpy(idx).to(dev)]
    lva.lva_evict_cache(kc, vc, w, lt, ko, vo, wo, lo, kept, budget, sinks, recent)
    torch.cuda.synchronize()
    assert lva.lva_device_error() == (0, 0)
    assert np.array_equal(kept.cpu().numpy(), want_kept)
    assert lo.tolist() == [min(n, budget) for n in lens]
    for got, ref in zip((ko, vo, wo), want):
        assert np.array_equal(bits(got), bits(ref))          # rows past the new length included
    if not in_place:
        assert np.array_equal(bits(kc), bits(k0)) and lt.tolist() == lens


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_bad_length_is_reported_and_left(in_place):
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    g = torch.Generator().manual_seed(2)
    kc, vc, w = normal(g, dev, 3, 2, 20, 64), normal(g, dev, 3, 2, 20, 64), torch.rand((3, 2, 20), generator=g).to(dev)
    lt = i32([20, 21, -4], dev)
    ko, vo, wo = (kc, vc, w) if in_place else (kc.clone(), vc.clone(), w.clone())
    k0 = kc.clone()
    kept = torch.zeros((3, 2, 7), dtype=torch.int32, device=dev)
    lva.lva_evict_cache(kc, vc, w, lt, ko, vo, wo, lt, kept, 7)
    torch.cuda.synchronize()
    status, detail = lva.lva_device_error()
    assert status == 1 and detail in (1, 2)
    assert lt.tolist() == [7, 21, -4] and (kept[1:] == -1).all()
    assert np.array_equal(bits(ko[1:]), bits(k0[1:]))


# ---------------------------------------------------------------- together


def test_a_rollout():
    """Prompt -> shared prefix -> steps of append and attention with weights -> eviction -> on."""
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    g = torch.Generator().manual_seed(21)
    B, hq, hk, d, lp, cap, budget = 4, 8, 2, 128, 333, 48, 30
    scale = float(np.float32(d ** -0.5))
    qkv = normal(g, dev, lp, hq + 2 * hk, d)
    pk, pv = qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    po, plse = torch.empty((lp, hq, d), dtype=torch.bfloat16, device=dev), torch.empty((hq, lp), device=dev)
    cu = i32([0, lp], dev)
    lva.lva_packed_attn(qkv[:, :hq], pk, pv, po, plse, cu, cu, scale)
    o_ref, lse_ref, mag = packed_attention(qkv[:, :hq].cpu(), pk.cpu(), pv.cpu(), [0, lp], [0, lp], scale, True)
    tol_o, tol_l = tolerances(qkv[:, :hq].cpu(), pk.cpu(), scale, mag, o_ref)
    assert (np.abs(po.double().cpu().numpy() - o_ref) <= tol_o).all()

    kc, vc = (torch.full((B, hk, cap, d), float("nan"), dtype=torch.bfloat16, device=dev) for _ in range(2))
    w = torch.full((B, hk, cap), float("nan"), device=dev)
    lens = torch.zeros(B, dtype=torch.int32, device=dev)
    kept = torch.empty((B, hk, budget), dtype=torch.int32, device=dev)
    # the same on the host, in float64, from the definitions
    hk_, hv_, hw_ = ([[np.zeros((0, d)) for _ in range(hk)] for _ in range(B)], [[np.zeros((0, d)) for _ in range(hk)] for _ in range(B)],
                     [[np.zeros(0) for _ in range(hk)] for _ in range(B)])
    o, lse = torch.empty((B, 1, hq, d), dtype=torch.bfloat16, device=dev), torch.empty((B, hq, 1), device=dev)
    for step in range(60):
        T = 3 if step % 20 == 5 else 1
        q, kn, vn = normal(g, dev, B, T, hq, d), normal(g, dev, B, T, hk, d), normal(g, dev, B, T, hk, d)
        ws = torch.empty(lva.lva_shared_prefix_workspace_bytes(B, T, hq, hk, d, lp, cap, True), dtype=torch.uint8, device=dev)
        o, lse = torch.empty_like(q), torch.empty((B, hq, T), device=dev)
        lva.lva_append_cache(kn, vn, kc, vc, w, lens, lens)
        lva.lva_shared_prefix_attn(q, pk, pv, kc, vc, lens, o, lse, ws, scale, weight=w)
        n = lens.tolist()
        wide = lambda rows: torch.stack([torch.stack([torch.from_numpy(np.concatenate([x, np.zeros((cap - len(x), d))])) for x in r]) for r in rows])
        for b in range(B):
            for h in range(hk):
                hk_[b][h] = np.concatenate([hk_[b][h], kn[b, :, h].double().cpu().numpy()])
                hv_[b][h] = np.concatenate([hv_[b][h], vn[b, :, h].double().cpu().numpy()])
                hw_[b][h] = np.concatenate([hw_[b][h], np.zeros(T)])
        o_ref, lse_ref, mag, w_ref = shared_prefix_attention(q.cpu(), pk.cpu(), pv.cpu(), wide(hk_), wide(hv_), n, scale)
        tol_o, tol_l = tolerances(q.cpu(), torch.cat([pk.cpu().reshape(-1, d), wide(hk_).reshape(-1, d)]), scale, mag, o_ref)
        assert (np.abs(o.double().cpu().numpy() - o_ref) <= tol_o).all(), step
        assert np.abs(lse.cpu().numpy() - lse_ref).max() <= 2 * tol_l, step
        for b in range(B):
            for h in range(hk):
                hw_[b][h] = hw_[b][h] + w_ref[b, h, :n[b]]
                got = w[b, h, :n[b]].double().cpu().numpy()
                assert (np.abs(got - hw_[b][h]) <= (4 * tol_l + 2.0 ** -20) * (step + 1) * hw_[b][h] + 1e-12).all(), step
                hw_[b][h] = got                              # further on from what the ranking reads
        if max(n) > cap - 3:
            lva.lva_evict_cache(kc, vc, w, lens, kc, vc, w, lens, kept, budget, 2, 8)
            for b in range(B):
                for h in range(hk):
                    idx = evict_kept(hw_[b][h], n[b], budget, 2, 8)
                    assert kept[b, h, :len(idx)].tolist() == idx.tolist()
                    hk_[b][h], hv_[b][h], hw_[b][h] = hk_[b][h][idx], hv_[b][h][idx], hw_[b][h][idx]
            assert lens.tolist() == [min(x, budget) for x in n]
    assert lva.lva_device_error() == (0, 0)
