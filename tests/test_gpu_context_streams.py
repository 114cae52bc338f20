"""The packed and cached attention calls, the append and the eviction on streams of their own,
back to back over one workspace, and captured into graphs."""
import numpy as np
import pytest
import torch

from tests.gpu_helpers import bits, require_gpu
from tests.test_gpu_context_cache import Case, i32, normal

pytestmark = pytest.mark.gpu

SMALL = (7, 1, 8, 2, 128, 400, 900, [900, 5, 0, 333, 64, 800, 700])
OTHER = (3, 4, 12, 4, 64, 3000, 700, [4, 700, 65])


def same(a, b):
    return all(np.array_equal(bits(x), bits(y)) for x, y in zip(a, b) if x is not None)


def test_two_streams_at_once():
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    cases = [Case(dev, 5, *SMALL, True), Case(dev, 6, *OTHER, True)]
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
    for ref, out in zip(refs, outs):
        assert all(same(ref, got) for got in out)


def test_one_workspace_for_calls_in_turn():
    # a call starts to write the workspace only when the call before has read its last part
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    cases = [Case(dev, 5, *SMALL, True), Case(dev, 6, *OTHER, True), Case(dev, 7, 5, 1, 10, 2, 128, 5000, 70, [1, 2, 3, 70, 9], False)]
    refs = [c.run(lva) for c in cases]
    ws = max((c.workspace(lva) for c in cases), key=lambda x: x.numel())
    outs = [[c.outputs() for _ in range(8)] for c in cases]
    torch.cuda.synchronize()
    for i in range(8):
        for c, out in zip(cases, outs):
            o, lse, w = out[i]
            lva.lva_shared_prefix_attn(c.q, c.pk, c.pv, c.kc, c.vc, c.lens_t, o, lse, ws, c.scale, weight=w)
    torch.cuda.synchronize()
    for ref, out in zip(refs, outs):
        assert all(same(ref, got) for got in out)


def test_packed_parts_captured_and_on_two_streams():
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    g = torch.Generator().manual_seed(9)
    ql, kl = [64, 0, 3], [8000, 100, 5000]
    q, k, v = normal(g, dev, 67, 8, 128), normal(g, dev, 13100, 2, 128), normal(g, dev, 13100, 2, 128)
    cq, ck = i32(np.cumsum([0] + ql).tolist(), dev), i32(np.cumsum([0] + kl).tolist(), dev)
    n = lva.lva_packed_workspace_bytes(3, 8, 2, 128, 67, 13100)
    assert n > 0

    def outputs():
        return torch.full_like(q, float("nan")), torch.full((8, 67), float("nan"), device=dev)

    def run(out, ws=None):
        lva.lva_packed_attn(q, k, v, *out, cq, ck, 0.09, workspace=ws)
        return out

    ref = run(outputs())
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.empty(n, dtype=torch.uint8, device=dev), None]          # one's own, and the allocator's
    outs = [[outputs() for _ in range(6)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(6):
        for st, ws, out in zip(streams, spaces, outs):
            with torch.cuda.stream(st):
                run(out[i], ws)
    torch.cuda.synchronize()
    assert all(same(ref, got) for out in outs for got in out)

    graphs, caught = [], [outputs(), outputs()]
    for out, ws in zip(caught, spaces):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            run(out, ws)
    # other lengths than those at the capture, with fewer parts and more
    for new in ([64, 0, 3], [1, 2, 64], [0, 0, 67]):
        cq.copy_(i32(np.cumsum([0] + new).tolist(), dev))
        ref = run(outputs())
        for graph, out in zip(graphs, caught):
            for x in out:
                x.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert same(ref, out)
    assert lva.lva_device_error() == (0, 0)


def test_a_captured_step():
    # append, attention with weights and eviction captured once; a run of replays leaves what
    # the same calls leave one by one
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    g = torch.Generator().manual_seed(12)
    B, T, hq, hk, d, lp, cap, budget = 5, 2, 6, 2, 64, 700, 40, 33
    pk, pv = normal(g, dev, lp, hk, d), normal(g, dev, lp, hk, d)
    feed = [(normal(g, dev, B, T, hq, d), normal(g, dev, B, T, hk, d), normal(g, dev, B, T, hk, d)) for _ in range(25)]
    ws = torch.empty(lva.lva_shared_prefix_workspace_bytes(B, T, hq, hk, d, lp, cap, True), dtype=torch.uint8, device=dev)

    class State:
        def __init__(self):
            self.q, self.kn, self.vn = (x.clone() for x in feed[0])
            self.kc, self.vc = (torch.zeros((B, hk, cap, d), dtype=torch.bfloat16, device=dev) for _ in range(2))
            self.w = torch.zeros((B, hk, cap), device=dev)
            self.lens = i32([0, 3, 33, 20, 7], dev)
            self.kept = torch.zeros((B, hk, budget), dtype=torch.int32, device=dev)
            self.o, self.lse = torch.zeros_like(self.q), torch.zeros((B, hq, T), device=dev)

        def step(self):
            lva.lva_append_cache(self.kn, self.vn, self.kc, self.vc, self.w, self.lens, self.lens)
            lva.lva_shared_prefix_attn(self.q, pk, pv, self.kc, self.vc, self.lens, self.o, self.lse, ws, 0.125, weight=self.w)
            lva.lva_evict_cache(self.kc, self.vc, self.w, self.lens, self.kc, self.vc, self.w, self.lens, self.kept, budget, 1, 4)

        def feed(self, new):
            for x, y in zip((self.q, self.kn, self.vn), new):
                x.copy_(y)

        def all(self):
            return [x.clone() for x in (self.o, self.lse, self.kc, self.vc, self.w, self.lens, self.kept)]

    eager, caught = State(), State()
    want = []
    for new in feed:
        eager.feed(new)
        eager.step()
        want.append(eager.all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught.step()
    for i, new in enumerate(feed):
        caught.feed(new)
        graph.replay()
        torch.cuda.synchronize()
        assert same(want[i], caught.all()), i
    assert lva.lva_device_error() == (0, 0)
    assert caught.lens.tolist() == [budget] * 5


@pytest.mark.parametrize("steps", [1, 40])
def test_append_and_evict_on_two_streams(steps):
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    g = torch.Generator().manual_seed(steps)
    B, hk, d, cap, budget = 3, 3, 128, 1100, 1050
    kn, vn = normal(g, dev, B, steps, hk, d), normal(g, dev, B, steps, hk, d)
    base = normal(g, dev, B, hk, cap, d), normal(g, dev, B, hk, cap, d), torch.rand((B, hk, cap), generator=g).to(dev)
    lens = [1060, 0, 1049]

    def state():
        return [x.clone() for x in base] + [i32(lens, dev), torch.zeros((B, hk, budget), dtype=torch.int32, device=dev)]

    def run(s):
        kc, vc, w, n, kept = s
        lva.lva_append_cache(kn, vn, kc, vc, w, n, n)
        lva.lva_evict_cache(kc, vc, w, n, kc, vc, w, n, kept, budget, 4, 100)

    ref = state()
    run(ref)
    states = [state() for _ in range(8)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i, s in enumerate(states):
        with torch.cuda.stream(streams[i % 2]):
            run(s)
    torch.cuda.synchronize()
    assert lva.lva_device_error() == (0, 0)
    assert all(same(ref, s) for s in states)
    assert ref[3].tolist() == [min(n + steps, budget) for n in lens]
