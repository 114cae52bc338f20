"""Argument checks of the packed, shared-prefix, append and evict calls: every bad call is
refused on the host, before anything reaches a GPU (no GPU needed)."""
import ctypes
import math

import pytest
import torch

import block_sparse_attention_lva_b200 as lva
from block_sparse_attention_lva_b200 import _binding as lb

OK, INVALID, UNSUPPORTED, CAPACITY = 0, 1, 2, 3


def packed_bytes(p):
    return lb._PACKED.pack(*[p[k] for k in ("num_seqs", "q_heads", "kv_heads", "d", "causal", "scale", "total_q", "total_k")],
                           *[p[f"{t}_{s}_stride"] for t in "qkvo" for s in ("token", "head")])


def packed(q=16, k=16, v=16, o=16, lse=4, cu_q=4, cu_k=4, ws=None, ws_bytes=0, **kw):
    p = dict(num_seqs=2, q_heads=4, kv_heads=2, d=64, causal=1, scale=0.125, total_q=100, total_k=100,
             q_token_stride=256, q_head_stride=64, k_token_stride=128, k_head_stride=64, v_token_stride=128,
             v_head_stride=64, o_token_stride=256, o_head_stride=64)
    p.update(kw)
    vp = ctypes.c_void_p
    return lb.lib.lva_packed_attn(packed_bytes(p), vp(q), vp(k), vp(v), vp(o), vp(lse), vp(cu_q),
                                  vp(cu_k), vp(ws), ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=96), UNSUPPORTED), (dict(d=0), UNSUPPORTED),
    (dict(q_heads=3), INVALID), (dict(kv_heads=0), INVALID), (dict(q_heads=0), INVALID), (dict(q_heads=-4, kv_heads=2), INVALID),
    (dict(q_heads=129, kv_heads=1, q_token_stride=129 * 64, o_token_stride=129 * 64), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
    (dict(scale=3e38), INVALID),
    (dict(num_seqs=-1), INVALID), (dict(total_q=-1), INVALID), (dict(total_k=-1), INVALID),
    (dict(total_q=1 << 31), UNSUPPORTED), (dict(total_k=1 << 31), UNSUPPORTED),
    (dict(q_token_stride=252), INVALID), (dict(k_token_stride=60), INVALID), (dict(v_head_stride=8), INVALID),
    (dict(o_head_stride=68), INVALID), (dict(k_token_stride=0), INVALID), (dict(v_token_stride=-128), INVALID),
    (dict(q_token_stride=1 << 39), INVALID),
    (dict(q=24), INVALID), (dict(k=8), INVALID), (dict(v=20), INVALID), (dict(o=17), INVALID), (dict(lse=6), INVALID),
    (dict(cu_q=2), INVALID), (dict(cu_k=1), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(o=None), INVALID), (dict(lse=None), INVALID), (dict(cu_q=None), INVALID),
    (dict(cu_k=None), INVALID),
    (dict(num_seqs=0, q=None), OK), (dict(total_q=0, q=None), OK),
    (dict(ws=8), INVALID), (dict(ws=256, ws_bytes=1000, total_k=5000), CAPACITY),
])
def test_packed(kw, status):
    assert packed(**kw) == status
    assert (lb.lib.lva_last_error_message() == b"") == (status == OK)


def test_parameter_layouts():
    # the packed bytes are the C structs (include/lva.h): five ints, a float, ten 64-bit integers
    assert lb._PACKED.size == lb._PREFIX.size == 104
    assert lb._PACKED.pack(1, 2, 3, 4, 5, 1.0, *range(10))[24:32] == (0).to_bytes(8, "little")


def test_packed_null_params():
    assert lb.lib.lva_packed_attn(None, *[ctypes.c_void_p(16)] * 8, 0, None) == INVALID


def test_packed_workspace():
    size = lva.lva_packed_workspace_bytes
    assert size(2, 4, 2, 64, 100, 100) == 0                   # one key block: nothing to cut
    assert size(1, 4, 2, 128, 100000, 100000) == 0            # tiles enough
    assert size(0, 4, 2, 64, 0, 100000) == 0
    assert 0 < size(1, 4, 2, 64, 1, 8000) < size(1, 4, 2, 128, 1, 8000)
    # never past 148 parts of 128 rows
    for args in ((6, 40, 8, 128, 962, 15269), (1, 128, 1, 64, 300, 1 << 20), (500, 1, 1, 128, 500, 1 << 24), (1, 2, 2, 128, 1, 1 << 30)):
        assert 0 <= size(*args) <= 148 * 128 * (128 * 4 + 4)
    assert size(2, 3, 2, 64, 100, 100) == -1 and size(2, 4, 2, 64, -1, 100) == -1
    assert lb.lib.lva_packed_workspace_bytes(None) == -1


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_packed_host_tensors_are_refused():
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        lva.lva_packed_attn(_bf(4, 2, 64), _bf(4, 1, 64), _bf(4, 1, 64), _bf(4, 2, 64), torch.zeros(2, 4), cu, cu, 0.1)


def prefix_params(**kw):
    p = dict(B=2, steps=1, q_heads=4, kv_heads=2, d=64, scale=0.125, prefix_len=100, capacity=50, q_token_stride=256,
             q_head_stride=64, k_token_stride=128, k_head_stride=64, v_token_stride=128, v_head_stride=64,
             o_token_stride=256, o_head_stride=64)
    p.update(kw)
    return lb._PREFIX.pack(*[p[k] for k in ("B", "steps", "q_heads", "kv_heads", "d", "scale", "prefix_len", "capacity")],
                           *[p[f"{t}_{s}_stride"] for t in "qkvo" for s in ("token", "head")])


def prefix(q=16, pk=16, pv=16, kc=16, vc=16, lens=4, o=16, lse=4, weight=None, ws=256, ws_bytes=1 << 40, **kw):
    vp = ctypes.c_void_p
    return lb.lib.lva_shared_prefix_attn(prefix_params(**kw), vp(q), vp(pk), vp(pv), vp(kc), vp(vc), vp(lens),
                                         vp(o), vp(lse), vp(weight), vp(ws), ws_bytes, None)


SIZES = [
    (dict(d=96), UNSUPPORTED), (dict(q_heads=3), INVALID), (dict(kv_heads=0), INVALID), (dict(B=-1), INVALID),
    (dict(steps=0), INVALID), (dict(steps=33), UNSUPPORTED), (dict(q_heads=130), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
    (dict(prefix_len=-1), INVALID), (dict(capacity=-1), INVALID), (dict(prefix_len=1 << 31), UNSUPPORTED),
    (dict(capacity=1 << 31), UNSUPPORTED), (dict(capacity=1 << 29), UNSUPPORTED), (dict(B=1 << 30), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(q_token_stride=252), INVALID), (dict(k_token_stride=60), INVALID), (dict(v_head_stride=4), INVALID),
    (dict(o_head_stride=0), INVALID),
    (dict(q=24), INVALID), (dict(pk=8), INVALID), (dict(pv=8), INVALID), (dict(kc=8), INVALID), (dict(vc=8), INVALID),
    (dict(o=8), INVALID), (dict(ws=8), INVALID), (dict(lens=2), INVALID), (dict(lse=2), INVALID), (dict(weight=2), INVALID),
    (dict(q=None), INVALID), (dict(pk=None), INVALID), (dict(kc=None), INVALID), (dict(lens=None), INVALID),
    (dict(o=None), INVALID), (dict(lse=None), INVALID), (dict(ws=None), INVALID), (dict(ws_bytes=1000), CAPACITY),
    (dict(B=0, q=None), OK),
])
def test_shared_prefix(kw, status):
    assert prefix(**kw) == status
    assert (lb.lib.lva_last_error_message() == b"") == (status == OK)


def test_shared_prefix_workspace():
    size = lambda w=0, **kw: lb.lib.lva_shared_prefix_workspace_bytes(prefix_params(**kw), w)
    for kw, _ in SIZES:
        assert size(**kw) == -1, kw
    assert lb.lib.lva_shared_prefix_workspace_bytes(None, 0) == -1
    assert 0 < size() < size(1) and size(B=0) >= 0 and size(prefix_len=0, capacity=0) == 0
    # the scores: [B, kv_heads, rows, capacity rounded to 64] floats
    assert size(1) - size() == 2 * 2 * 2 * 64 * 4
    assert prefix(ws_bytes=size() - 1) == CAPACITY and prefix(weight=4, ws_bytes=size()) == CAPACITY
    assert lva.lva_shared_prefix_workspace_bytes(2, 1, 4, 2, 64, 100, 50) == size()


def append(kn=16, vn=16, kc=16, vc=16, weight=None, lens=4, lens_out=4, ks=128, kh=64, vs=128, vh=64, B=2, steps=1, hk=2,
           cap=50, d=64):
    vp = ctypes.c_void_p
    return lb.lib.lva_append_cache(vp(kn), vp(vn), ks, kh, vs, vh, vp(kc), vp(vc), vp(weight), vp(lens), vp(lens_out), B, steps,
                                   hk, cap, d, None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=32), UNSUPPORTED), (dict(B=-1), INVALID), (dict(steps=-1), INVALID), (dict(hk=0), INVALID), (dict(cap=-1), INVALID),
    (dict(cap=1 << 31), UNSUPPORTED), (dict(steps=1 << 30), UNSUPPORTED), (dict(B=1 << 30, steps=1 << 10), UNSUPPORTED),
    (dict(ks=60), INVALID), (dict(kh=12), INVALID), (dict(vs=132), INVALID), (dict(vh=0), INVALID),
    (dict(kn=8), INVALID), (dict(vn=4), INVALID), (dict(kc=8), INVALID), (dict(vc=24), INVALID), (dict(weight=3), INVALID),
    (dict(lens=2), INVALID), (dict(lens_out=2), INVALID), (dict(lens_out=8), INVALID), (dict(lens=8), INVALID),
    (dict(B=1 << 16, steps=1 << 20, hk=1), UNSUPPORTED),       # 2^31 CTAs
    (dict(kn=None), INVALID), (dict(vc=None), INVALID), (dict(lens=None), INVALID), (dict(lens_out=None), INVALID),
    (dict(B=0, kn=None), OK),
])
def test_append(kw, status):
    assert append(**kw) == status
    assert (lb.lib.lva_last_error_message() == b"") == (status == OK)


MB = 1 << 20


def evict(k=MB, v=2 * MB, w=3 * MB, lens=4, ko=4 * MB, vo=5 * MB, wo=6 * MB, lo=4, kept=4, B=2, hk=2, cap=50, d=64, budget=20,
          sinks=2, recent=5):
    vp = ctypes.c_void_p
    return lb.lib.lva_evict_cache(vp(k), vp(v), vp(w), vp(lens), vp(ko), vp(vo), vp(wo), vp(lo), vp(kept), B, hk, cap, d, budget,
                                  sinks, recent, None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=32), UNSUPPORTED), (dict(B=-1), INVALID), (dict(hk=0), INVALID), (dict(cap=-1), INVALID),
    (dict(budget=0), INVALID), (dict(budget=51), INVALID), (dict(sinks=-1), INVALID), (dict(recent=-1), INVALID),
    (dict(sinks=21), INVALID), (dict(sinks=10, recent=11), INVALID), (dict(recent=1 << 62), INVALID),
    (dict(B=1 << 28), UNSUPPORTED), (dict(cap=1 << 31), UNSUPPORTED),
    (dict(k=None), INVALID), (dict(w=None), INVALID), (dict(lens=None), INVALID), (dict(vo=None), INVALID), (dict(lo=None), INVALID),
    (dict(kept=None), INVALID), (dict(lo=8), INVALID),
    (dict(k=MB + 8), INVALID), (dict(vo=5 * MB + 2), INVALID), (dict(w=3 * MB + 2), INVALID), (dict(kept=2), INVALID),
    # in place: all three or none
    (dict(ko=MB), INVALID), (dict(ko=MB, vo=2 * MB), INVALID), (dict(wo=3 * MB), INVALID),
    # outputs over inputs, or over one another (a cache is 2 * 2 * 50 * 128 bytes)
    (dict(ko=MB + 16), INVALID), (dict(ko=MB - 16), INVALID), (dict(vo=MB + 25584), INVALID), (dict(ko=2 * MB + 16), INVALID),
    (dict(wo=3 * MB + 4), INVALID), (dict(vo=4 * MB + 16), INVALID), (dict(k=MB, v=MB, ko=MB, vo=MB, wo=3 * MB), INVALID),
    (dict(B=0, k=None), OK),
])
def test_evict(kw, status):
    assert evict(**kw) == status
    assert (lb.lib.lva_last_error_message() == b"") == (status == OK)


def test_cache_host_tensors_are_refused():
    i = torch.zeros(1, dtype=torch.int32)
    q, kv, c, w = _bf(1, 1, 2, 64), _bf(5, 1, 64), _bf(1, 1, 8, 64), torch.zeros(1, 1, 8)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        lva.lva_shared_prefix_attn(q, kv, kv, c, c, i, q, torch.zeros(1, 2, 1), torch.zeros(9), 0.1)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        lva.lva_append_cache(_bf(1, 1, 1, 64), _bf(1, 1, 1, 64), c, c, w, i, i)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        lva.lva_evict_cache(c, c, w, i, c, c, w, i, torch.zeros((1, 1, 4), dtype=torch.int32), 4)


class _Cuda:
    """A host tensor that says it is on cuda:0 (for checks that read no data)."""
    is_cuda = True

    def __init__(self, t):
        self.dtype, self.shape, self.stride = t.dtype, t.shape, t.stride

    def get_device(self):
        return 0


def test_steps_view_wants_one_token_stride():
    from block_sparse_attention_lva_b200._binding import _steps_view
    t = _bf(2, 6, 2, 64)[:, :3]
    with pytest.raises(ValueError, match="one stride"):
        _steps_view(_Cuda(t), "q", (2, 3, 2, 64), 0)
