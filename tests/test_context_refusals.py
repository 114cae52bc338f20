"""Argument checks of the packed, shared-prefix, append and evict calls: every bad call is
refused on the host, before anything reaches a GPU (no GPU needed)."""
import ctypes
import math

import pytest
import torch

import block_sparse_attention_lva_b200 as lva
from block_sparse_attention_lva_b200 import _binding as lb

OK, INVALID, UNSUPPORTED, CAPACITY = 0, 1, 2, 3


def packed(q=16, k=16, v=16, o=16, lse=4, cu_q=4, cu_k=4, **kw):
    p = dict(num_seqs=2, q_heads=4, kv_heads=2, d=64, causal=1, scale=0.125, total_q=100, total_k=100,
             q_token_stride=256, q_head_stride=64, k_token_stride=128, k_head_stride=64, v_token_stride=128,
             v_head_stride=64, o_token_stride=256, o_head_stride=64)
    p.update(kw)
    vp = ctypes.c_void_p
    return lb.lib.lva_packed_attn(ctypes.byref(lb.LvaPackedParams(**p)), vp(q), vp(k), vp(v), vp(o), vp(lse), vp(cu_q),
                                  vp(cu_k), None)


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
])
def test_packed(kw, status):
    assert packed(**kw) == status
    assert (lb.lib.lva_last_error_message() == b"") == (status == OK)


def test_packed_null_params():
    assert lb.lib.lva_packed_attn(None, *[ctypes.c_void_p(16)] * 7, None) == INVALID


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_packed_host_tensors_are_refused():
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        lva.lva_packed_attn(_bf(4, 2, 64), _bf(4, 1, 64), _bf(4, 1, 64), _bf(4, 2, 64), torch.zeros(2, 4), cu, cu, 0.1)
