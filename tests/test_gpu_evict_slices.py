"""In-place eviction at every width of a column slice (csrc/cache_ops.cu, move_in_place_kernel)."""
import numpy as np
import pytest
import torch

from oracle.packed import evict_kept
from tests.gpu_helpers import require_gpu
from tests.test_gpu_context_cache import i32

pytestmark = pytest.mark.gpu


# A column slice of the in-place move is 2 (32 bytes) to 16 units wide, by the number of planes:
# slices double up to units / 2 until planes x 2 x slices reaches three thread blocks a multiprocessor
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,hk", [(10, 3), (30, 2), (40, 3), (77, 3)])
def test_evict_in_place_at_every_slice_width(B, hk, d):
    import block_sparse_attention_lva_b200 as lva
    dev = require_gpu()
    assert torch.cuda.get_device_properties(dev).multi_processor_count == 148       # what the plane counts stand for
    cap, budget, sinks, recent = 2100, 1801, 3, 200
    g = torch.Generator().manual_seed(B + d)
    gd = torch.Generator(device=dev).manual_seed(B + d)
    kc, vc = (torch.randn((B, hk, cap, d), generator=gd, device=dev).to(torch.bfloat16) for _ in range(2))
    w = torch.exp(2 * torch.randn((B, hk, cap), generator=g)).to(dev)
    lens = [[cap, 2050, 1801, 700, 0, 1802][b % 6] for b in range(B)]
    k0, v0, w0, wh = kc.clone(), vc.clone(), w.clone(), w.cpu().numpy()
    want, want_kept = [kc.clone(), vc.clone(), w.clone()], np.full((B, hk, budget), -1)
    for b, n in enumerate(lens):
        for h in range(hk):
            idx = evict_kept(wh[b, h], n, budget, sinks, recent)
            want_kept[b, h, :len(idx)] = idx
            for dst, src in zip(want, (k0, v0, w0)):
                dst[b, h, :len(idx)] = src[b, h, torch.from_numpy(idx).to(dev)]
    lt = i32(lens, dev)
    kept = torch.full((B, hk, budget), -5, dtype=torch.int32, device=dev)
    lva.lva_evict_cache(kc, vc, w, lt, kc, vc, w, lt, kept, budget, sinks, recent)
    torch.cuda.synchronize()
    assert lva.lva_device_error() == (0, 0)
    assert np.array_equal(kept.cpu().numpy(), want_kept) and lt.tolist() == [min(n, budget) for n in lens]
    for got, ref in zip((kc, vc, w), want):
        assert torch.equal(got.view(torch.int32), ref.view(torch.int32))
