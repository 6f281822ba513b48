"""Shared-prefix attention of a DecodePool first called while a graph is captured: what it
writes to belongs to the pool, not to the graph."""
import numpy as np
import pytest
import torch

from fp8_paged_kv_gb300 import fpk_decode_status
from fp8_paged_kv_gb300.pool import DecodePool
from workloads import custom

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("fp8", [True, False])
def test_first_call_in_a_capture(fp8):
    wl = custom(3, B=4, Hq=16, Hkv=2, ps=16, prompt_lens=[300, 310, 40, 7], steps=0)
    pool = DecodePool(wl, fp8=fp8, device=DEV)
    pool.prefill()
    pool.page_table[1, :10] = pool.page_table[0, :10]
    pool.q.copy_(torch.from_numpy(np.random.default_rng(2).standard_normal((4, 16, 128)).astype(np.float32)))
    starts, pre = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 2], [160]))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        before = torch.cuda.memory_allocated()      # (the capture's own generator state among it)
        pool.attend_shared(starts, pre, use_mask=False)
        after = torch.cuda.memory_allocated()
    assert after == before
    # a call of its own before the graph has ever run, the graph, and a call after it is gone
    got = []
    for call in (lambda: pool.attend_shared(starts, pre, use_mask=False), graph.replay, graph.replay,
                 lambda: (graph.reset(), pool.attend_shared(starts, pre, use_mask=False))):
        pool.out16.fill_(float("nan"))
        call()
        torch.cuda.synchronize()
        assert fpk_decode_status(pool.prefix_workspace) == 0
        got.append((pool.out16.clone(), pool.lse.clone()))
    assert got[0][0].any() and torch.isfinite(got[0][0]).all()
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
