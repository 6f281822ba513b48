"""A compaction between decode steps whose tables map every growth page ahead of the
context: requests go on into those pages, the pages freed are given to another
request, and each step's attention is the oracle's over what the ledger says."""
import numpy as np
import pytest
import torch

import oracle
from fp8_paged_kv_gb300.ledger import PageLedger
from fp8_paged_kv_gb300.pool import DecodePool, to_device
from workloads import custom

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("fp8", [True, False])
def test_compaction_with_pages_mapped_ahead(fp8):
    lens, steps = [300, 47, 160, 15, 96], 40
    wl = custom(9, B=5, Hq=8, Hkv=2, ps=16, prompt_lens=lens, steps=steps, pool_factor=1.6, extra_pages=9)
    pool = DecodePool(wl, fp8=fp8, device=DEV)
    led = PageLedger(wl.num_pages, wl.page_table.shape[1], wl.B, 16, wl.live_tags, wl.page_table, wl.prompt_lens)
    pool.prefill()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    rng = np.random.default_rng(1)

    def tables():
        pool.page_table.copy_(to_device(led.page_table, DEV))
        pool.expected_tags.copy_(to_device(led.expected, DEV))
        pool.seq_lens.copy_(i32(led.lens))

    for step in range(steps):
        if step == 3:
            led.release(0)                        # a long request leaves
            tables()
            src, dst = led.compact()
            assert len(src)
            pool.compact(i32(src), i32(dst))
            torch.cuda.synchronize()
            assert np.array_equal(pool.page_table.cpu().numpy(), led.page_table)
            assert np.array_equal(pool.expected_tags.cpu().numpy().view(np.uint32), led.expected)
            assert np.array_equal(pool.live_tags.cpu().numpy().view(np.uint32), led.tags)
        if step == 5:
            pool.bump(i32(led.admit(0, 260)))     # another one takes pages that were freed
            tables()
        got = [p for r in range(wl.B) if led.lens[r] for p in led.grow(r)]
        assert not [p for r in range(1, wl.B) for p in got if p in led.held[r]]   # theirs were mapped already
        if got:
            pool.bump(i32(got))
        tables()
        for name, H in (("q", wl.Hq), ("k_new", wl.Hkv), ("v_new", wl.Hkv)):
            getattr(pool, name).copy_(torch.from_numpy(rng.standard_normal((wl.B, H, 128)).astype(np.float32)))
        pool.append()
        pool.validate()
        pool.attend()
        torch.cuda.synchronize()
        assert not pool.abort_mask.any()
        if step < 3 or step % 6 == 5:
            rows = slice(1, None)                 # (request 0's new prompt is never written)
            o, l_ = oracle.paged_attention(pool.q.view(torch.int16).cpu().numpy().view(np.uint16), pool.pool_bytes(),
                                           led.page_table, np.where(np.arange(wl.B) > 0, led.lens, 0), fp8=fp8,
                                           k_scale=wl.k_scale, v_scale=wl.v_scale, sm_scale=wl.sm_scale, Hkv=wl.Hkv,
                                           page_size=16, num_pages=wl.num_pages)
            out, lse = pool.out.cpu().numpy(), pool.lse.cpu().numpy()
            assert (np.abs(out - o) <= 2e-3 + 1e-2 * np.abs(o))[rows].all()
            assert (np.abs(lse - l_) <= 1e-3 + 2.0 ** -16 * np.abs(l_))[rows].all()
    for r in range(wl.B):
        led.release(r)
    assert len(led.free) == wl.num_pages
