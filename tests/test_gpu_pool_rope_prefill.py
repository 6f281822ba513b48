"""DecodePool.rope_prefill writes what the library's calls write, for each kind of pool, prompts and later chunks."""
import numpy as np
import pytest
import torch

from fp8_paged_kv_gb300 import fpk_rope_prefill_bf16, fpk_rope_prefill_fp8, fpk_rope_prefill_fp8_block
from fp8_paged_kv_gb300.pool import DecodePool
from fp8_paged_kv_gb300.rope import rope_inv_freq
from workloads import custom

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("kind", ["fp8", "bf16", "block"])
@pytest.mark.parametrize("guard", [True, False])
@pytest.mark.parametrize("interleaved", [True, False])
def test_prompts_and_chunks(kind, guard, interleaved):
    lens, B = [100, 0, 33], 3
    wl = custom(5, B=B, Hq=8, Hkv=2, ps=32, prompt_lens=lens, steps=1)
    wl.expected_tags[2, 1] ^= np.uint32(1)                        # a stale mapping: guarded writes leave that page alone
    a, b = (DecodePool(wl, fp8=kind != "bf16", device=DEV, block_scales=kind == "block") for _ in range(2))
    freqs, scale = rope_inv_freq(96, 10000.0, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    for counts, first in (([60, 0, 30], None), ([40, 0, 3], [60, 0, 30])):
        T = sum(counts)
        q, k, v = (torch.randn(T, h, 128, device=DEV, generator=g).to(torch.bfloat16) for h in (8, 2, 2))
        cu, start, q_out = i32([0, *np.cumsum(counts)]), None if first is None else i32(first), torch.empty_like(q)
        tags = (b.live_tags, b.expected_tags, None) if guard else (None, None, None)
        kw = dict(Hkv=2, page_size=32, num_pages=wl.num_pages, rot_dim=96, interleaved=interleaved, rot_scale=scale)
        rows = (q, k, v, cu, start, freqs, q_out, b.kv_pool)
        if kind == "fp8":
            fpk_rope_prefill_fp8(*rows, b.k_scale, b.v_scale, b.page_table, *tags, **kw)
        elif kind == "bf16":
            fpk_rope_prefill_bf16(*rows, b.page_table, *tags, **kw)
        else:
            fpk_rope_prefill_fp8_block(*rows, b.kv_scales, b.page_table, *tags, **kw)
        before = a.kv_pool.clone()
        mine = q.clone()
        a.rope_prefill(mine, k, v, cu, start, freqs, rot_dim=96, interleaved=interleaved, rot_scale=scale, guard=guard)
        torch.cuda.synchronize()
        assert torch.equal(mine.view(torch.int16), q_out.view(torch.int16))
        assert torch.equal(a.kv_pool.view(torch.uint8), b.kv_pool.view(torch.uint8))
        assert not torch.equal(a.kv_pool.view(torch.uint8), before.view(torch.uint8))
        if kind == "block":
            assert torch.equal(a.kv_scales, b.kv_scales)
    stale = int(wl.page_table[2, 1])
    page = a.kv_pool.view(torch.uint8).view(wl.num_pages, -1)[stale]
    untouched = DecodePool(wl, fp8=kind != "bf16", device=DEV).kv_pool.view(torch.uint8).view(wl.num_pages, -1)[stale]
    assert torch.equal(page, untouched) == guard
