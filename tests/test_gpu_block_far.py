"""Prompt attention over the longest context that it takes, 2^31 - 256 tokens: a page of 256 tokens mapped 2^23 - 1 times,
so that a row is the attention over one page, and its lse ln(2^23 - 1) more.

Bounds, from the arithmetic.  A CTA adds 2^24 blocks / 152 CTAs (110377) of a unit; a row's sum grows eight times a
block by fp32 additions of half a step each: off by 8 * 110377 * 2^-24 = 0.053 of itself at most.  O is added up by the
tensor cores, at most 16 times a block, each of which may cut a whole step off: 16 * 110377 * 2^-23 = 0.211 of it.  All
values are positive, so that these are relative to the result.  Merging 152 partials, weights (2^-11) and scores (2^-15,
of sums below 8) come to less than 2^-9, and bf16 to 2^-8: 0.28 for results, 0.06 for lse.  Causal rows see up to 299
tokens of 2^31 fewer, which is nothing here."""
import math

import numpy as np
import pytest
import torch

from block_helpers import attend, bf16, context
from fp8_paged_kv_gb300 import fpk_decode_status, fpk_paged_prefill_attn_fp8_block, fpk_prefill_workspace_bytes
from test_gpu_block_attention import DEV, SM, dev, scene

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [False, True])
def test_the_longest_context(causal):
    n, pages = 300, (1 << 23) - 1
    s = scene([256], [n], Hq=1, Hkv=1, ps=256, seed=1)
    page = int(s["table"][0, 0])
    s["pool"][page, :, :, 1] &= 0x7F
    table = torch.full((1, pages), page, dtype=torch.int32, device=DEV)
    lens = torch.tensor([pages * 256], dtype=torch.int32, device=DEV)
    q = dev(s["q"])
    out, lse = torch.full_like(q, 7.0), torch.full((n, 1), 7.0, device=DEV)
    ws = torch.zeros(fpk_prefill_workspace_bytes(1, n, 1, 1), dtype=torch.uint8, device=DEV)
    fpk_paged_prefill_attn_fp8_block(q, dev(s["cu"]), dev(s["pool"]).reshape(-1), dev(s["scales"]), table, lens, None, out, lse, ws,
                                     causal=causal, Hkv=1, page_size=256, num_pages=s["P"], sm_scale=SM)
    torch.cuda.synchronize()
    assert fpk_decode_status(ws) == 0
    k, v, ev = context(s["pool"], s["scales"], s["table"][0], 256, 0, 256)
    ref, ref_lse, size, sb, _ = attend(bf16(s["q"])[:, 0], k, v, ev, np.full(n, 256), SM)
    assert np.all(v >= 0) and sb.max() < 64
    assert np.all(np.abs(bf16(out)[:, 0] - ref) <= 0.28 * size)
    assert np.all(np.abs(bf16(lse)[:, 0] - ref_lse - math.log(pages)) <= 0.06)
