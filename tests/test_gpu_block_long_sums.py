"""Prompt attention over long contexts: O's sums keep what fp32 holds.

Positive values, so that nothing cancels and what the tensor cores cut off shows, and queries that are all but 0.  A
tile's products are added up there over 64 blocks at most, 16 additions a block, each of which may cut a step off:
64 * 16 * 2^-23 = 2^-13 of O.  Adding those up takes half a step 2 * 16 times, weights 2^-22 and scores 2^-19 at most:
2^-18.  The sum of weights is off by what lse is.  bf16 results: half a step of theirs."""
import numpy as np
import pytest
import torch

from block_helpers import bf16, context
from block_torch import blocks, check_rows, codes
from fp8_paged_kv_gb300 import fpk_decode_status, fpk_paged_prefill_attn_fp8_block, fpk_prefill_workspace_bytes
from test_gpu_block_attention import DEV, SM, dev, run, scene

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("n", [4, 32])  # units of one row tile, and of both
@pytest.mark.parametrize("B", [1, 152])  # cut between CTAs, or whole
@pytest.mark.parametrize("L", [131072, 20000, 8192])
def test_sums(L, B, n, causal):
    Hq, Hkv, ps = 8, 1, 256
    s = scene([L], [n], Hq=Hq, Hkv=Hkv, ps=ps, seed=L, spread=0)
    v = blocks(s, s["pool"], 1)
    v &= 0x7F
    s["q"] *= 2.0 ** -8
    pool, scales = dev(s["pool"]).reshape(-1), dev(s["scales"])
    q = dev(s["q"]).repeat(B, 1, 1)
    table, lens = dev(s["table"]).repeat(B, 1), dev(s["lens"]).repeat(B)
    cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device=DEV)
    out, lse = torch.full_like(q, 7.0), torch.full((B * n, Hq), 7.0, device=DEV)
    ws = torch.zeros(fpk_prefill_workspace_bytes(B, B * n, Hq, Hkv), dtype=torch.uint8, device=DEV)
    fpk_paged_prefill_attn_fp8_block(q, cu, pool, scales, table, lens, None, out, lse, ws, causal=causal, Hkv=Hkv, page_size=ps,
                                     num_pages=s["P"], sm_scale=SM)
    torch.cuda.synchronize()
    assert fpk_decode_status(ws) == 0
    k, v, _ = (torch.from_numpy(np.ascontiguousarray(x)).to(DEV) for x in context(s["pool"], s["scales"], s["table"][0], L, 0, ps))
    e = q[:n].double().reshape(-1, 128) @ k.T * SM
    assert (q[:n].double().abs().reshape(-1, 128) @ k.abs().T * SM).max() < 0.125   # scores off by 2^-20 at most
    hidden = torch.arange(L, device=DEV) >= (torch.arange(n, device=DEV) + (L - n + 1 if causal else L)).clamp(max=L).repeat_interleave(Hq).unsqueeze(1)
    e.masked_fill_(hidden, -torch.inf)
    z = torch.logsumexp(e, 1)
    ref = (torch.exp(e - z.unsqueeze(1)) @ v).view(1, n, Hq, 128)
    le = (lse.double().view(B, n, Hq) - z.view(1, n, Hq)).abs()
    assert torch.all(le <= L / 16 * 2.0 ** -24 + 2.0 ** -19), float(le.max())  # an addition per 16 tokens
    half = torch.exp2(torch.floor(torch.log2(ref)) - 8)
    err = (out.double().view(B, n, Hq, 128) - ref).abs()
    bound = half + (2.0 ** -13 + 2.0 ** -18 + le.unsqueeze(-1)) * ref
    assert torch.all(err <= bound), f"{int((err > bound).sum())} of {err.numel()}, by {float(((err - half) / ref).max()):.1e} behind rounding"


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("counts", [[40, 5], [3, 300]])
@pytest.mark.parametrize("up", [True, False])
def test_maxima_that_grow(counts, causal, up):
    """Scores that rise by 80 over the context, or fall: what was kept meets another maximum, or keeps its own."""
    s = scene([30000, 17003], counts, Hq=16, Hkv=2, ps=256, seed=sum(counts), spread=0)
    k = blocks(s, s["pool"], 0)
    k[...] = 0
    for r, L in enumerate(s["lens"]):
        for j in range(-(-int(L) // 256)):
            x = j * 256 / 30000 if up else 1 - j * 256 / 30000
            k[s["table"][r, j], :, :, :, 0] = codes(10.0 * x)
    s["scales"][..., 0] = 127
    s["q"] *= 0.125
    s["q"][..., 0] = 1.0
    check_rows(s, run(s, causal=causal, sm=8.0), causal=causal, sm=8.0, weight=2.0 ** -22, floor=2.0 ** -32)
