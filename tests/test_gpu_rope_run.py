"""A prompt and its answer under one rotation: a prompt written by the prefill, in one call or in
chunks, and the tokens behind it by appends leave the pool that one prefill of
all of them leaves, bit for bit, and the same rotated queries."""
import numpy as np
import pytest
import torch

from fp8_paged_kv_gb300 import (fpk_rope_append_bf16, fpk_rope_append_fp8, fpk_rope_prefill_bf16,
                                fpk_rope_prefill_fp8)
from fp8_paged_kv_gb300.rope import rope_inv_freq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D, HQ, HKV, B = 128, 12, 3, 3


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("ps", [16, 64])
def test_prompt_and_answer(fp8, inter, ps):
    prompts, more = [70, 1, 200], 37
    total = [n + more for n in prompts]
    maxp = -(-max(total) // ps)
    g = torch.Generator(device=DEV).manual_seed(ps)
    q, k, v = ([torch.randn(n, h, D, device=DEV, generator=g).to(torch.bfloat16) for n in total] for h in (HQ, HKV, HKV))
    P = B * maxp + 2
    table = torch.randperm(P, generator=g, device=DEV)[:B * maxp].view(B, maxp).to(torch.int32)
    f, scale = rope_inv_freq(96, 10000.0, scaling="yarn", factor=4.0, original_len=512, device=DEV)
    sc = tuple(torch.tensor([x], device=DEV) for x in (0.013, 0.021)) if fp8 else ()
    kw = dict(Hkv=HKV, page_size=ps, num_pages=P, rot_dim=96, interleaved=inter, rot_scale=scale)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)  # noqa: E731

    def empty():
        x = torch.full((2 * P * HKV * ps * D,), 0x25, dtype=torch.uint8 if fp8 else torch.int16, device=DEV)
        return x if fp8 else x.view(torch.bfloat16)

    def prefill(pool, spans):
        """Tokens [a, b) of each request; their rotated queries."""
        rows = [torch.cat([x[r][a:b] for r, (a, b) in enumerate(spans)]) for x in (q, k, v)]
        out = torch.empty_like(rows[0])
        cu = i32(np.concatenate([[0], np.cumsum([b - a for a, b in spans])]))
        (fpk_rope_prefill_fp8 if fp8 else fpk_rope_prefill_bf16)(*rows, cu, i32([a for a, _ in spans]), f, out, pool, *sc,
                                                                 table, **kw)
        return list(out.split([b - a for a, b in spans]))

    def append(pool, t):
        rows = [torch.stack([x[r][n + t] for r, n in enumerate(prompts)]) for x in (q, k, v)]
        out = torch.empty_like(rows[0])
        (fpk_rope_append_fp8 if fp8 else fpk_rope_append_bf16)(*rows, f, out, pool, *sc, table,
                                                               i32([n + t + 1 for n in prompts]), **kw)
        return out

    whole = empty()
    want = prefill(whole, [(0, n) for n in total])
    for cuts in ([1.0], [0.3, 0.77, 1.0]):
        pool, got, at = empty(), [[] for _ in range(B)], [0] * B
        for c in cuts:
            to = [int(n * c) for n in prompts]
            for r, x in enumerate(prefill(pool, list(zip(at, to)))):
                got[r].append(x)
            at = to
        for t in range(more):
            for r, x in enumerate(append(pool, t)):
                got[r].append(x[None])
        torch.cuda.synchronize()
        assert torch.equal(pool.view(torch.uint8), whole.view(torch.uint8))
        for r in range(B):
            assert torch.equal(torch.cat(got[r]), want[r])
