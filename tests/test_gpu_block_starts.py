"""cu_seqlens that decrease set the status word and leave every row alone, however few rows they come to."""
import numpy as np
import pytest
import torch

from fp8_paged_kv_gb300 import fpk_decode_status, fpk_paged_prefill_attn_fp8_block, fpk_prefill_workspace_bytes
from test_gpu_block_attention import DEV, SM, dev, scene

pytestmark = pytest.mark.gpu
N = 256


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("empty", [0, 40, 1100])
@pytest.mark.parametrize("cu", [[0, 5, 0, 5], [0, 3, 1, 2], [0, N, N - 1, N], [0, 200, 100, 150], [0, 1 << 30, -5, 7]])
def test_starts(cu, empty, causal):
    """empty: requests without rows behind them, so that a plan makes the list, near or far."""
    cu = np.array(cu + cu[-1:] * empty, np.int32)
    B = len(cu) - 1
    s = scene([40], [1], Hq=16, Hkv=2, ps=16, seed=3)
    g = torch.Generator(device=DEV).manual_seed(1)
    q = torch.randn(N, 16, 128, device=DEV, generator=g).to(torch.bfloat16)
    out, lse = torch.full_like(q, 7.0), torch.full((N, 16), 7.0, device=DEV)
    ws = torch.zeros(fpk_prefill_workspace_bytes(B, N, 16, 2), dtype=torch.uint8, device=DEV)
    table, lens = dev(s["table"]).expand(B, -1).contiguous(), dev(s["lens"]).expand(B).contiguous()

    def call(starts):
        fpk_paged_prefill_attn_fp8_block(q, dev(starts), dev(s["pool"]).reshape(-1), dev(s["scales"]), table, lens, None, out, lse,
                                         ws, causal=causal, Hkv=2, page_size=16, num_pages=s["P"], sm_scale=SM)
        torch.cuda.synchronize()

    call(cu)
    assert fpk_decode_status(ws) != 0 and torch.all(out == 7) and torch.all(lse == 7)
    ws[:4] = 0
    good = np.minimum(np.maximum.accumulate(cu.clip(0)), N).astype(np.int32)
    call(good)              # the same workspace answers the next call
    assert fpk_decode_status(ws) == 0
    last = int(good[-1])
    assert torch.all(out[last:] == 7) and not torch.any(lse[:last] == 7)
