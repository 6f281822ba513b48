"""Angles at positions up to the largest: the query of a token is rotated whatever its
position, so contexts of 2^31 - 1 tokens need no pages.  Where a pair's two products
nearly cancel, a bf16 result is small and shows the angle's error.  The reference
turns by the product of two unit vectors whose angles are exact in 64 bits."""
import numpy as np
import pytest
import torch

from fp8_paged_kv_gb300 import fpk_rope_append_bf16, fpk_rope_prefill_bf16

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D, HQ, N = 128, 64, 48


def turned(q, pos, f):
    """q float64 [N][HQ][D] by halves, and each pair's magnitude."""
    lo, hi = (pos & 0xFFFF).astype(np.float64), (pos - (pos & 0xFFFF)).astype(np.float64)
    u = np.exp(1j * lo[:, None] * f) * np.exp(1j * hi[:, None] * f)   # 15 + 24 and 16 + 24 bits: exact angles
    z = (q[..., :D // 2] + 1j * q[..., D // 2:]) * u[:, None]
    mag = np.abs(q[..., :D // 2]) + np.abs(q[..., D // 2:])
    return np.concatenate([z.real, z.imag], -1), np.concatenate([mag, mag], -1)


@pytest.mark.parametrize("append", [True, False])
@pytest.mark.parametrize("top", [20, 24, 26, 27, 28, 29, 30, 31])
def test_far_angles(append, top):
    rng = np.random.default_rng(top)
    pos = np.sort(rng.integers(1 << (top - 1), (1 << top) - 2, N))
    pos[-1] = (1 << top) - 2
    f = np.concatenate([[1.0], rng.uniform(0.25, 1.0, D // 2 - 1)]).astype(np.float32)
    g = torch.Generator().manual_seed(top)
    q = torch.randn(N, HQ, D, generator=g).to(torch.bfloat16)
    k = torch.zeros(N, 1, D, dtype=torch.bfloat16, device=DEV)
    out = torch.zeros(N, HQ, D, dtype=torch.bfloat16, device=DEV)
    pool = torch.zeros(2 * 16 * D, dtype=torch.bfloat16, device=DEV)
    table, abort = torch.zeros(N, 1, dtype=torch.int32, device=DEV), torch.zeros(N, dtype=torch.uint8, device=DEV)
    i32 = lambda x: torch.from_numpy(np.asarray(x, np.int32)).to(DEV)  # noqa: E731
    kw = dict(abort_mask=abort, Hkv=1, page_size=16, num_pages=1, rot_dim=D)
    ft = torch.from_numpy(f).to(DEV)
    if append:
        fpk_rope_append_bf16(q.to(DEV), k, k, ft, out, pool, table, i32(pos + 1), **kw)
    else:
        fpk_rope_prefill_bf16(q.to(DEV), k, k, i32(np.arange(N + 1)), i32(pos), ft, out, pool, table, **kw)
    torch.cuda.synchronize()
    assert abort.all() and not pool.any()
    y, mag = turned(q.double().numpy(), pos, f.astype(np.float64))
    err = np.abs(out.double().cpu().numpy() - y)
    tol = 2.0 ** -8 * np.abs(y) + (2.0 ** -20 + 3 * 2.0 ** -24) * mag
    assert (err <= tol).all(), f"{(err / tol).max():.1f} of the tolerance"
    assert (2.0 ** -8 * np.abs(y) < 2.0 ** -21 * mag).sum() > 20   # results that show it
