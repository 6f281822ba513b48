"""Values that are no numbers in shared-prefix attention: a NaN scale, query, key or
value makes the rows that meet it NaN, as the formula does, and no others, and scores
of -inf have no weight.  Tolerances are those of test_gpu_prefix.py."""
import numpy as np
import pytest
import torch

from fp8_paged_kv_gb300 import fpk_decode_status
from test_gpu_prefix import BOTH, D, TILE, call, make, reference

pytestmark = pytest.mark.gpu
# what a request has: the shared pages alone, own tokens behind them, one own token, no shared page, no group
GROUPS = [(256, [256, 300, 256, 257]), (0, [40, 256])]


def run(c, nan, what=""):
    """nan: bool [B][Hq] (or with D), the outputs that are NaN; the others are right."""
    s = call(c)
    torch.cuda.synchronize()
    assert fpk_decode_status(s["ws"]) == 0
    out, lse = s["out"].double().cpu().numpy(), s["lse"].double().cpu().numpy()
    full = np.broadcast_to(nan[..., None] if nan.ndim == 2 else nan, out.shape)
    assert np.array_equal(np.isnan(out), full), f"{what}: {np.argwhere(np.isnan(out) != full)[:4]}"
    if nan.ndim == 2:
        assert np.array_equal(np.isnan(lse), nan), what
    return out, lse


def close(c, out, lse, ref):
    ro, rl, A, ds = ref
    n, w = int(c["lens"].max()), 2.0 ** -11 if c["fp8"] else 2.0 ** -8
    tol = 2.0 ** -8 * np.abs(ro) + (w + 2 * ds[..., None] + n * 2.0 ** -24) * A + 1e-12
    live = ~np.isnan(out)
    assert (np.abs(out - ro)[live] <= tol[live]).all()
    live = ~np.isnan(lse) & np.isfinite(rl)
    assert np.array_equal(np.isneginf(lse), np.isneginf(rl) & ~np.isnan(lse))
    assert (np.abs(lse - rl)[live] <= (ds + n * 2.0 ** -24 + 2.0 ** -20 * np.abs(rl))[live]).all()


@BOTH
def test_nan_scales(fp8):
    c = make(GROUPS, fp8=fp8, lead=1, G=4)
    nan = np.ones((c["B"], 8), bool)
    for name in ("sm", "ks") if fp8 else ("sm",):
        run({**c, name: float("nan")}, nan, name)


@BOTH
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nan_queries(fp8, bad):
    # (an infinite query has scores of both signs of infinity, and NaN)
    c = make(GROUPS, fp8=fp8, lead=1, G=4, seed=1)
    ref = reference(c)
    nan = np.zeros((c["B"], 8), bool)
    for r in range(c["B"]):
        c["q"][r, (3 * r) % 8, (11 * r) % D] = bad
        nan[r, (3 * r) % 8] = True
    close(c, *run(c, nan), ref)


@BOTH
@pytest.mark.parametrize("r,t", [(1, 100), (2, 299), (4, 256), (6, 255), (0, 3)])
def test_nan_keys(fp8, r, t):
    # one token's key of kv head 1: in the shared pages, behind them, the only own one, in no shared page
    c = make(GROUPS, fp8=fp8, lead=1, G=4, seed=2)
    ref = reference(c)
    pool = c["pool"].view(c["P"], 2, 1, 2, TILE * D)
    pool[c["table"][r, t // 16], 1, 0, 0, t % 16 * D + 5] = 0x7F if fp8 else float("nan")
    nan = np.zeros((c["B"], 8), bool)
    nan[[1, 2, 3, 4] if r == 1 else [r], 4:] = True
    close(c, *run(c, nan), ref)


@BOTH
@pytest.mark.parametrize("r,t", [(1, 100), (4, 256), (6, 255)])
def test_nan_values(fp8, r, t):
    c = make(GROUPS, fp8=fp8, lead=1, G=4, seed=3)
    ref = reference(c)
    pool = c["pool"].view(c["P"], 2, 1, 2, TILE * D)
    pool[c["table"][r, t // 16], 0, 0, 1, 9 * TILE + t % 16] = 0x7F if fp8 else float("nan")
    nan = np.zeros((c["B"], 8, D), bool)
    nan[[1, 2, 3, 4] if r == 1 else [r], :4, 9] = True
    out, lse = run(c, nan)
    close(c, out, lse, ref)
