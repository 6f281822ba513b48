"""Causal rows that see nothing are 0 and -inf whatever their query holds, beside rows that see something."""
import numpy as np
import pytest
import torch

from block_torch import check_rows
from test_gpu_block_attention import SM, run, scene

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("what", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("Hq,Hkv", [(16, 2), (10, 2), (4, 4)])
def test_queries_that_are_not_finite(Hq, Hkv, what):
    lens, counts = [10, 1, 140, 300], [37, 300, 150, 420]
    s = scene(lens, counts, Hq=Hq, Hkv=Hkv, ps=16, seed=Hq)
    clean = run(s, causal=True)
    check_rows(s, clean, causal=True, sm=SM)
    blind = np.zeros(s["T"], bool)
    for a, n, L in zip(s["cu"], counts, lens):
        blind[a:a + n - L] = True
    s["q"][torch.from_numpy(blind)] = what
    s["q"][26] = what                      # the last row of the first request that sees nothing; 27 sees a token
    s["q"][30, Hq - 1, 77] = what
    out, lse = run(s, causal=True)
    hit = np.zeros(lse.shape, bool)
    hit[30, Hq - 1] = True
    assert blind[26] and not blind[27]
    assert np.all(out[blind] == 0) and np.all(np.isneginf(lse[blind]))
    assert np.isnan(out[hit]).all() and np.isnan(lse[hit]).all()
    assert np.array_equal(out[~hit], clean[0][~hit]) and np.array_equal(lse[~hit], clean[1][~hit])


@pytest.mark.parametrize("sm", [float("nan"), float("inf"), 0.0])
def test_scales_that_are_not_finite(sm):
    """A scale that makes NaN of every score leaves these rows alone too."""
    s = scene([10, 140], [37, 150], Hq=16, Hkv=2, ps=16, seed=1)
    out, lse = run(s, causal=True, sm=sm)
    blind = np.r_[:27, 37:47]
    assert np.all(out[blind] == 0) and np.all(np.isneginf(lse[blind]))
    if sm != sm:
        seen = np.setdiff1d(np.arange(s["T"]), blind)
        assert np.isnan(out[seen]).all() and np.isnan(lse[seen]).all()
