"""Keys whose scores are -inf (bf16 cache): such tokens have no weight, and where a row has
no other token its result is empty, 0 and -inf.  The reference is in 64 bits, over the
other tokens alone; tolerances are those of test_gpu_prefix.py."""
import numpy as np
import pytest
import torch

from fp8_paged_kv_gb300 import fpk_decode_status
from test_gpu_prefix import D, TILE, call, make

pytestmark = pytest.mark.gpu
PS = 16


def without(c, gone):
    """Attention over the tokens that gone[r] (bool [L]) leaves, and the magnitudes that the tolerances take."""
    pool = c["pool"].view(c["P"], c["Hkv"], 1, 2, TILE * D).double().numpy()
    B, Hkv, G = c["B"], c["Hkv"], c["G"]
    out, lse = np.zeros((B, Hkv, G, D)), np.full((B, Hkv, G), -np.inf)
    A, ds = np.zeros((B, Hkv, G, D)), np.zeros((B, Hkv, G))
    for r in range(B):
        L = int(c["lens"][r])
        x = pool[c["table"][r, :-(-L // PS)]]
        keep = np.flatnonzero(~gone[r])
        if not keep.size:
            continue
        k = x[:, :, 0, 0].reshape(-1, Hkv, TILE, D).transpose(1, 0, 2, 3).reshape(Hkv, -1, D)[:, keep]
        v = x[:, :, 0, 1].reshape(-1, Hkv, D, TILE).transpose(1, 0, 3, 2).reshape(Hkv, -1, D)[:, keep]
        q = c["q"][r].double().numpy().reshape(Hkv, G, D)
        s = np.einsum("hgd,hld->hgl", q, k) * c["sm"]
        m = s.max(-1, keepdims=True)
        p = np.exp(s - m)
        z = p.sum(-1, keepdims=True)
        out[r] = np.einsum("hgl,hld->hgd", p, v) / z
        A[r] = np.einsum("hgl,hld->hgd", p, np.abs(v)) / z
        lse[r] = (m + np.log(z))[..., 0]
        ds[r] = 2 * 2.0 ** -17 * np.abs(q).max(-1) * np.abs(k).sum(-1).max(-1)[:, None] * c["sm"]
    return [x.reshape(B, Hkv * G, *x.shape[3:]) for x in (out, lse, A, ds)]


def run(c, gone):
    """gone(r, t): the token's key is far below any other, its score -inf."""
    x = c["pool"].view(c["P"], c["Hkv"], 1, 2, TILE, D)
    c["q"] = c["q"].abs().clamp(min=0.5)
    marks = []
    for r in range(c["B"]):
        mark = np.array([bool(gone(r, t)) for t in range(c["lens"][r])])
        for t in np.flatnonzero(mark):
            x[c["table"][r, t // PS], :, 0, 0, t % PS] = -3e38
        marks.append(mark)
    s = call(c)
    torch.cuda.synchronize()
    assert fpk_decode_status(s["ws"]) == 0
    out, lse = s["out"].double().cpu().numpy(), s["lse"].double().cpu().numpy()
    ro, rl, A, ds = without(c, marks)
    n = int(c["lens"].max())
    assert np.array_equal(np.isneginf(lse), np.isneginf(rl))
    assert not out[np.isneginf(rl)].any()
    assert (np.abs(out - ro) <= 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2 * ds[..., None] + n * 2.0 ** -24) * A).all()
    live = np.isfinite(rl)
    assert (np.abs(lse - rl)[live] <= (ds + n * 2.0 ** -24 + 2.0 ** -20 * np.abs(rl))[live]).all()


@pytest.mark.parametrize("n", [3, 40])
def test_first_token_of_every_page(n):
    run(make([(300, [310 + i % 90 for i in range(n)])], fp8=False, G=8, lead=2), lambda r, t: t % PS == 0)


@pytest.mark.parametrize("n", [3, 40])
def test_whole_prefix(n):
    # rows have their own tokens alone; one that has none is empty
    run(make([(304, [304] + [310 + i % 90 for i in range(n)])], fp8=False, G=8), lambda r, t: t < 304)


def test_first_blocks_of_the_prefix():
    # the running maximum stays -inf through whole blocks and pieces
    run(make([(2000, [2001, 2100, 2000])], fp8=False, Hkv=1, G=8), lambda r, t: t < 1990)


def test_own_tokens():
    # rows have the prefix alone; of requests that share nothing one keeps a token, one none
    run(make([(304, [350, 304, 900]), (0, [300, 290])], fp8=False, G=4),
        lambda r, t: t >= 304 if r < 3 else t != 299)


def test_everything():
    run(make([(304, [350, 304])], fp8=False, G=4, lead=1), lambda r, t: True)
