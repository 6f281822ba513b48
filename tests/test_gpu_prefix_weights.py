"""Softmax weights of shared-prefix attention: as exact as those of the framework's
other decode attention, which the outputs show where values nearly cancel.

A weight enters the second product as two parts, each rounded by half a step at
most, the second one what the first left: w = 2^-11 2^-11 (f16, e4m3 cache) or
2^-8 2^-8 (bf16 cache) of it.  f16 parts below 2^-14 are off by up to 2^-25 instead,
of at least the largest weight's 1.  So per output |d| <= 2^-8 |ref| +
(w + 2 ds + n 2^-24) A + n 2^-25 max |v| / z (e4m3 cache alone), A the weighted mean of
|v|, ds the error of a score, z the sum of exp(s - max) (which is at least 1).
"""
import math

import numpy as np
import pytest
import torch

from fp8_paged_kv_gb300 import fpk_decode_status
from test_gpu_prefix import BOTH, D, TILE, call, make, reference

pytestmark = pytest.mark.gpu


def close(c, s, ref):
    torch.cuda.synchronize()
    assert fpk_decode_status(s["ws"]) == 0
    ro, _, A, ds = ref
    n = int(c["lens"].max())
    v = c["pool"].view(c["P"], c["Hkv"], c["ps"] // TILE, 2, TILE * D)[..., 1, :]
    v = v.view(torch.float8_e4m3fn).float() * c["vs"] if c["fp8"] else v.float()
    w, small = (2.0 ** -22, n * 2.0 ** -25 * v.nan_to_num(0).abs().max().item()) if c["fp8"] else (2.0 ** -16, 0.0)
    tol = 2.0 ** -8 * np.abs(ro) + (w + 2 * ds[..., None] + n * 2.0 ** -24) * A + small
    err = np.abs(s["out"].double().cpu().numpy() - ro)
    assert (err <= tol).all(), f"{(err / tol).max():.2f} of the tolerance"


def cancelling(fp8, **k):
    """Tokens in turn of weight 1 and p, of values x and -y with x / y near p: what is left is
    the error of p.  p lies 0.15 of a step of one part above a value halfway between two."""
    c = make(fp8=fp8, Hkv=1, seed=3, **k)
    pool = c["pool"].view(c["P"], 1, c["ps"] // TILE, 2, TILE * D)
    x, y, p, key = (11.0, 13.0, 3465.3 / 4096, 8.0) if fp8 else (217 / 256, 1.0, 433.3 / 512, 1.0)
    kv = torch.zeros(TILE, D), torch.zeros(D, TILE)
    kv[0][1::2, 0] = -key
    size = 2.0 ** (torch.arange(D) % 4 - 2.0)
    kv[1][:, 0::2], kv[1][:, 1::2] = (size * x)[:, None], (-size * y)[:, None]
    for i in range(2):
        t = kv[i].reshape(-1)
        pool[..., i, :] = t.to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else t.to(torch.bfloat16)
    c["q"].zero_()
    c["q"][..., 0] = 1.0
    c["sm"] = -math.log(p) / (key * (float(np.float32(c["ks"])) if fp8 else 1.0))
    return c


@BOTH
@pytest.mark.parametrize("n", [3, 40])
def test_cancelling_values_in_the_prefix(fp8, n):
    # 24 and 320 rows: one row tile in turn, and both
    c = cancelling(fp8, groups=[(256, [257 + i % 3 for i in range(n)])], G=8)
    close(c, call(c), reference(c))


@BOTH
def test_cancelling_values_of_a_request_alone(fp8):
    c = cancelling(fp8, groups=[(32, [300, 200, 256]), (0, [256, 128, 511])], G=5, lead=2)
    close(c, call(c), reference(c))


@BOTH
def test_outlier_channels(fp8):
    # a few dims of V thirty times as large
    c = make([(400, [401, 500, 450, 610]), (0, [256, 300])], fp8=fp8, G=8, seed=4, sigma=0.25)
    pool = c["pool"].view(c["P"], 2, c["ps"] // TILE, 2, TILE * D)
    v = pool[..., 1, :].reshape(c["P"], 2, -1, D, TILE)
    if fp8:
        small = (v.view(torch.float8_e4m3fn).float() / 16).to(torch.float8_e4m3fn)
        small[..., ::37, :] = (small[..., ::37, :].float() * 30).to(torch.float8_e4m3fn)
        v = small.view(torch.uint8)
    else:
        v = v.clone()
        v[..., ::37, :] *= 30
    pool[..., 1, :] = v.reshape(pool[..., 1, :].shape)
    close(c, call(c), reference(c))
