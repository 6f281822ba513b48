"""Frequencies of rotary positions (CPU): the plain rule, and what each long-context
scaling leaves and divides."""
import math

import pytest
import torch

from fp8_paged_kv_gb300.rope import rope_inv_freq


def freqs(*a, **k):
    f, s = rope_inv_freq(*a, device="cpu", **k)
    return f.double(), s


def test_plain_and_linear():
    f, s = freqs(64, 10000.0)
    assert s == 1.0 and f.shape == (32,)
    for i in range(32):
        assert f[i].item() == pytest.approx(10000.0 ** (-i / 32), rel=2 ** -24)
    g, _ = freqs(64, 10000.0, scaling="linear", factor=4.0)
    assert torch.equal(g, f / 4)                       # a power of two divides exactly


def test_ntk_ends():
    f, _ = freqs(128, 10000.0)
    g, _ = freqs(128, 10000.0, scaling="ntk", factor=8.0)
    assert g[0] == f[0] and (g[-1] * 8 / f[-1]).item() == pytest.approx(1, rel=1e-6)
    assert bool((g[1:] < f[1:]).all())


def test_yarn_bands():
    f, _ = freqs(128, 10000.0)
    g, s = freqs(128, 10000.0, scaling="yarn", factor=8.0, original_len=4096)
    assert s == pytest.approx(0.1 * math.log(8) + 1)
    turns = 4096 * f / (2 * math.pi)
    i = torch.arange(64)
    fast, slow = i[turns > 32 * 1.2], i[turns < 1 / 1.2]
    assert len(fast) and len(slow)
    assert torch.equal(g[fast], f[fast]) and torch.equal(g[slow], f[slow] / 8)
    ratio = f / g
    assert bool((ratio[1:] >= ratio[:-1] - 1e-6).all()) and ratio.max() <= 8 and ratio.min() >= 1


@pytest.mark.parametrize("bad", [dict(rot_dim=0), dict(rot_dim=15), dict(rot_dim=16, base=1.0),
                                 dict(rot_dim=16, factor=0.5), dict(rot_dim=16, scaling="other"),
                                 dict(rot_dim=2, scaling="ntk", factor=2.0),
                                 dict(rot_dim=16, scaling="yarn", factor=2.0),
                                 dict(rot_dim=16, scaling="yarn", original_len=512, beta_fast=1.0)])
def test_refusals(bad):
    with pytest.raises(ValueError):
        rope_inv_freq(**bad, device="cpu")
