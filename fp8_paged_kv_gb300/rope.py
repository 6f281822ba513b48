"""Frequencies of rotary positions, as fpk_rope_append_* and fpk_rope_prefill_* take them."""
from __future__ import annotations

import math

import torch


def rope_inv_freq(rot_dim: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
                  original_len: int | None = None, beta_fast: float = 32.0, beta_slow: float = 1.0,
                  device="cuda"):
    """(inv_freq, rot_scale): float32 [rot_dim / 2] on `device` and the magnitude of
    the rotation.  inv_freq[i] = base ** (-2 i / rot_dim), for contexts `factor`
    times as long as those a model was trained on changed by `scaling`:

    None      nothing
    "linear"  every frequency divided by factor (position interpolation, Chen et al. 2023)
    "ntk"     base multiplied by factor ** (rot_dim / (rot_dim - 2)): the slowest pair is
              divided by factor, the fastest stays
    "yarn"    pairs that turn more than beta_fast times within original_len stay, those
              below beta_slow turns are divided by factor, a linear ramp over the pair
              index between; rot_scale = 0.1 ln(factor) + 1 (YaRN, Peng et al. 2023)
    """
    if rot_dim <= 0 or rot_dim % 2 or not base > 1.0 or not factor >= 1.0:
        raise ValueError("rope_inv_freq: rot_dim is positive and even, base > 1, factor >= 1")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"rope_inv_freq: unknown scaling {scaling!r}")
    if scaling == "ntk":
        if rot_dim < 4:
            raise ValueError("rope_inv_freq: ntk needs two pairs at least")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    f = base ** (-2.0 * i / rot_dim)
    scale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        if not original_len or original_len < 1 or not beta_fast > beta_slow > 0:
            raise ValueError("rope_inv_freq: yarn needs original_len, and beta_fast > beta_slow > 0")

        def pair_of(turns):  # the (fractional) pair that makes so many turns within original_len
            return rot_dim * math.log(original_len / (2 * math.pi * turns)) / (2 * math.log(base))

        # (either may lie before the first pair or behind the last: the ramp's slope is theirs all the same)
        lo, hi = math.floor(pair_of(beta_fast)), math.ceil(pair_of(beta_slow))
        ramp = ((i - lo) / max(hi - lo, 1)).clamp(0.0, 1.0)
        f = f * (1.0 - ramp) + f / factor * ramp
        scale = 0.1 * math.log(factor) + 1.0
    return f.to(torch.float32).to(device), scale
