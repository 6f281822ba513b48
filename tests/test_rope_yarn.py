"""YaRN's ramp wherever its band lies (CPU): before the first pair, over all of them,
behind the last."""
import math

import pytest

from test_rope_freq import freqs


@pytest.mark.parametrize("rot,base,orig,fast,slow", [(64, 10000.0, 131072, 32, 1), (64, 10000.0, 1 << 20, 32, 1), (128, 10000.0, 4096, 32, 1),
                                                     (96, 500000.0, 8192, 32, 1), (128, 10000.0, 3, 32, 1),
                                                     (128, 10000.0, 40, 32, 1), (16, 100.0, 4096, 500, 100),
                                                     (128, 10000.0, 4096, 4.02, 4.0)])
def test_yarn_edges(rot, base, orig, fast, slow):
    # wherever the band lies: pairs faster than it stay, slower ones are divided by the factor, between them
    # the share divided grows with the index, from the pair at the band's fast edge to the one at its slow edge
    f, _ = freqs(rot, base)
    g, _ = freqs(rot, base, scaling="yarn", factor=4.0, original_len=orig, beta_fast=fast, beta_slow=slow)
    place = lambda turns: rot * math.log(orig / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
    lo, hi = math.floor(place(fast)), math.ceil(place(slow))
    for i in range(rot // 2):
        share = min(max((i - lo) / (hi - lo), 0.0), 1.0)
        assert g[i].item() == pytest.approx(f[i].item() * (1 - 0.75 * share), rel=2 ** -22), i
        turns = orig * f[i].item() / (2 * math.pi)
        if turns > fast * base ** (2 / rot):
            assert g[i] == f[i]
        if turns < slow / base ** (2 / rot):
            assert g[i] == f[i] / 4
