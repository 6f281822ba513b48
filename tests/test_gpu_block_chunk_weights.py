"""Softmax weights of prompt attention where little is left of them: values that cancel, a block beside one whose V
scale is far larger, tokens beside one that has nearly all the weight.

A weight enters the second product as two f16 parts, each rounded by half a step at most, the second one what the first
left: off by 2^-11 2^-11 of it.  The largest weight times V's scale is 2^7 at least there, and a second part below 2^-14
is off by 2^-25: by 2^-32 of that largest one."""
import pytest

from block_torch import cancelling, check_rows, outlier_block, sink
from test_gpu_block_attention import SM, run, scene

pytestmark = pytest.mark.gpu
TWO_PARTS = dict(weight=2.0 ** -22, floor=2.0 ** -32)
BOTH = pytest.mark.parametrize("causal", [True, False])


@BOTH
@pytest.mark.parametrize("Hq,Hkv", [(16, 2), (10, 2), (4, 4)])
@pytest.mark.parametrize("lens,counts", [([256, 47, 1000], [4, 47, 300]), ([700] * 30, [65] * 30), ([9000], [3])])
def test_cancelling_values(Hq, Hkv, lens, counts, causal):
    s = scene(lens, counts, Hq=Hq, Hkv=Hkv, ps=32, seed=3)
    sm = cancelling(s)
    check_rows(s, run(s, causal=causal, sm=sm), causal=causal, sm=sm, **TWO_PARTS)


@BOTH
@pytest.mark.parametrize("far", [8, 16, 20, 24])
def test_a_block_of_a_far_larger_scale(far, causal):
    s = scene([48, 700, 200, 33], [4, 100, 200, 1], Hq=16, Hkv=2, ps=32, seed=far, spread=0)
    outlier_block(s, far)
    check_rows(s, run(s, causal=causal), causal=causal, sm=SM, **TWO_PARTS)


@BOTH
@pytest.mark.parametrize("far", [12, 18, 24])
def test_a_token_of_nearly_all_the_weight(far, causal):
    s = scene([1000, 77, 700], [40, 77, 300], Hq=16, Hkv=2, ps=16, seed=far, spread=0)
    sm = sink(s, far)
    check_rows(s, run(s, causal=causal, sm=sm), causal=causal, sm=sm, **TWO_PARTS)


@BOTH
def test_values_as_they_come(causal):
    """Ordinary values, every row: prompts, chunks behind a context, drafts."""
    s = scene([1024, 2000, 130, 600], [1024, 300, 4, 5], Hq=16, Hkv=2, ps=64, seed=8)
    check_rows(s, run(s, causal=causal), causal=causal, sm=SM, **TWO_PARTS)
