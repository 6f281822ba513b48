"""Softmax weights of decode attention over block scales where little is left of them: values that cancel, a block beside
one whose V scale is far larger, tokens beside one that has nearly all the weight.

A weight enters the second product as two f16 parts of up to 2^14, each rounded by half a step at most, the second one
what the first left: off by 2^-11 2^-11 of it, and by 2^-25 2^-14 of the largest weight times V's scale where the second
part is below 2^-14."""
import pytest

from block_torch import cancelling, check_rows, outlier_block, sink
from test_gpu_block_attention import SM, run, scene

pytestmark = pytest.mark.gpu
TWO_PARTS = dict(weight=2.0 ** -22, floor=2.0 ** -39)


@pytest.mark.parametrize("Hq,Hkv", [(16, 2), (7, 1), (4, 4)])
def test_cancelling_values(Hq, Hkv):
    s = scene([256, 47, 1000], [1] * 3, Hq=Hq, Hkv=Hkv, ps=32, seed=3)
    sm = cancelling(s)
    check_rows(s, run(s, sm=sm), causal=None, sm=sm, **TWO_PARTS)


@pytest.mark.parametrize("splits", [0, 1])  # (1: a request's tiles meet in one CTA)
@pytest.mark.parametrize("far", [8, 16, 20, 24])
def test_a_block_of_a_far_larger_scale(far, splits):
    s = scene([48, 700, 200, 33], [1] * 4, Hq=16, Hkv=2, ps=32, seed=far, spread=0)
    outlier_block(s, far)
    check_rows(s, run(s, splits=splits), causal=None, sm=SM, **TWO_PARTS)


@pytest.mark.parametrize("far", [12, 20, 28, 34])
def test_a_token_of_nearly_all_the_weight(far):
    s = scene([1000, 77, 17], [1] * 3, Hq=16, Hkv=2, ps=16, seed=far, spread=0)
    sm = sink(s, far)
    check_rows(s, run(s, sm=sm), causal=None, sm=sm, **TWO_PARTS)
