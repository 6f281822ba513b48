"""Requests that have no answer beside requests that have one, many units to a CTA: every live row
against 64 bits, every row of a dead request (by its abort flag, a bad page, an empty context) and
every row that sees nothing exactly 0 and -inf."""
import pytest

from block_torch import check_rows
from test_gpu_block_attention import SM, run, scene

pytestmark = pytest.mark.gpu
HEADS = [(64, 8), (40, 8), (8, 8), (16, 8), (32, 8)]


def kill(s, dead, how):
    mask = [0] * len(s["counts"])
    for r in dead:
        if how == "flag":
            mask[r] = 1
        elif how == "page":
            s["table"][r, (int(s["lens"][r]) - 1) // s["ps"]] = s["P"]
        else:
            s["lens"][r] = 0
    return mask


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("dead,how", [((0,), "flag"), ((3,), "page"), ((7,), "empty"), ((1, 2, 5), "flag")])
def test_prompts(Hq, Hkv, causal, dead, how):
    s = scene([1024] * 8, [1024] * 8, Hq=Hq, Hkv=Hkv, ps=64, seed=Hq + len(dead))
    check_rows(s, run(s, causal=causal, mask=kill(s, dead, how)), causal=causal, sm=SM, dead=dead)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("B,how", [(64, "flag"), (30, "page"), (64, "empty")])
def test_drafts(Hq, Hkv, B, causal, how):
    """Units of one row tile, of a warp's 32 rows (some more at 5 heads to a kv head), two dead neighbours at a time."""
    n = -(-32 * Hkv // Hq)
    lens = [n + 37 * r % 600 for r in range(B)]
    s = scene(lens, [n] * B, Hq=Hq, Hkv=Hkv, ps=16, seed=Hq + B)
    dead = tuple(r for r in range(B) if r % 7 in (1, 2) or r == B - 1)
    check_rows(s, run(s, causal=causal, mask=kill(s, dead, how)), causal=causal, sm=SM, dead=dead)


@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_rows_before_their_context(Hq, Hkv):
    """Causal chunks much longer than their context: units that see nothing beside units that see something."""
    lens, counts = [300, 2, 520, 33, 700, 1, 260, 900], [300, 600, 520, 700, 90, 513, 800, 300]
    s = scene(lens, counts, Hq=Hq, Hkv=Hkv, ps=32, seed=Hq)
    check_rows(s, run(s, causal=True), causal=True, sm=SM)


@pytest.mark.parametrize("causal", [True, False])
def test_all_dead_but_one(causal):
    s = scene([700] * 12, [512] * 12, Hq=64, Hkv=8, ps=16, seed=5)
    dead = tuple(r for r in range(12) if r != 9)
    check_rows(s, run(s, causal=causal, mask=kill(s, dead, "flag")), causal=causal, sm=SM, dead=dead)
