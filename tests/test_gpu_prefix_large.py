"""Shared-prefix decode attention where a CTA has many blocks and several pieces:
units of one and of two row tiles after one another, prefixes cut over CTAs, own
contexts in several splits; and one workspace for calls of different shapes.  The
reference is the plain attention in 64 bits, on the device; tolerances are those of
the small cases."""
import numpy as np
import pytest
import torch

from fp8_paged_kv_gb300 import fpk_prefix_workspace_bytes
from test_gpu_prefix import BOTH, D, DEV, TILE, call, check, make, reference

pytestmark = pytest.mark.gpu


def reference_on_device(c):
    Hkv, G, ps, P, B = c["Hkv"], c["G"], c["ps"], c["P"], c["B"]
    pool = c["pool"].view(P, Hkv, ps // TILE, 2, TILE * D).to(DEV)
    out, A = torch.zeros(B, Hkv * G, D, dtype=torch.float64), torch.zeros(B, Hkv * G, D, dtype=torch.float64)
    lse, ds = torch.full((B, Hkv * G), -np.inf, dtype=torch.float64), torch.zeros(B, Hkv * G, dtype=torch.float64)
    for r in range(B):
        L = int(c["lens"][r])
        if L <= 0:
            continue
        n = -(-L // ps)
        x = pool[torch.from_numpy(c["table"][r, :n].astype(np.int64)).to(DEV)]
        x = (x.view(torch.float8_e4m3fn).float() if c["fp8"] else x).double()
        k = x[:, :, :, 0].reshape(n, Hkv, -1, TILE, D).permute(1, 0, 2, 3, 4).reshape(Hkv, -1, D)[:, :L]
        v = x[:, :, :, 1].reshape(n, Hkv, -1, D, TILE).permute(1, 0, 2, 4, 3).reshape(Hkv, -1, D)[:, :L]
        if c["fp8"]:
            k, v = k * float(np.float32(c["ks"])), v * float(np.float32(c["vs"]))
        q = c["q"][r].to(DEV).double().view(Hkv, G, D)
        s = q @ k.transpose(1, 2) * c["sm"]
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        z = p.sum(-1, keepdim=True)
        out[r], A[r] = (p @ v / z).reshape(-1, D).cpu(), (p @ v.abs() / z).reshape(-1, D).cpu()
        lse[r] = (m + z.log()).reshape(-1).cpu()
        ds[r] = (2 * 2.0 ** -17 * q.abs().amax(-1) * k.abs().sum(-1).amax(-1)[:, None] * abs(c["sm"])).reshape(-1).cpu()
    return out.numpy(), lse.numpy(), A.numpy(), ds.numpy()


SCENES = {
    # 768 rows a head: three units of both tiles, each cut over many CTAs
    "one group": dict(groups=[(9000, [9001 + 37 * i % 500 for i in range(96)])], Hkv=4, G=8, ps=64),
    # 640 rows and 12: a unit of one tile after two of both
    "odd tail": dict(groups=[(5003, [5004 + 61 * i % 300 for i in range(163)])], Hkv=2, G=4, ps=32),
    # units of one tile and of both, short and long prefixes, in turn
    "mixed": dict(groups=[(7000, [7100] * 2), (3000, [3500 + i for i in range(33)]), (1500, [1501] * 5),
                          (4777, [5000 - 13 * i for i in range(17)]), (200, [1800] * 40), (8000, [8191] * 3)],
                  Hkv=8, G=5, ps=16, lead=2, tail=2),
    # many groups that each fit one tile
    "small units": dict(groups=[(600 + 131 * i, [601 + 131 * i + 5 * r for r in range(2 + i % 5)]) for i in range(40)],
                        Hkv=4, G=7, ps=16),
}


@BOTH
@pytest.mark.parametrize("name", SCENES)
def test_many_blocks_and_pieces(fp8, name):
    c = make(**SCENES[name], fp8=fp8, sigma=1.6, seed=len(name))
    ref = reference_on_device(c)
    s = call(c)
    check(c, s, ref, name)
    first = s["out"].clone(), s["lse"].clone()
    for _ in range(3):
        call(c, state=s)
    check(c, s, ref, name)
    assert torch.equal(first[0], s["out"]) and torch.equal(first[1], s["lse"])


@BOTH
def test_one_workspace_for_every_shape(fp8):
    """Calls of other shapes in between, with and without groups, leave nothing behind that a call would read."""
    shapes = [dict(groups=[(300, [400, 350, 301])], Hkv=2, G=4, ps=16), dict(groups=[], Hkv=8, G=8, ps=16, lead=9),
              dict(groups=[(1000, [1100] * 70)], Hkv=1, G=8, ps=64), dict(groups=[], Hkv=1, G=1, ps=32, lead=3),
              dict(groups=[(64, [65] * 5), (129, [700, 130])], Hkv=4, G=2, ps=16, lead=1)]
    cases = [make(**x, fp8=fp8, seed=i) for i, x in enumerate(shapes)]
    refs = [reference(c) for c in cases]
    n = max(fpk_prefix_workspace_bytes(c["B"], c["Hkv"] * c["G"], c["Hkv"]) for c in cases)
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    states = [call(c, ws=ws) for c in cases]
    for i in (0, 2, 1, 4, 3, 1, 0, 3, 2, 4):
        states[i]["out"].fill_(float("nan"))
        states[i]["lse"].fill_(float("nan"))
        call(cases[i], state=states[i])
        check(cases[i], states[i], refs[i], f"shape {i}")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c, s in zip(cases, states):
            call(c, state=s, stream=torch.cuda.current_stream())
    for s in states:
        s["out"].fill_(float("nan"))
    graph.replay()
    for c, s, ref in zip(cases, states, refs):
        check(c, s, ref, "graph")


@BOTH
@pytest.mark.parametrize("G,ps", [(1, 16), (2, 32), (3, 64), (5, 256), (6, 16), (7, 128), (8, 16)])
def test_no_groups_shapes(fp8, G, ps):
    c = make([], fp8=fp8, Hkv=3, G=G, ps=ps, lead=13, tail=2, seed=G)
    check(c, call(c), reference(c))


@BOTH
def test_no_groups_dead_requests(fp8):
    c = make([], fp8=fp8, lead=6, seed=3)
    table, lens = c["table"].copy(), c["lens"].copy()
    abort = np.array([0, 1, 0, 0, 0, 0], np.uint8)
    table[2, 1], table[3, 0], table[4, 0] = -1, c["P"], -9
    lens[5] = table.shape[1] * c["ps"] + 1
    lens[0] = 0
    check(c, call(c, abort=abort, table=table, lens=lens), reference(c, abort=abort, table=table, lens=lens))


@BOTH
def test_more_groups_than_a_warp_looks_up_at_once(fp8):
    groups = [(40 + i % 90, [41 + i % 90 + (7 * i + r) % 60 for r in range(2 + i % 2)]) for i in range(150)]
    c = make(groups, fp8=fp8, Hkv=1, G=4, lead=3, seed=8)
    assert c["B"] > 256
    check(c, call(c), reference(c))
    lens = c["lens"].copy()
    lens[::5] = 0                      # groups whose first, last or all requests are dead
    check(c, call(c, lens=lens), reference(c, lens=lens))
