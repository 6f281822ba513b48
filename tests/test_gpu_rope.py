"""GPU parity of rotary positions with the cache write, against 64-bit rotations.

Tolerances: a rotated value v in fp32 is off by at most (2^-20 + 3 2^-24) times
the pair's magnitude R = rot_scale (|x| + |y|) (the cosine and sine by 2^-20, two
products and a sum by half a step each); bf16 results add half a step,
2^-8 |v|.  e4m3 codes equal those of v / scale computed in 64 bits, except where
v / scale lies that close to a rounding boundary: such a code may be the next
one.  Values and their codes are bit-exact, and nothing else is written.
"""
import numpy as np
import pytest
import torch

import oracle
from fp8_paged_kv_gb300 import (fpk_kv_append_fp8, fpk_rope_append_bf16, fpk_rope_append_fp8,
                                fpk_rope_prefill_bf16, fpk_rope_prefill_fp8)
from fp8_paged_kv_gb300.rope import rope_inv_freq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D, TILE = 128, 16
KS, VS = np.float32(0.013), np.float32(0.021)


def rotated(x, pos, f, rot, inter, scale):
    """x float64 [T][H][D] rotated, and the magnitude of each value's pair."""
    y, mag = x.copy(), np.abs(x)
    a = pos.astype(np.float64)[:, None, None] * f.astype(np.float64)
    c, s = np.cos(a) * np.float64(np.float32(scale)), np.sin(a) * np.float64(np.float32(scale))
    i0, i1 = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    p, q = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = p * c - q * s, q * c + p * s
    mag[..., i0] = mag[..., i1] = (np.abs(p) + np.abs(q)) * abs(scale)
    return y, mag


def scene(T_of, first, *, fp8, Hq, Hkv, ps, seed, spare=2):
    """Requests with T_of[r] new tokens from position first[r]; a pool of sentinels."""
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    T, B = sum(T_of), len(T_of)
    ends = [f + t for f, t in zip(first, T_of)]
    maxp = max(1, max(-(-e // ps) for e in ends))
    need = [list(range(f // ps, -(-e // ps))) if t else [] for f, e, t in zip(first, ends, T_of)]
    P = sum(map(len, need)) + spare
    perm = rng.permutation(P)
    table, at = np.full((B, maxp), -1, np.int32), 0
    for r, js in enumerate(need):
        for j in js:
            table[r, j] = perm[at]
            at += 1
    bf = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
    tags = rng.integers(0, 1 << 31, P).astype(np.int32)
    n = 2 * P * Hkv * ps * D
    return dict(fp8=fp8, Hq=Hq, Hkv=Hkv, ps=ps, B=B, T=T, P=P, table=table, live=tags,
                expected=np.where(table >= 0, tags[np.maximum(table, 0)], 0).astype(np.int32),
                q=bf(T, Hq, D) if Hq else None, k=bf(T, Hkv, D), v=bf(T, Hkv, D),
                cu=np.concatenate([[0], np.cumsum(T_of)]).astype(np.int32), first=np.array(first, np.int32),
                pos=np.concatenate([np.arange(f, f + t) for f, t in zip(first, T_of)] or [[]]).astype(np.int64),
                req=np.repeat(np.arange(B), T_of), n=n,
                pool=np.full(n, 0xA5 if fp8 else 0xA5A5, np.uint8 if fp8 else np.uint16))


def dev(x):
    if x is None or isinstance(x, torch.Tensor):
        return None if x is None else x.to(DEV)
    return torch.from_numpy(x.view(np.int16) if x.dtype == np.uint16 else x).to(DEV)


def launch(c, f, *, rot, inter=False, scale=1.0, append=False, guard=False, in_place=False, start=True, stream=None,
           state=None):
    s = state if state is not None else {}
    if not s:
        s.update({k: dev(c[k]) for k in ("q", "k", "v", "cu", "first", "table", "live", "expected", "pool")})
        if not c["fp8"]:
            s["pool"] = s["pool"].view(torch.bfloat16)
        s["lens"] = dev((c["first"] + np.diff(c["cu"])).astype(np.int32))
        s["qo"] = s["q"] if in_place or s["q"] is None else torch.full_like(s["q"], 7.0)
        s["f"] = dev(f)
        s["ks"], s["vs"] = dev(np.array([KS])), dev(np.array([VS]))
        s["abort"] = torch.zeros(c["B"], dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
    tags = (s["live"], s["expected"], s["abort"]) if guard else ()
    sc = (s["ks"], s["vs"]) if c["fp8"] else ()
    kw = dict(Hkv=c["Hkv"], page_size=c["ps"], num_pages=c["P"], rot_dim=rot, interleaved=inter, rot_scale=scale,
              stream=stream)
    if append:
        (fpk_rope_append_fp8 if c["fp8"] else fpk_rope_append_bf16)(
            s["q"], s["k"], s["v"], s["f"], s["qo"], s["pool"], *sc, s["table"], s["lens"], *tags, **kw)
    else:
        (fpk_rope_prefill_fp8 if c["fp8"] else fpk_rope_prefill_bf16)(
            s["q"], s["k"], s["v"], s["cu"], s["first"] if start else None, s["f"], s["qo"], s["pool"], *sc,
            s["table"], *tags, **kw)
    return s


def check(c, s, f, *, rot, inter=False, scale=1.0, refused=()):
    torch.cuda.synchronize()
    eps = 2.0 ** -20 + 3 * 2.0 ** -24
    if c["Hq"]:
        y, mag = rotated(c["q"].double().numpy(), c["pos"], f, rot, inter, scale)
        got = s["qo"].double().cpu().numpy()
        turned = np.arange(D) < rot
        err = np.abs(got - y)
        assert (err <= 2.0 ** -8 * np.abs(y) + eps * mag * turned + 1e-30).all(), err.max()
        assert np.array_equal(got[..., rot:], c["q"].double().numpy()[..., rot:])
    y, mag = rotated(c["k"].double().numpy(), c["pos"], f, rot, inter, scale)
    mag = mag * (np.arange(D) < rot)
    Hkv, ps, P = c["Hkv"], c["ps"], c["P"]
    shape = (P, Hkv, ps // TILE, 2, TILE * D)
    got = s["pool"].cpu() if c["fp8"] else s["pool"].view(torch.int16).cpu()
    got = got.numpy().reshape(shape)
    got = got if c["fp8"] else got.view(np.uint16)
    kg, vg = got[..., 0, :].reshape(*shape[:3], TILE, D), got[..., 1, :].reshape(*shape[:3], D, TILE)
    want = c["pool"].reshape(shape).copy()
    kw, vw = want[..., 0, :].reshape(*shape[:3], TILE, D), want[..., 1, :].reshape(*shape[:3], D, TILE)
    kept = [i for i in range(c["T"]) if i not in refused and (c["req"][i], "all") not in refused]
    page = c["table"][c["req"], c["pos"] // ps] if c["T"] else []
    at = lambda i: (page[i], slice(None), c["pos"][i] % ps // TILE)  # noqa: E731
    vbits = c["v"].view(torch.int16).numpy().view(np.uint16)
    for i in kept:
        p, _, t = at(i)
        row = c["pos"][i] % TILE
        g = kg[p, :, t, row]
        if c["fp8"]:
            v = y[i] / np.float64(KS)
            tol = (eps * mag[i] + 2.0 ** -23 * np.abs(y[i])) / np.float64(KS)   # one more step for the division
            lo, hi = (oracle.e4m3_decode(oracle.e4m3_encode((v + d).astype(np.float32))) for d in (-tol, tol))
            val = oracle.e4m3_decode(g)
            assert ((val >= lo) & (val <= hi)).all()
            exact = oracle.e4m3_decode(oracle.e4m3_encode(v.astype(np.float32)))
            assert (val != exact).mean() < 0.01
            assert np.array_equal(vg[p, :, t, :, row], oracle.quantize_bf16(vbits[i], VS))
        else:
            val = torch.from_numpy(g.view(np.int16).copy()).view(torch.bfloat16).double().numpy()
            assert (np.abs(val - y[i]) <= 2.0 ** -8 * np.abs(y[i]) + eps * mag[i] + 1e-30).all()
            assert np.array_equal(vg[p, :, t, :, row], vbits[i])
        kw[p, :, t, row], vw[p, :, t, :, row] = g, vg[p, :, t, :, row]
    assert np.array_equal(kg, kw) and np.array_equal(vg, vw), "slots of other tokens changed"


BOTH = pytest.mark.parametrize("fp8", [True, False])
LAYOUT = pytest.mark.parametrize("inter", [False, True])


def freqs(rot):
    return rope_inv_freq(rot, 10000.0, device="cpu")[0].numpy()


@BOTH
@LAYOUT
@pytest.mark.parametrize("rot", [16, 32, 48, 64, 96, 112, 128])
def test_prefill(fp8, inter, rot):
    c = scene([37, 0, 1, 16, 100, 15], [0, 0, 0, 0, 0, 0], fp8=fp8, Hq=8, Hkv=2, ps=32, seed=rot)
    f = freqs(rot)
    for start in (True, False):
        check(c, launch(c, f, rot=rot, inter=inter, scale=1.25, start=start), f, rot=rot, inter=inter, scale=1.25)


@BOTH
@LAYOUT
@pytest.mark.parametrize("ps", [16, 64, 256])
def test_chunks_from_any_position(fp8, inter, ps):
    c = scene([5, 40, 17, 1, 16, 33], [3, 1000, 15, 4095, 16, 77], fp8=fp8, Hq=5, Hkv=5, ps=ps, seed=ps)
    f = freqs(64)
    check(c, launch(c, f, rot=64, inter=inter), f, rot=64, inter=inter)


@BOTH
@LAYOUT
@pytest.mark.parametrize("B,Hq,Hkv", [(1, 64, 8), (1, 1, 1), (3, 7, 1), (64, 8, 8), (300, 40, 8), (5, 32, 32)])
def test_append(fp8, inter, B, Hq, Hkv):
    c = scene([1] * B, [(17 * r * r) % 900 for r in range(B)], fp8=fp8, Hq=Hq, Hkv=Hkv, ps=16, seed=B + Hq)
    f = freqs(96)
    s = launch(c, f, rot=96, inter=inter, append=True, guard=True)
    check(c, s, f, rot=96, inter=inter)
    assert not s["abort"].any()


@BOTH
def test_far_positions(fp8):
    # angles near the ends of int32: in fp32 the product alone would be off by whole turns
    f = freqs(128)
    first = [2 ** 24 - 1, 2 ** 24 + 1, 131071]
    c = scene([1, 1, 1], first, fp8=fp8, Hq=4, Hkv=2, ps=256, seed=1)
    check(c, launch(c, f, rot=128, append=True), f, rot=128)
    check(c, launch(c, f, rot=128), f, rot=128)


def test_last_int32_position():
    # no table reaches it: the query is rotated, the key refused
    f = freqs(128)
    c = scene([1], [0], fp8=True, Hq=4, Hkv=2, ps=256, seed=1)
    s = launch(c, f, rot=128, append=True, guard=True)
    s["lens"].fill_(2 ** 31 - 1)
    s["pool"].fill_(0xA5)
    launch(c, f, rot=128, append=True, guard=True, state=s)
    c["pos"][:] = 2 ** 31 - 2
    c["table"] = np.zeros((1, (2 ** 31) // 256), np.int32)
    check(c, s, f, rot=128, refused=(0,))
    assert s["abort"].tolist() == [1]


@BOTH
def test_in_place_and_without_queries(fp8):
    f = freqs(128)
    c = scene([20, 3], [5, 0], fp8=fp8, Hq=6, Hkv=3, ps=16, seed=3)
    check(c, launch(c, f, rot=128, in_place=True), f, rot=128)
    c = scene([20, 3], [5, 0], fp8=fp8, Hq=0, Hkv=3, ps=16, seed=3)
    check(c, launch(c, f, rot=128), f, rot=128)


@BOTH
@pytest.mark.parametrize("append", [True, False])
def test_guard(fp8, append):
    """Stale tags, pages out of range and positions behind the table: those tokens are not written."""
    n = [1] * 6 if append else [20] * 6
    c = scene(n, [40, 41, 42, 43, 44, 45], fp8=fp8, Hq=4, Hkv=2, ps=32, seed=8)
    j = 1
    c["expected"][0, j] += 1
    c["table"][1, j], c["table"][2, j] = -1, c["P"]
    f = freqs(64)
    s = launch(c, f, rot=64, append=append, guard=True)
    bad = [i for i in range(c["T"]) if c["req"][i] < 3 and c["pos"][i] // 32 == j]
    safe = dict(c, table=np.where((c["table"] >= 0) & (c["table"] < c["P"]), c["table"], 0))
    check(safe, s, f, rot=64, refused=bad)
    assert s["abort"].tolist() == [1, 1, 1, 0, 0, 0]
    # without tags only the pages out of range are refused, and no mask is needed
    s = launch(c, f, rot=64, append=append)
    check(safe, s, f, rot=64, refused=[i for i in bad if c["req"][i] > 0])


@BOTH
def test_empty_requests_are_left_alone(fp8):
    f = freqs(64)
    c = scene([1, 1, 1], [9, 10, 11], fp8=fp8, Hq=4, Hkv=2, ps=16, seed=2)
    s = launch(c, f, rot=64, append=True, guard=True)
    s["lens"][1] = 0
    s["qo"].fill_(7.0)
    s["pool"].copy_(dev(c["pool"]) if fp8 else dev(c["pool"]).view(torch.bfloat16))
    launch(c, f, rot=64, append=True, guard=True, state=s)
    torch.cuda.synchronize()
    assert (s["qo"][1] == 7.0).all() and not s["abort"].any()
    s["qo"][1] = torch.from_numpy(rotated(c["q"].double().numpy(), c["pos"], f, 64, False, 1.0)[0][1]).to(DEV)
    check(c, s, f, rot=64, refused=(1,))


def test_nan_inf_and_saturation():
    f = freqs(128)
    c = scene([4], [0], fp8=True, Hq=1, Hkv=1, ps=16, seed=4)
    c["k"][0, 0, :] = float("nan")
    c["v"][1, 0, :] = float("inf")
    c["k"][2, 0, :], c["k"][3, 0, :] = 1e30, 0.0
    s = launch(c, f, rot=128)
    torch.cuda.synchronize()
    pool = s["pool"].cpu().numpy().reshape(c["P"], 1, 1, 2, TILE * D)[c["table"][0, 0], 0, 0]
    k, v = pool[0].reshape(TILE, D), pool[1].reshape(D, TILE)
    assert ((k[0] & 0x7F) == 0x7F).all() and (v[:, 1] == 0x7E).all()
    assert ((k[2] & 0x7F) == 0x7E).all() and ((k[3] & 0x7F) == 0).all()


def test_unrotated_write_equals_the_append():
    # position 0 turns nothing: the bytes are those of fpk_kv_append_fp8
    c = scene([1] * 5, [0] * 5, fp8=True, Hq=4, Hkv=3, ps=16, seed=5)
    s = launch(c, freqs(128), rot=128, append=True)
    pool = dev(c["pool"])
    fpk_kv_append_fp8(s["k"], s["v"], pool, s["ks"], s["vs"], s["table"], s["lens"], Hkv=3, D=D, page_size=16,
                      num_pages=c["P"])
    torch.cuda.synchronize()
    assert torch.equal(pool, s["pool"])


@BOTH
@pytest.mark.parametrize("append", [True, False])
def test_stream_and_graph(fp8, append):
    f = freqs(64)
    n, first = ([1] * 3, [9, 10, 700]) if append else ([30, 1, 50], [9, 10, 700])
    c = scene(n, first, fp8=fp8, Hq=4, Hkv=2, ps=16, seed=2)
    side = torch.cuda.Stream(device=DEV)
    s = launch(c, f, rot=64, append=append, stream=side)
    side.synchronize()
    check(c, s, f, rot=64)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        launch(c, f, rot=64, append=append, state=s)
    other = scene(n, first, fp8=fp8, Hq=4, Hkv=2, ps=16, seed=6)
    for key in ("q", "k", "v", "table"):
        s[key].copy_(dev(other[key]))
    s["pool"].copy_(dev(other["pool"]) if fp8 else dev(other["pool"]).view(torch.bfloat16))
    g.replay()
    check(other, s, f, rot=64)


def test_many_requests():
    # more requests than one CTA's scan holds
    n = [(r % 3) for r in range(5000)]
    c = scene(n, [(7 * r) % 40 for r in range(5000)], fp8=True, Hq=1, Hkv=1, ps=16, seed=9)
    f = freqs(32)
    check(c, launch(c, f, rot=32), f, rot=32)


@BOTH
def test_shortest_lengths_leave_everything(fp8):
    for low in (0, -1, -2 ** 31):
        c = scene([1, 1, 1], [3, 40, 7], fp8=fp8, Hq=4, Hkv=2, ps=16, seed=12)
        f = freqs(64)
        s = launch(c, f, rot=64, append=True, guard=True)
        torch.cuda.synchronize()
        s["pool"].copy_(dev(c["pool"]).view(s["pool"].dtype))
        s["qo"].fill_(7.0)
        s["abort"].zero_()
        s["lens"].fill_(low)
        launch(c, f, rot=64, append=True, guard=True, state=s)
        torch.cuda.synchronize()
        assert (s["qo"] == 7.0).all() and not s["abort"].any()
        assert torch.equal(s["pool"].view(torch.uint8).cpu(), torch.from_numpy(c["pool"]).view(torch.uint8))


@BOTH
@pytest.mark.parametrize("t0,n", [(0, 1), (1, 14), (2, 13), (3, 9), (4, 8), (5, 11), (8, 8), (7, 2), (0, 15), (15, 1), (15, 33)])
def test_ragged_tiles(fp8, t0, n):
    # every width of piece that a tile's values may be written in
    c = scene([n, 0, n], [t0, 5, 32 + t0], fp8=fp8, Hq=9, Hkv=9, ps=32, seed=t0 * 16 + n)
    f = freqs(96)
    check(c, launch(c, f, rot=96), f, rot=96)


def test_more_tokens_than_offsets_name():
    # rows behind the last request are nobody's: left as they are
    c = scene([20, 5], [0, 3], fp8=True, Hq=4, Hkv=2, ps=16, seed=5)
    f = freqs(128)
    whole = {k: torch.cat([c[k], torch.ones(9, *c[k].shape[1:], dtype=c[k].dtype)]) for k in ("q", "k", "v")}
    s = launch(dict(c, **whole), f, rot=128)
    torch.cuda.synchronize()
    assert (s["qo"][c["T"]:] == 7.0).all()
    s["qo"] = s["qo"][:c["T"]]
    check(c, s, f, rot=128)
