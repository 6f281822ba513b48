"""GPU parity of forks and compactions with numpy: bytes, tables, lengths and tags
are bit-exact, refused ones fail closed, and nothing else changes."""
import numpy as np
import pytest
import torch

from fp8_paged_kv_gb300 import fpk_kv_compact, fpk_kv_fork

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D, TILE = 128, 16


def scene(lens, *, el=1, Hkv=2, ps=16, layers=1, spare=12, extra=2, seed=0):
    rng = np.random.default_rng(seed)
    n = [-(-x // ps) for x in lens]
    B, P = len(lens), sum(n) + spare
    perm = rng.permutation(P).astype(np.int32)
    table, at = np.full((B, max(n) + extra), -1, np.int32), 0
    for r in range(B):
        table[r, :n[r]] = perm[at:at + n[r]]
        at += n[r]
    live = rng.integers(0, 1 << 32, P, dtype=np.uint64).astype(np.uint32)
    live[0] = 0xFFFFFFFF                         # the next tag wraps
    return dict(el=el, Hkv=Hkv, ps=ps, layers=layers, B=B, P=P, table=table, live=live, lens=np.array(lens, np.int32),
                expected=np.where(table >= 0, live[np.maximum(table, 0)], 0).astype(np.uint32), free=perm[at:],
                abort=np.zeros(B, np.uint8),
                pool=rng.integers(0, 256, (layers, P, Hkv, ps // TILE, 2 * TILE * D * el), dtype=np.uint8))


def put(c):
    d = {k: torch.from_numpy(c[k].view(np.int32) if c[k].dtype == np.uint32 else c[k]).to(DEV)
         for k in ("table", "live", "lens", "expected", "abort", "pool")}
    d["pool"] = d["pool"].reshape(-1)
    if c["el"] == 2:
        d["pool"] = d["pool"].view(torch.bfloat16)
    return d


def same(c, d, but=()):
    torch.cuda.synchronize()
    for k in ("table", "live", "lens", "expected", "abort"):
        assert np.array_equal(d[k].cpu().numpy().view(c[k].dtype), c[k]), k
    got = d["pool"].view(torch.uint8).cpu().numpy().reshape(c["pool"].shape)
    if len(but):
        got = got.copy()
        got[:, list(but)] = c["pool"][:, list(but)]
    assert np.array_equal(got, c["pool"]), "pool"


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def fork(c, d, parent, child, fresh, mask=True, stream=None):
    fpk_kv_fork(d["pool"], d["table"], d["expected"], d["lens"], d["live"], d["abort"] if mask else None, i32(parent),
                i32(child), i32(fresh), layers=c["layers"], Hkv=c["Hkv"], D=D, page_size=c["ps"], num_pages=c["P"],
                stream=stream)


def compact(c, d, src, dst, stream=None):
    fpk_kv_compact(d["pool"], d["table"], d["expected"], d["lens"], d["live"], i32(src), i32(dst), layers=c["layers"],
                   Hkv=c["Hkv"], D=D, page_size=c["ps"], num_pages=c["P"], stream=stream)


def plain_fork(c, parent, child, fresh):
    """Returns the fresh pages that a refused fork may have written."""
    loose = set()
    table, expected, lens, live, pool = (c[k].copy() for k in ("table", "expected", "lens", "live", "pool"))
    for p, ch, f in zip(parent, child, fresh):
        if not 0 <= ch < c["B"]:
            continue
        ok = 0 <= p < c["B"] and p != ch
        L = max(int(lens[p]), 0) if ok else 0
        n, rem = -(-L // c["ps"]), L % c["ps"]
        ok = ok and n <= table.shape[1] and (rem == 0 or 0 <= f < c["P"])
        if ok:
            row = table[p, :n]
            ok = bool(((row >= 0) & (row < c["P"])).all()) and np.array_equal(live[row], expected[p, :n])
        c["table"][ch], c["expected"][ch] = -1, 0
        c["lens"][ch] = L if ok else 0
        if not ok:
            c["abort"][ch] = 1
            if 0 <= f < c["P"]:
                loose.add(f)
            continue
        c["table"][ch, :n], c["expected"][ch, :n] = row, expected[p, :n]
        if rem:
            c["live"][f] = live[f] + np.uint32(1)
            c["table"][ch, n - 1], c["expected"][ch, n - 1] = f, c["live"][f]
            t = -(-rem // TILE)
            c["pool"][:, f, :, :t] = pool[:, row[-1], :, :t]
    return loose


def plain_compact(c, src, dst):
    ok = [(s, t) for s, t in zip(src, dst) if 0 <= s < c["P"] and 0 <= t < c["P"]]
    live, to = c["live"].copy(), dict(ok)
    for r in range(c["B"]):
        for j in range(min(-(-max(int(c["lens"][r]), 0) // c["ps"]), c["table"].shape[1])):
            p = int(c["table"][r, j])
            if p in to and live[p] == c["expected"][r, j]:
                c["table"][r, j], c["expected"][r, j] = to[p], live[to[p]] + np.uint32(1)
    for s, t in ok:
        c["live"][t] += np.uint32(1)
        c["pool"][:, t] = c["pool"][:, s]


SHAPE = pytest.mark.parametrize("el,Hkv,ps,layers", [(1, 2, 16, 1), (2, 2, 16, 3), (1, 8, 64, 2), (2, 1, 256, 2), (1, 3, 32, 5)])


@SHAPE
@pytest.mark.parametrize("rem", [0, 1, 15, 16, 17])
def test_fork(el, Hkv, ps, layers, rem):
    c = scene([2 * ps + rem, 0, 0, ps - 1, 0, 5], el=el, Hkv=Hkv, ps=ps, layers=layers, seed=rem)
    d = put(c)
    f = c["free"]
    args = [0, 0, 3], [1, 4, 2], [f[0], f[1], f[2]]
    fork(c, d, *args)
    assert not plain_fork(c, *args)
    same(c, d)
    assert not d["abort"].any()


def test_fork_edges():
    # an empty parent, a parent of one token, no fork at all, a full table
    c = scene([0, 1, 0, 64, 0, 0], extra=0, spare=9)
    d = put(c)
    args = [0, 1, 3], [2, 4, 5], [-1, c["free"][0], -1]
    fork(c, d, *args)
    fork(c, d, [], [], [])
    plain_fork(c, *args)
    same(c, d)


@pytest.mark.parametrize("mask", [True, False])
def test_fork_refuses(mask):
    c = scene([40, 40, 40, 40, 40, 0, 0, 0, 0, 0, 0, 7, 0], seed=3)
    c["expected"][1, 1] += 1                    # stale
    c["table"][2, 0] = c["P"]                   # out of range
    c["lens"][3] = 16 * c["table"].shape[1] + 1  # over-long
    d = put(c)
    f = c["free"]
    parent, child = [1, 2, 3, -1, 13, 4, 4, 11, 0, 4], [5, 6, 7, 8, 9, 10, 12, 11, 13, -1]
    fresh = [f[0], f[1], f[2], f[3], f[4], -1, c["P"], f[5], f[6], f[7]]
    fork(c, d, parent, child, fresh, mask=mask)
    loose = plain_fork(c, parent, child, fresh)
    if not mask:
        c["abort"][:] = 0
    same(c, d, but=loose)
    if mask:
        assert d["abort"].nonzero().view(-1).tolist() == [5, 6, 7, 8, 9, 10, 11, 12]


@SHAPE
def test_compact(el, Hkv, ps, layers):
    c = scene([5 * ps, 3 * ps + 1, 0, 7], el=el, Hkv=Hkv, ps=ps, layers=layers, seed=7)
    c["table"][2, :2], c["expected"][2, :2], c["lens"][2] = c["table"][0, :2], c["expected"][0, :2], 2 * ps
    c["expected"][0, 4] += 1                     # stale: stays
    c["table"][3, 1], c["expected"][3, 1] = c["table"][0, 2], c["expected"][0, 2]   # behind its context: stays
    d = put(c)
    src = np.sort(np.concatenate([c["table"][0, [0, 2, 4]], c["table"][1, [3]], c["table"][3, [0]]]))
    dst = c["free"][:5]
    compact(c, d, src, dst)
    plain_compact(c, src, dst)
    same(c, d)


def test_compact_edges():
    c = scene([40, 33], seed=1)
    d = put(c)
    compact(c, d, [], [])
    same(c, d)
    src = np.sort(np.array([-3, c["table"][0, 0], c["table"][1, 1], c["P"]]))
    dst = np.array([c["free"][0], c["free"][1], c["P"] + 4, c["free"][2]])
    compact(c, d, src, dst)
    plain_compact(c, src, dst)
    same(c, d)
    c["lens"][:] = [2 ** 31 - 1, -5]             # over-long and negative contexts stay within the table
    d["lens"].copy_(torch.from_numpy(c["lens"]))
    src, dst = [int(c["table"][0, 2])], [int(c["free"][4])]
    compact(c, d, src, dst)
    plain_compact(c, src, dst)
    same(c, d)


def test_many_moves():
    c = scene([16 * 300] * 3, layers=2, spare=900, seed=2)
    d = put(c)
    src, dst = np.sort(c["table"][:, :300].reshape(-1)[::2]), c["free"][:450]
    compact(c, d, src, dst)
    plain_compact(c, src, dst)
    same(c, d)


def test_pool_beyond_32_bits():
    # layers and pages whose byte offsets pass 2^32
    Hkv, ps, layers, P = 8, 64, 3, 20000
    page = 2 * Hkv * ps * D
    pool = torch.zeros(layers * P * page, dtype=torch.uint8, device=DEV)
    v = pool.view(layers, P, page)
    s, t = [19990, 19995], [19000, 5]
    for layer in range(layers):
        for k, p in enumerate(s):
            v[layer, p] = 10 * layer + k + 1
    table, lens = i32([[19990, 19995]]), i32([2 * ps])
    live = torch.zeros(P, dtype=torch.int32, device=DEV)
    exp = torch.zeros(1, 2, dtype=torch.int32, device=DEV)
    fpk_kv_compact(pool, table, exp, lens, live, i32(s), i32(t), layers=layers, Hkv=Hkv, D=D, page_size=ps, num_pages=P)
    torch.cuda.synchronize()
    for layer in range(layers):
        for k, p in enumerate(t):
            assert bool((v[layer, p] == 10 * layer + k + 1).all())
    assert table.tolist() == [t] and exp.tolist() == [[1, 1]]
    assert int(pool.count_nonzero()) == 4 * layers * page


def test_stream_and_graph():
    c = scene([40, 0, 100, 0], seed=4)
    d = put(c)
    side = torch.cuda.Stream(device=DEV)
    torch.cuda.synchronize()
    args = [0, 2], [1, 3], c["free"][:2]
    p, ch, f = i32(args[0]), i32(args[1]), i32(args[2])
    src, dst = i32(np.sort(c["table"][2, :2])), i32(c["free"][2:4])
    torch.cuda.synchronize()
    kw = dict(layers=1, Hkv=c["Hkv"], D=D, page_size=c["ps"], num_pages=c["P"])

    def both(stream=None):
        fpk_kv_fork(d["pool"], d["table"], d["expected"], d["lens"], d["live"], d["abort"], p, ch, f, stream=stream, **kw)
        fpk_kv_compact(d["pool"], d["table"], d["expected"], d["lens"], d["live"], src, dst, stream=stream, **kw)

    both(side)
    side.synchronize()
    first = {k: v.clone() for k, v in d.items()}
    plain_fork(c, *args)
    plain_compact(c, src.tolist(), dst.tolist())
    same(c, d)
    fresh = put(scene([40, 0, 100, 0], seed=4))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for k in d:
        d[k].copy_(fresh[k])
    g.replay()
    torch.cuda.synchronize()
    for k in d:
        assert torch.equal(d[k].view(torch.uint8), first[k].view(torch.uint8)), k
