"""GPU parity of shared-prefix decode attention with a plain one in 64 bits.

The reference reads every request's own table and knows nothing of groups.
Tolerance per output, from the roundings the kernel makes (each at most half a
step): |d| <= 2^-8 |ref| (the bf16 result) + (w + 2 ds + n 2^-24) A, where A is the
softmax-weighted mean of |v|, w the rounding of one softmax weight (f16 2^-11
over the e4m3 cache, bf16 2^-8 over the bf16 cache), ds the error of a score and
n 2^-24 an fp32 sum over n tokens; for lse |d| <= ds + n 2^-24 + 2^-20 |ref|.
ds: the e4m3 parts of the query leave out at most 2^-17 of the head's largest
|q| per value, and a sum of 128 products in fp32 errs by 2^-17 of the sum of
their magnitudes at most; both are taken with the largest |k| sums of the case.
"""
import numpy as np
import pytest
import torch

from fp8_paged_kv_gb300 import (FpkError, fpk_decode_status, fpk_paged_decode_attn_bf16_prefix,
                                fpk_paged_decode_attn_fp8_prefix, fpk_prefix_workspace_bytes)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D, TILE = 128, 16


def make(groups, *, fp8=True, Hkv=2, G=4, ps=16, lead=0, tail=0, sigma=1.0, seed=0, spare=3):
    """groups: [(prefix tokens, [context length of each request])]; `lead` requests
    before and `tail` requests behind the groups share nothing.  Unwritten slots and
    pages nobody holds are NaN codes."""
    rng = np.random.default_rng(seed)
    lens = [11 + 7 * i for i in range(lead)]
    starts, pre = [lead], []
    for p, ls in groups:
        lens += ls
        pre.append(p)
        starts.append(len(lens))
    lens += [5 + 40 * i for i in range(tail)]
    B = len(lens)
    maxp = max(1, max(-(-max(L, 0) // ps) for L in lens))
    rows, nid = [[] for _ in range(B)], 0
    for g, (p, ls) in enumerate(groups):
        share = min([p] + [L for L in ls if L > 0]) // ps if ls else 0
        ids = list(range(nid, nid + max(share, 0)))
        nid += len(ids)
        for r in range(starts[g], starts[g + 1]):
            if lens[r] > 0:
                rows[r] = list(ids)
    for r in range(B):
        more = -(-max(lens[r], 0) // ps) - len(rows[r])
        rows[r] += list(range(nid, nid + more))
        nid += more
    P = nid + spare
    perm = rng.permutation(P)
    table = np.full((B, maxp), -1, np.int32)
    for r in range(B):
        table[r, :len(rows[r])] = perm[rows[r]]
    g = torch.Generator().manual_seed(seed)
    tiles = torch.randn(P, Hkv, ps // TILE, 2, TILE * D, generator=g) * sigma
    scale = 0.03 * sigma
    if fp8:
        pool = (tiles / scale).to(torch.float8_e4m3fn).view(torch.uint8)
        nan = torch.tensor(0x7F, dtype=torch.uint8)
    else:
        pool, nan = tiles.to(torch.bfloat16), torch.tensor(float("nan"), dtype=torch.bfloat16)
    wrote = np.zeros((P, ps), bool)
    for r in range(B):
        for j, p in enumerate(table[r]):
            if p >= 0:
                wrote[p, :max(0, min(ps, lens[r] - j * ps))] = True
    gone = torch.from_numpy(~wrote).view(P, 1, ps // TILE, TILE)
    k, v = pool[..., 0, :].view(P, Hkv, -1, TILE, D), pool[..., 1, :].view(P, Hkv, -1, D, TILE)
    k.masked_fill_(gone[..., None], nan.item())
    v.masked_fill_(gone[..., None, :], nan.item())
    q = (torch.randn(B, Hkv * G, D, generator=g) * sigma).to(torch.bfloat16)
    return dict(fp8=fp8, Hkv=Hkv, G=G, ps=ps, P=P, B=B, pool=pool.reshape(-1), table=table, q=q,
                lens=np.array(lens, np.int32), starts=starts, pre=pre, ks=scale, vs=scale * 1.5, sm=D ** -0.5)


def reference(c, abort=None, table=None, lens=None):
    table, lens = c["table"] if table is None else table, c["lens"] if lens is None else lens
    B, Hkv, G, ps, P = c["B"], c["Hkv"], c["G"], c["ps"], c["P"]
    pool = c["pool"].view(P, Hkv, ps // TILE, 2, TILE * D)
    out = np.zeros((B, Hkv * G, D))
    lse = np.full((B, Hkv * G), -np.inf)
    A, ds = np.zeros((B, Hkv * G, D)), np.zeros((B, Hkv * G))
    for r in range(B):
        L = int(lens[r])
        n = -(-max(L, 0) // ps)
        if L <= 0 or n > table.shape[1] or (abort is not None and abort[r]):
            continue
        ids = table[r, :n]
        if (ids < 0).any() or (ids >= P).any():
            continue
        x = pool[torch.from_numpy(ids.astype(np.int64))]
        x = (x.view(torch.float8_e4m3fn).float() if c["fp8"] else x).double().numpy()
        k = x[:, :, :, 0].reshape(n, Hkv, -1, TILE, D).transpose(1, 0, 2, 3, 4).reshape(Hkv, -1, D)[:, :L]
        v = x[:, :, :, 1].reshape(n, Hkv, -1, D, TILE).transpose(1, 0, 2, 4, 3).reshape(Hkv, -1, D)[:, :L]
        if c["fp8"]:
            k, v = k * np.float32(c["ks"]).item(), v * np.float32(c["vs"]).item()
        q = c["q"][r].double().numpy().reshape(Hkv, G, D)
        s = np.einsum("hgd,hld->hgl", q, k) * c["sm"]
        m = s.max(-1, keepdims=True)
        p = np.exp(s - m)
        z = p.sum(-1, keepdims=True)
        out[r] = (np.einsum("hgl,hld->hgd", p, v) / z).reshape(-1, D)
        A[r] = (np.einsum("hgl,hld->hgd", p, np.abs(v)) / z).reshape(-1, D)
        lse[r] = (m + np.log(z)).reshape(-1)
        mag = np.abs(q).max(-1) * np.abs(k).sum(-1).max(-1)[:, None] * abs(c["sm"])
        ds[r] = (2 * 2.0 ** -17 * mag).reshape(-1)
    return out, lse, A, ds


def call(c, abort=None, table=None, lens=None, starts=None, pre=None, ws=None, stream=None, state=None):
    s = state if state is not None else {}
    if not s:
        t = lambda a: torch.as_tensor(np.asarray(a)).to(DEV)  # noqa: E731
        s.update(q=c["q"].to(DEV), pool=c["pool"].to(DEV), ks=torch.tensor([c["ks"]], dtype=torch.float32, device=DEV),
                 vs=torch.tensor([c["vs"]], dtype=torch.float32, device=DEV),
                 table=t(c["table"] if table is None else table), lens=t(c["lens"] if lens is None else lens),
                 starts=t(np.array(c["starts"] if starts is None else starts, np.int32)),
                 pre=t(np.array(c["pre"] if pre is None else pre, np.int32)),
                 abort=None if abort is None else t(np.array(abort, np.uint8)),
                 out=torch.full((c["B"], c["Hkv"] * c["G"], D), float("nan"), dtype=torch.bfloat16, device=DEV),
                 lse=torch.full((c["B"], c["Hkv"] * c["G"]), float("nan"), device=DEV))
        s["ws"] = ws if ws is not None else torch.zeros(fpk_prefix_workspace_bytes(c["B"], c["Hkv"] * c["G"], c["Hkv"]),
                                                        dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
    sc = (s["ks"], s["vs"]) if c["fp8"] else ()
    f = fpk_paged_decode_attn_fp8_prefix if c["fp8"] else fpk_paged_decode_attn_bf16_prefix
    f(s["q"], s["pool"], *sc, s["table"], s["lens"], s["abort"], s["starts"], s["pre"], s["out"], s["lse"], s["ws"],
      Hkv=c["Hkv"], page_size=c["ps"], num_pages=c["P"], sm_scale=c["sm"], stream=stream)
    return s


def check(c, s, ref, what=""):
    torch.cuda.synchronize()
    assert fpk_decode_status(s["ws"]) == 0, what
    out, lse = s["out"].double().cpu().numpy(), s["lse"].double().cpu().numpy()
    ro, rl, A, ds = ref
    dead = np.isneginf(rl)
    assert np.all(out[dead] == 0) and np.all(np.isneginf(lse[dead])), f"{what}: dead rows"
    n = max(1, int(c["lens"].max()))
    w = 2.0 ** -11 if c["fp8"] else 2.0 ** -8
    live = ~dead
    assert np.isfinite(out[live]).all() and np.isfinite(lse[live]).all(), what
    tol = 2.0 ** -8 * np.abs(ro) + (w + 2 * ds[..., None] + n * 2.0 ** -24) * A + 1e-12
    err = np.abs(out - ro)
    assert (err[live] <= tol[live]).all(), f"{what}: {(err / tol)[live].max():.2f} of the tolerance"
    ltol = ds + n * 2.0 ** -24 + 2.0 ** -20 * np.abs(np.where(dead, 0, rl))
    lerr = np.where(dead, 0, np.abs(lse - np.where(dead, lse, rl)))
    assert (lerr[live] <= ltol[live]).all(), f"{what}: lse {lerr.max():.2e}"


def run(c, **k):
    s = call(c, **k)
    check(c, s, reference(c, **{x: k[x] for x in ("abort", "table", "lens") if x in k}))
    return s


BOTH = pytest.mark.parametrize("fp8", [True, False])


@BOTH
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("ps", [16, 64, 256])
def test_sizes(fp8, G, ps):
    run(make([(300, [301, 300 + ps, 512, 777]), (2 * ps + 3, [3 * ps, 2 * ps + 4, 1000])], fp8=fp8, G=G, ps=ps,
             lead=1, tail=2, seed=G + ps))


@BOTH
@pytest.mark.parametrize("n", [2, 15, 16, 17, 31, 32, 33, 40, 64, 65])
def test_rows(fp8, n):
    # n requests x 8 heads: below, at and above one and two tiles of 128 rows
    run(make([(256, [257 + 3 * i for i in range(n)])], fp8=fp8, Hkv=1, G=8, seed=n))


@BOTH
@pytest.mark.parametrize("pre", [0, 1, 15, 16, 127, 128, 129, 143, 144, 1000, 2048])
def test_prefix_lengths(fp8, pre):
    run(make([(pre, [pre + 1, pre + 20, pre + 130, pre + 300])], fp8=fp8, G=8, seed=pre))


@BOTH
@pytest.mark.parametrize("Hkv,G", [(1, 1), (3, 8), (16, 4), (32, 1)])
def test_heads(fp8, Hkv, G):
    run(make([(200, [201, 240, 333]), (100, [101, 102])], fp8=fp8, Hkv=Hkv, G=G, seed=Hkv))


@BOTH
def test_single_tokens_and_empty(fp8):
    run(make([(1, [1, 1, 1]), (16, [16, 16, 0, 17]), (0, []), (64, [0, 0]), (50, [0, 64, 1])], fp8=fp8, lead=2, tail=3))
    run(make([(1, [1])], fp8=fp8, Hkv=1, G=1))
    run(make([(0, [0])], fp8=fp8))


@BOTH
def test_no_groups(fp8):
    run(make([], fp8=fp8, lead=3, tail=4))


@BOTH
def test_long_and_many_splits(fp8):
    run(make([(20000, [20001, 20500, 23000])], fp8=fp8, Hkv=1, G=8, ps=64, seed=5))


@BOTH
def test_many_groups_and_requests(fp8):
    rng = np.random.default_rng(9)
    groups = []
    for _ in range(40):
        p = int(rng.integers(0, 200))
        groups.append((p, [p + int(x) for x in rng.integers(0, 150, int(rng.integers(0, 9)))]))
    run(make(groups, fp8=fp8, Hkv=2, G=3, lead=5, tail=5, seed=11))


def test_large_batch():
    # more requests than the threads that plan the work
    run(make([(40, [41 + i % 60 for i in range(900)]), (20, [21 + i % 30 for i in range(700)])], Hkv=1, G=2, seed=4))


@BOTH
def test_prefix_longer_than_a_request(fp8):
    # what is shared is bounded by the shortest live request
    c = make([(400, [401, 60, 500, 450])], fp8=fp8)
    for r in (0, 2, 3):
        c["table"][r, :3] = c["table"][1, :3]
    run(c)


@BOTH
def test_claimed_prefix_beyond_whole_pages(fp8):
    c = make([(64, [90, 95, 99])], fp8=fp8, ps=32)
    run(c, pre=[75])
    run(c, pre=[-5])


@BOTH
def test_aborted_leader_and_members(fp8):
    c = make([(300, [310, 320, 400, 330]), (100, [101, 140])], fp8=fp8, tail=1)
    abort = np.array([1, 0, 1, 0, 0, 1, 0], np.uint8)
    table = c["table"].copy()
    table[0, :5] = -7                      # an aborted leader's row may say anything
    run(c, abort=abort, table=table)
    run(c, abort=np.ones(7, np.uint8))


@BOTH
def test_bad_pages(fp8):
    c = make([(200, [210, 300, 260]), (64, [100, 90])], fp8=fp8)
    for r, j, p in ((0, 2, -1), (1, 15, c["P"]), (2, 16, -9), (4, 5, 1 << 30), (3, 4, -2), (1, 12, -2)):
        table = c["table"].copy()
        table[r, j] = p
        ref = reference(c, table=table)
        if j < 12 and r < 3:               # the leader's shared page: nobody agrees with it
            for x in ref[0], ref[2]:
                x[:3] = 0
            ref[1][:3] = -np.inf
        check(c, call(c, table=table), ref, (r, j))


@BOTH
def test_disagreeing_table_fails_closed(fp8):
    c = make([(200, [210, 300, 260, 280])], fp8=fp8, spare=5)
    used = set(c["table"][c["table"] >= 0].tolist())
    table = c["table"].copy()
    table[2, 7] = next(p for p in range(c["P"]) if p not in used)
    ref = reference(c)
    ref[0][2] = 0
    ref[1][2] = -np.inf
    check(c, call(c, table=table), ref)


@BOTH
def test_over_long(fp8):
    c = make([(100, [120, 130, 140])], fp8=fp8)
    lens = c["lens"].copy()
    lens[1] = c["table"].shape[1] * 16 + 1
    run(c, lens=lens)
    lens[1] = 2 ** 31 - 1
    run(c, lens=lens)


@BOTH
def test_unruly_groups_stay_in_range(fp8):
    # starts outside [0, B] are clamped, one below an earlier one counts as that one
    c = make([(100, [120, 130, 140, 150])], fp8=fp8)
    run(c, starts=[-4, 900], pre=[64])
    run(c, starts=[0, 4, 2, 4], pre=[64, 64, 32])


@BOTH
@pytest.mark.parametrize("sigma", [0.0, 20.0])
def test_flat_and_peaked_scores(fp8, sigma):
    c = make([(500, [510, 600, 700])], fp8=fp8, seed=2)
    c["q"] = (c["q"].float() * sigma).to(torch.bfloat16)
    run(c)


@BOTH
def test_rising_scores(fp8):
    # every block of 128 tokens raises the maximum by far more than the last
    c = make([(2000, [2001, 2100])], fp8=fp8, Hkv=1, G=8, seed=3)
    x = c["pool"].view(c["P"], 1, 1, 2, TILE * D)
    step = np.zeros(c["P"], np.float32)
    for r in range(2):
        for j, p in enumerate(c["table"][r]):
            if p >= 0:
                step[p] = 1 + j // 8
    k = torch.from_numpy(step).view(-1, 1).expand(-1, TILE * D)
    if c["fp8"]:
        x[:, 0, 0, 0] = (k * 3.0).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        x[:, 0, 0, 0] = (k * 0.09).to(torch.bfloat16)
    c["q"] = torch.full_like(c["q"], 4.0)
    run(c)


@BOTH
def test_negative_and_zero_scale(fp8):
    c = make([(300, [310, 400, 333])], fp8=fp8)
    for sm in (-0.1, 0.0):
        c["sm"] = sm
        run(c)


def test_infinite_keys_bf16():
    # a key whose score is -inf has no weight; rows of nothing else are dead by formula
    c = make([(300, [310, 400, 333])], fp8=False)
    x = c["pool"].view(c["P"], 2, 1, 2, TILE * D)
    x[:, :, :, 0, :D] = -3e38            # token 0 of every page
    c["q"] = c["q"].abs().clamp(min=0.5)
    s = call(c)
    torch.cuda.synchronize()
    out = s["out"].float()
    assert torch.isfinite(out).all()


@BOTH
def test_bits_repeat_and_workspace_is_reused(fp8):
    big = make([(900, [910 + i for i in range(20)])], fp8=fp8, Hkv=2, G=8, seed=1)
    small = make([(30, [40, 50])], fp8=fp8, Hkv=2, G=8, seed=2)
    ws = torch.zeros(fpk_prefix_workspace_bytes(20, 16, 2), dtype=torch.uint8, device=DEV)
    a = call(big, ws=ws)
    torch.cuda.synchronize()
    first = a["out"].clone(), a["lse"].clone()
    run(small, ws=ws)
    call(big, state=a)
    torch.cuda.synchronize()
    assert torch.equal(first[0], a["out"]) and torch.equal(first[1], a["lse"])


@BOTH
def test_other_stream_and_graph(fp8):
    c = make([(500, [510, 600, 700, 501])], fp8=fp8, G=8, seed=6)
    s = call(c)
    torch.cuda.synchronize()
    want = s["out"].clone()
    side = torch.cuda.Stream(device=DEV)
    s["out"].fill_(float("nan"))
    torch.cuda.synchronize()
    call(c, state=s, stream=side)
    side.synchronize()
    assert torch.equal(want, s["out"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(c, state=s)
    # the graph follows what the buffers hold when it is replayed
    other = make([(500, [510, 600, 700, 501])], fp8=fp8, G=8, seed=7)
    for key in ("q", "pool"):
        s[key].copy_(other[key])
    s["table"].copy_(torch.from_numpy(other["table"]))
    s["pre"].fill_(333)
    g.replay()
    check(other, s, reference(other))
    g.replay()
    check(other, s, reference(other))


def test_workspace_too_small():
    c = make([(30, [40, 50])])
    with pytest.raises(FpkError, match="workspace"):
        call(c, ws=torch.zeros(128, dtype=torch.uint8, device=DEV))


@BOTH
def test_without_lse(fp8):
    c = make([(300, [310, 400, 333])], fp8=fp8)
    s = call(c)
    torch.cuda.synchronize()
    want = s["out"].clone()
    kept, s["lse"] = s["lse"], None
    s["out"].zero_()
    call(c, state=s)
    torch.cuda.synchronize()
    assert torch.equal(want, s["out"])
    s["lse"] = kept
