"""GPU parity of attention over caches with block scales, against 64 bits.

Bounds, from the arithmetic (A_s = sm sum |q| |k| of the row's largest token,
A_v = sum of weights times |V|):
* a score is a sum of 128 fp32 products: off by at most 128 2^-24 = 2^-17 of A_s;
  chunks: the query's two e4m3 parts leave out at most 2^-17 of its largest value,
  2^-17 sm max|q| sum |k| <= 2^-17 A_q with A_q that sum.  Scaling, shifts and the
  power of two add 4 2^-24 of |s| and 2^-22 of the weight.
* weights change by twice the scores' error d; sums of L terms by L 2^-24 at most;
  decode: a weight in two f16 parts loses 2^-22 of it.  |out - ref| <=
  (2 d + 2^-20 + L 2^-24) A_v.
* chunks: one f16 part loses 2^-11 of a weight, or 2^-25 of the largest weight times
  V's scale (its unit U) for small ones: 2^-11 A_v + 448 L 2^-25 U; bf16 results add
  2^-8 |ref|.
* lse: d + L 2^-24 + 2^-20, and 2^-23 of itself.
"""
import numpy as np
import pytest
import torch

from block_helpers import D, NAN, TILE, attend, bf16, context
from fp8_paged_kv_gb300 import (fpk_decode_status, fpk_decode_workspace_bytes, fpk_paged_decode_attn_fp8_block,
                                fpk_paged_prefill_attn_fp8_block, fpk_prefill_workspace_bytes)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SM = D ** -0.5


def scene(lens, counts, *, Hq, Hkv, ps, seed, spread=2, spare=3, qscale=1.0):
    """Contexts of lens[r] tokens in shuffled pages; stale slots and pages hold NaN codes and wild scales."""
    rng = np.random.default_rng(seed)
    tpp = ps // TILE
    maxp = max([1] + [-(-x // ps) for x in lens]) + 1
    P = sum(-(-x // ps) for x in lens if x > 0) + spare
    perm, at = rng.permutation(P), 0
    pool = np.full((P, Hkv, tpp, 2, TILE * D), NAN, np.uint8)
    scales = np.full((P, Hkv, tpp, 2), 255, np.uint8)
    table = np.full((len(lens), maxp), -1, np.int32)
    for r, L in enumerate(lens):
        for j in range(-(-L // ps)):
            page = perm[at]
            at += 1
            table[r, j] = page
            for t in range(min(tpp, -(-(L - j * ps) // TILE))):
                n = min(TILE, L - j * ps - t * TILE)
                codes = (rng.standard_normal((2, Hkv, n, D)) * 100).clip(-448, 448)
                codes = torch.from_numpy(codes).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
                pool[page, :, t, 0].reshape(Hkv, TILE, D)[:, :n] = codes[0]
                pool[page, :, t, 1].reshape(Hkv, D, TILE)[:, :, :n] = codes[1].transpose(0, 2, 1)
                scales[page, :, t] = 127 - 7 + rng.integers(-spread, spread + 1, (Hkv, 2))
    T = sum(counts)
    q = torch.from_numpy(rng.standard_normal((T, Hq, D)) * qscale).to(torch.bfloat16)
    return dict(lens=np.array(lens, np.int32), counts=counts, Hq=Hq, Hkv=Hkv, ps=ps, P=P, T=T, table=table, pool=pool,
                scales=scales, q=q, cu=np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))


def dev(x):
    return (torch.from_numpy(np.ascontiguousarray(x)) if isinstance(x, np.ndarray) else x).to(DEV)


def run(s, *, causal=None, mask=None, sm=SM, ws=None, splits=0, extra_rows=0):
    """causal None: decode."""
    T = s["T"] + extra_rows
    q = dev(torch.cat((s["q"], s["q"][:1].expand(extra_rows, -1, -1))) if extra_rows else s["q"])
    geo = dict(Hkv=s["Hkv"], page_size=s["ps"], num_pages=s["P"], sm_scale=sm)
    pool, scales, table, lens = dev(s["pool"]).reshape(-1), dev(s["scales"]), dev(s["table"]), dev(s["lens"])
    mask = None if mask is None else dev(np.array(mask, np.uint8))
    out = torch.full((T, s["Hq"], D), 7.0, dtype=torch.float32 if causal is None else torch.bfloat16, device=DEV)
    lse = torch.full((T, s["Hq"]), 7.0, device=DEV)
    B = len(s["counts"])
    if causal is None:
        if ws is None:
            ws = torch.zeros(fpk_decode_workspace_bytes(B, s["Hq"], s["Hkv"], D, splits), dtype=torch.uint8, device=DEV)
        fpk_paged_decode_attn_fp8_block(q, pool, scales, table, lens, mask, out, lse, ws, num_splits=splits, **geo)
    else:
        if ws is None:
            ws = torch.zeros(fpk_prefill_workspace_bytes(B, T, s["Hq"], s["Hkv"]), dtype=torch.uint8, device=DEV)
        fpk_paged_prefill_attn_fp8_block(q, dev(s["cu"]), pool, scales, table, lens, mask, out, lse, ws, causal=causal, **geo)
    torch.cuda.synchronize()
    assert fpk_decode_status(ws) == 0
    if extra_rows:
        assert torch.all(out[s["T"]:] == 7) and torch.all(lse[s["T"]:] == 7), "rows behind the last request were written"
    return bf16(out[:s["T"]]), bf16(lse[:s["T"]])


def check(s, got, *, causal=None, dead=(), sm=SM, rows=None):
    G = s["Hq"] // s["Hkv"]
    q = bf16(s["q"])
    worst = 0.0
    for r, n in enumerate(s["counts"]):
        L, a = int(s["lens"][r]), int(s["cu"][r])
        out, lse = got[0][a:a + n], got[1][a:a + n]
        if r in dead or L <= 0:
            assert np.all(out == 0) and np.all(np.isneginf(lse)), f"request {r}"
            continue
        take = np.arange(n) if rows is None or n <= rows else np.unique(np.linspace(0, n - 1, rows).astype(int))
        limit = np.repeat([L - n + i + 1 if causal else L for i in take], G)
        for h in range(s["Hkv"] if n else 0):
            k, v, ev = context(s["pool"], s["scales"], s["table"][r], L, h, s["ps"])
            qs = q[a + take, h * G:(h + 1) * G].reshape(-1, D)
            ref, ref_lse, size, sb, unit = attend(qs, k, v, ev, limit, sm)
            o, l_ = out[take, h * G:(h + 1) * G].reshape(-1, D), lse[take, h * G:(h + 1) * G].reshape(-1)
            none = limit <= 0
            assert np.all(o[none] == 0) and np.all(np.isneginf(l_[none])), f"request {r}, head {h}: rows that see nothing"
            d = 2.0 ** -17 * sb + 2.0 ** -20
            if causal is not None:
                d = d + 2.0 ** -17 * abs(sm) * np.abs(qs).max(1) * np.abs(k).sum(1).max()
            w = (2 * d + 2.0 ** -20 + L * 2.0 ** -24)[:, None] * size
            if causal is not None:
                w = w + 2.0 ** -11 * size + (448.0 * L * 2.0 ** -25 * unit)[:, None] + 2.0 ** -8 * np.abs(ref)
            err = np.abs(o - ref)
            assert np.all(err[~none] <= w[~none] + 1e-30), (
                f"request {r}, head {h}: {np.sum(err > w)} of {err.size}, worst {np.max((err / (w + 1e-30))[~none]):.2f} of the bound")
            el = np.abs(l_[~none] - ref_lse[~none])
            assert np.all(el <= (d + L * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * np.abs(np.where(none, 0, ref_lse)))[~none]), f"lse {el.max()}"
            worst = max(worst, float(np.max(err[~none] / (w[~none] + 1e-30), initial=0)))
    return worst


@pytest.mark.parametrize("Hq,Hkv,ps", [(64, 8, 16), (10, 2, 64), (7, 7, 48), (7, 1, 256), (32, 8, 32)])
@pytest.mark.parametrize("lens", [[1], [16, 17, 0, 300], [2049], [5, 1030, 77, 640, 31]])
def test_decode(Hq, Hkv, ps, lens):
    s = scene(lens, [1] * len(lens), Hq=Hq, Hkv=Hkv, ps=ps, seed=Hq + len(lens))
    check(s, run(s))


@pytest.mark.parametrize("splits", [1, 3, 40, 1000])
def test_decode_splits(splits):
    s = scene([700, 64, 1333], [1] * 3, Hq=16, Hkv=2, ps=16, seed=splits)
    check(s, run(s, splits=splits))


@pytest.mark.parametrize("spread", [0, 10, 40])
def test_decode_scales_far_apart(spread):
    """Weights meet V under its scale whatever the order of the blocks' magnitudes."""
    s = scene([400, 100], [1, 1], Hq=16, Hkv=2, ps=16, seed=spread, spread=0)
    rng = np.random.default_rng(spread)
    s["scales"][..., 1] = 127 + rng.integers(-spread - 7, spread - 7 + 1, s["scales"].shape[:-1]).clip(-50, 30)
    check(s, run(s))
    s["counts"], s["cu"] = [1, 1], np.array([0, 1, 2], np.int32)
    check(s, run(s, causal=True), causal=True)


def test_decode_dead_requests():
    s = scene([40, 40, 40, 40, 40], [1] * 5, Hq=8, Hkv=2, ps=16, seed=4)
    s["table"][1, 2], s["table"][3, 0] = s["P"], -1
    s["lens"][4] = 1 << 20
    check(s, run(s, mask=[0, 0, 1, 0, 0]), dead=(1, 2, 3, 4))


@pytest.mark.parametrize("spread", [0, 10, 40])
@pytest.mark.parametrize("causal", [True, False])
def test_chunks_scales_far_apart(spread, causal):
    s = scene([400, 100], [150, 40], Hq=16, Hkv=2, ps=16, seed=spread, spread=0)
    rng = np.random.default_rng(spread)
    s["scales"][..., 1] = 127 + rng.integers(-spread - 7, spread - 7 + 1, s["scales"].shape[:-1]).clip(-50, 30)
    check(s, run(s, causal=causal), causal=causal)


GEOMETRIES = [(64, 8, 16), (10, 2, 64), (7, 7, 48), (7, 1, 256), (32, 8, 32), (6, 1, 16)]


@pytest.mark.parametrize("Hq,Hkv,ps", GEOMETRIES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,counts", [([1], [1]), ([5], [5]), ([16, 17, 0, 300], [3, 17, 2, 40]),
                                         ([129, 130, 255, 700], [129, 2, 0, 65]), ([2049], [4])])
def test_chunks(Hq, Hkv, ps, causal, lens, counts):
    s = scene(lens, counts, Hq=Hq, Hkv=Hkv, ps=ps, seed=Hq + len(lens) + causal)
    check(s, run(s, causal=causal, extra_rows=3), causal=causal)


@pytest.mark.parametrize("Hq,Hkv", [(16, 2), (5, 1), (4, 4)])
def test_more_queries_than_tokens(Hq, Hkv):
    """Causal rows before the context's first token see nothing; cross attention sees a short context."""
    s = scene([10, 1, 140], [37, 300, 150], Hq=Hq, Hkv=Hkv, ps=16, seed=2)
    check(s, run(s, causal=True), causal=True)
    check(s, run(s, causal=False), causal=False)


@pytest.mark.parametrize("causal", [True, False])
def test_long_and_many(causal):
    """Units of many blocks cut between CTAs, whole units, and requests of one row."""
    s = scene([3000, 1, 4000, 517], [700, 1, 90, 517], Hq=16, Hkv=2, ps=32, seed=7)
    check(s, run(s, causal=causal), causal=causal, rows=9)
    s = scene([6000], [1], Hq=8, Hkv=1, ps=64, seed=8)
    check(s, run(s, causal=causal), causal=causal)
    lens = [1 + 37 * i % 211 for i in range(70)]
    s = scene(lens, [1 + i % 3 for i in range(70)], Hq=8, Hkv=2, ps=16, seed=9)
    check(s, run(s, causal=causal), causal=causal)


@pytest.mark.parametrize("causal", [True, False])
def test_chunks_of_dead_requests(causal):
    s = scene([40, 300, 40, 40, 40, 0], [3, 200, 2, 1, 2, 4], Hq=8, Hkv=2, ps=16, seed=4)
    s["table"][1, 18], s["table"][3, 0] = s["P"], -1
    s["lens"][4] = 1 << 20
    check(s, run(s, causal=causal, mask=[0, 0, 1, 0, 0, 0]), causal=causal, dead=(1, 2, 3, 4, 5))


@pytest.mark.parametrize("qscale,sm", [(40.0, SM), (2.0 ** -90, 1.0), (1.0, -0.3), (0.0, 1.0), (1.0, 0.0)])
def test_ranges_of_queries_and_scales(qscale, sm):
    s = scene([200, 33], [40, 9], Hq=8, Hkv=2, ps=16, seed=6, qscale=qscale)
    check(s, run(s, causal=True, sm=sm), causal=True, sm=sm)
    d = scene([200, 33], [1, 1], Hq=8, Hkv=2, ps=16, seed=6, qscale=qscale)
    check(d, run(d, sm=sm), sm=sm)


def test_calls_share_a_workspace_and_repeat_their_bits():
    shapes = [([3000, 1], [40, 1], 16, 2), ([64], [64], 8, 8), ([900] * 12, [7] * 12, 16, 2), ([3000, 1], [40, 1], 16, 2)]
    ws = torch.zeros(max(fpk_prefill_workspace_bytes(len(n), sum(n), hq, hk) for _, n, hq, hk in shapes), dtype=torch.uint8, device=DEV)
    first = None
    for lens, counts, Hq, Hkv in shapes:
        s = scene(lens, counts, Hq=Hq, Hkv=Hkv, ps=16, seed=5)
        got = run(s, causal=True, ws=ws)
        check(s, got, causal=True, rows=5)
        first = first or got
    assert np.array_equal(first[0], got[0]) and np.array_equal(first[1], got[1])


@pytest.mark.parametrize("Hq,Hkv", [(16, 2), (5, 5)])
@pytest.mark.parametrize("where", [50, 200, 391])
def test_nan_values_reach_only_rows_that_see_them(Hq, Hkv, where):
    """V of one token is NaN in three dims, K of another wholly: rows before them are as without, rows behind are NaN."""
    L, n, ps = 400, 390, 16
    s = scene([L], [n], Hq=Hq, Hkv=Hkv, ps=ps, seed=where)
    clean = run(s, causal=True)
    page, t, slot = s["table"][0, where // ps], where % ps // TILE, where % TILE
    dims = [0, 77, 127]
    s["pool"][page, 0, t, 1].reshape(D, TILE)[dims, slot] = NAN
    out, lse = run(s, causal=True)
    sees = np.arange(n) + L - n >= where  # query i is token L - n + i
    G = Hq // Hkv
    assert np.array_equal(out[~sees], clean[0][~sees]) and np.array_equal(lse, clean[1])
    assert np.array_equal(out[:, G:], clean[0][:, G:])
    bad = np.isnan(out[sees][:, :G])
    assert np.all(bad[..., dims]) and bad.sum() == bad[..., dims].size
    s["pool"][page, 0, t, 0].reshape(TILE, D)[slot, 3] = NAN | 0x80
    out, lse = run(s, causal=True)
    assert np.array_equal(out[~sees], clean[0][~sees]) and np.array_equal(lse[~sees], clean[1][~sees])
    assert np.all(np.isnan(out[sees][:, :G])) and np.all(np.isnan(lse[sees][:, :G])) and np.array_equal(lse[:, G:], clean[1][:, G:])
