"""GPU parity of writes into caches with block scales, against 64-bit references.

Without a rotation every product with 2^-e is exact, so codes and scales are bit
for bit those of the definition, and nothing else is written.  With one, a
rotated value is off by at most err = (2^-20 + 3 2^-24) times its pair's
magnitude (as for the caches with one scale): a block's exponent is that of the
largest exact value, or of one within err of it; a code's value lies within half
a step of e4m3 at that exponent (2^-4 relative, 2^-10 of the scale below the
normal codes) of a value within err of the exact one.
"""
import numpy as np
import pytest
import torch

from block_helpers import D, HIGH, LOW, NAN, TILE, VALUES, bf16, clamped, exponent, finite_top, write_tokens
from fp8_paged_kv_gb300 import (fpk_kv_append_fp8_block, fpk_kv_compact_block, fpk_kv_fork_block,
                                fpk_kv_prefill_fp8_block, fpk_rope_append_fp8_block, fpk_rope_prefill_fp8_block)
from fp8_paged_kv_gb300.rope import rope_inv_freq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def scene(counts, first, *, Hkv, ps, seed, spread=6.0, Hq=0):
    """Requests with counts[r] new tokens from first[r], in a pool of stale bytes; magnitudes over 2^+-spread."""
    rng = np.random.default_rng(seed)
    ends = [f + n for f, n in zip(first, counts)]
    maxp = max(1, max(-(-e // ps) for e in ends)) + 1
    need = [list(range(f // ps, -(-e // ps))) if n else [] for f, e, n in zip(first, ends, counts)]
    P = sum(map(len, need)) + 2
    perm, at = rng.permutation(P), 0
    table = np.full((len(counts), maxp), -1, np.int32)
    for r, js in enumerate(need):
        for j in js:
            table[r, j] = perm[at]
            at += 1
    tpp, T = ps // TILE, sum(counts)
    pool = rng.integers(0, 256, (P, Hkv, tpp, 2, TILE * D), dtype=np.uint8)
    scales = rng.integers(LOW + 127 - 3, HIGH + 127 + 4, (P, Hkv, tpp, 2)).astype(np.uint8)
    tags = rng.integers(0, 1 << 31, P).astype(np.int32)

    def values(h):
        x = rng.standard_normal((T, h, D)) * 2.0 ** rng.uniform(-spread, spread, (T, h, 1))
        return torch.from_numpy(x).to(torch.bfloat16)

    return dict(counts=counts, first=np.array(first, np.int32), Hkv=Hkv, Hq=Hq, ps=ps, P=P, T=T, table=table, pool=pool,
                scales=scales, live=tags, expected=np.where(table >= 0, tags[np.maximum(table, 0)], 0).astype(np.int32),
                cu=np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), k=values(Hkv), v=values(Hkv),
                q=values(Hq) if Hq else None)


def dev(x):
    return None if x is None else (torch.from_numpy(np.ascontiguousarray(x)) if isinstance(x, np.ndarray) else x).to(DEV)


def run(s, kind, *, tags=True, rope=None, seq_lens=None):
    """The call's pool, scales, abort mask and queries."""
    pool, scales, mask = dev(s["pool"]).reshape(-1), dev(s["scales"]), torch.zeros(len(s["counts"]), dtype=torch.uint8, device=DEV)
    guard = (dev(s["live"]), dev(s["expected"]), mask) if tags else (None, None, None)
    geo = dict(Hkv=s["Hkv"], page_size=s["ps"], num_pages=s["P"])
    lens = dev(s["first"] + np.array(s["counts"], np.int32)) if seq_lens is None else dev(seq_lens)
    k, v, table, q = dev(s["k"]), dev(s["v"]), dev(s["table"]), dev(s["q"])
    out = None if q is None else torch.full_like(q, 7.0)
    if rope is not None:
        freqs, more = rope
        if kind == "append":
            fpk_rope_append_fp8_block(q, k, v, freqs, out, pool, scales, table, lens, *guard, **more, **geo)
        else:
            fpk_rope_prefill_fp8_block(q, k, v, dev(s["cu"]), dev(s["first"]), freqs, out, pool, scales, table, *guard, **more, **geo)
    elif kind == "append":
        fpk_kv_append_fp8_block(k, v, pool, scales, table, lens, *guard, D=D, **geo)
    else:
        fpk_kv_prefill_fp8_block(k, v, dev(s["cu"]), dev(s["first"]), pool, scales, table, *guard, D=D, **geo)
    torch.cuda.synchronize()
    return pool.cpu().numpy().reshape(s["pool"].shape), scales.cpu().numpy(), mask.cpu().numpy(), out


def expected(s, skip=()):
    pool, scales, k, v = s["pool"].copy(), s["scales"].copy(), bf16(s["k"]), bf16(s["v"])
    for r, n in enumerate(s["counts"]):
        a = s["cu"][r]
        if n and r not in skip:
            write_tokens(pool, scales, s["table"][r], int(s["first"][r]), k[a:a + n], v[a:a + n], s["ps"])
    return pool, scales


def check(got, want, what=""):
    assert np.array_equal(got[1], want[1]), f"{what}: {np.sum(got[1] != want[1])} scales differ"
    assert np.array_equal(got[0], want[0]), f"{what}: {np.sum(got[0] != want[0])} codes differ"


@pytest.mark.parametrize("Hkv,ps", [(1, 16), (3, 64), (8, 16), (9, 256), (16, 48)])
@pytest.mark.parametrize("lens", [[1], [16, 17, 1, 0, 40], [3, 130, 15, 33]])
def test_prompts_from_the_start(Hkv, ps, lens):
    s = scene(lens, [0] * len(lens), Hkv=Hkv, ps=ps, seed=Hkv * 100 + len(lens))
    got = run(s, "prefill")
    check(got, expected(s))
    assert not got[2].any()


@pytest.mark.parametrize("Hkv,ps", [(1, 32), (5, 16), (8, 128)])
@pytest.mark.parametrize("spread", [0.0, 6.0, 60.0])
def test_chunks_behind_earlier_tokens(Hkv, ps, spread):
    counts, first = [1, 15, 2, 64, 7, 0, 33], [15, 1, 31, 5, 250, 9, 16 * 5 + 8]
    s = scene(counts, first, Hkv=Hkv, ps=ps, seed=int(spread) + Hkv, spread=spread)
    check(run(s, "prefill", tags=False), expected(s))


@pytest.mark.parametrize("Hkv,ps", [(1, 16), (8, 16), (3, 64), (8, 240)])
@pytest.mark.parametrize("spread", [0.0, 6.0])
def test_appends_at_every_slot(Hkv, ps, spread):
    first = list(range(0, 33)) + [ps - 1, ps, 3 * ps + 7]
    s = scene([1] * len(first), first, Hkv=Hkv, ps=ps, seed=Hkv + ps, spread=spread)
    got = run(s, "append")
    check(got, expected(s))
    assert not got[2].any()


@pytest.mark.parametrize("Hkv", [2, 8])
def test_tokens_one_by_one(Hkv):
    """A prompt appended token by token, and the same in chunks: the definition's bytes; a call repeated: the same."""
    n, ps = 37, 32
    s = scene([n], [0], Hkv=Hkv, ps=ps, seed=5)
    pool, scales = s["pool"].copy(), s["scales"].copy()
    one = dict(s, counts=[1], cu=np.array([0, 1], np.int32))
    for t in range(n):
        one.update(first=np.array([t], np.int32), k=s["k"][t:t + 1], v=s["v"][t:t + 1])
        write_tokens(pool, scales, s["table"][0], t, bf16(one["k"]), bf16(one["v"]), ps)
        for kind in ("append", "prefill", "append"):
            got = run(one, kind)
            check(got, (pool, scales), f"token {t}, {kind}")
        one.update(pool=got[0], scales=got[1])


def test_special_values():
    """Infinities saturate and count for nothing, NaN is 0x7F, zeros and tiny values get the least exponent."""
    n, Hkv, ps = 16, 6, 16
    s = scene([n], [0], Hkv=Hkv, ps=ps, seed=9)
    k, v = s["k"], s["v"]
    k[3, 0, 5], k[4, 0, 6], v[2, 0, 7], v[15, 0, 0] = np.inf, -np.inf, np.inf, np.nan
    k[:, 1], v[:, 1] = 0, -0.0
    k[:, 2], v[:, 2] = 2.0 ** -60, 2.0 ** -120
    k[:, 3], v[:, 3] = 1e30, -3e38
    k[:, 4], v[:, 4] = np.nan, np.inf
    k[0, 5, 0], v[0, 5, 0] = 448.0 * 2 ** 7, 449.0  # at a border, and behind it
    got = run(s, "prefill")
    check(got, expected(s))
    page = s["table"][0, 0]
    e = clamped(got[1])[page, :, 0]
    assert list(e[1]) == [LOW, LOW] and list(e[2]) == [LOW, LOW] and list(e[3]) == [HIGH, HIGH] and list(e[4]) == [LOW, LOW]
    assert np.all(got[0][page, 4, 0, 0] == NAN) and np.all(got[0][page, 4, 0, 1] == 0x7E)
    one = dict(s, counts=[1], first=np.array([4], np.int32), cu=np.array([0, 1], np.int32), k=k[4:5], v=v[4:5])
    check(run(one, "append"), expected(one))


def test_refused_pages():
    """A stale tag, a page outside the pool, a context behind the table: nothing of the request is written."""
    s = scene([5, 3, 4, 2, 6], [0, 13, 7, 3, 0], Hkv=3, ps=16, seed=11)
    s["expected"][0, 0] += 1
    s["table"][2, 0] = s["P"]
    s["table"][3, 0] = -1
    got = run(s, "prefill")
    assert list(got[2]) == [1, 0, 1, 1, 0]
    check(got, expected(s, skip=(0, 2, 3)))
    a = scene([1, 1, 1, 1], [4, 4, 4, 4], Hkv=3, ps=16, seed=12)
    a["expected"][0, 0] += 1
    a["table"][2, 0] = 1 << 30
    got = run(a, "append")
    assert list(got[2]) == [1, 0, 1, 0]
    check(got, expected(a, skip=(0, 2)))
    got = run(a, "append", seq_lens=np.array([0, 5, -3, 1 << 30], np.int32))
    assert list(got[2]) == [0, 0, 0, 1]
    check(got, expected(a, skip=(0, 2, 3)))


def rotated(x, pos, f, rot, inter, scale):
    y, mag = x.copy(), np.abs(x)
    a = pos.astype(np.float64)[:, None, None] * f.astype(np.float64)
    c, s = np.cos(a) * np.float64(np.float32(scale)), np.sin(a) * np.float64(np.float32(scale))
    i0, i1 = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    p, q = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = p * c - q * s, q * c + p * s
    mag[..., i0] = mag[..., i1] = (np.abs(p) + np.abs(q)) * abs(scale)
    return y, mag


@pytest.mark.parametrize("kind", ["append", "prefill"])
@pytest.mark.parametrize("rot,inter,Hq,Hkv,ps", [(128, False, 16, 2, 16), (64, True, 40, 8, 64), (96, False, 7, 7, 32), (16, True, 0, 9, 16)])
def test_rotated_keys(kind, rot, inter, Hq, Hkv, ps):
    counts, first = ([1] * 6, [0, 15, 16, 9, 131070, 77]) if kind == "append" else ([1, 40, 16, 3], [7, 0, 32, 99991])
    s = scene(counts, first, Hkv=Hkv, ps=ps, seed=rot + Hkv, Hq=Hq, spread=2.0)
    f, _ = rope_inv_freq(rot, 10000.0, device=DEV)
    got, scales, mask, out = run(s, kind, rope=(f, dict(rot_dim=rot, interleaved=inter, rot_scale=1.25)))
    assert not mask.any()
    pos = np.concatenate([np.arange(a, a + n) for a, n in zip(first, counts)])
    err = 2.0 ** -20 + 3 * 2.0 ** -24
    if Hq:
        y, mag = rotated(bf16(s["q"]), pos, f.cpu().numpy(), rot, inter, 1.25)
        assert np.all(np.abs(bf16(out) - y) <= err * mag + 2.0 ** -8 * np.abs(y) + 1e-30)
    y, mag = rotated(bf16(s["k"]), pos, f.cpu().numpy(), rot, inter, 1.25)
    # values, and everything that is no key: the definition's bytes, from keys that stand in for the rotated ones
    want = expected(s)
    assert np.array_equal(got[..., 1, :], want[0][..., 1, :]) and np.array_equal(scales[..., 1], want[1][..., 1])
    seen = np.zeros(got.shape[:4] + (TILE,), bool)
    for r, n in enumerate(counts):
        for a in range(first[r] // TILE, -(-(first[r] + n) // TILE)):
            p0, p1 = max(first[r], a * TILE), min(first[r] + n, a * TILE + TILE)
            page, tile, t0 = s["table"][r, p0 // ps], p0 % ps // TILE, p0 % TILE
            i = s["cu"][r] + p0 - first[r]
            for h in range(Hkv):
                x, e_of = y[i:i + p1 - p0, h], err * mag[i:i + p1 - p0, h]
                old = int(clamped(s["scales"])[page, h, tile, 0]) if t0 else LOW
                e = int(scales[page, h, tile, 0]) - 127
                lo, hi = (max(old, int(exponent(finite_top(np.abs(x) + d * e_of, None)))) for d in (-1, 1))
                assert lo <= e <= hi
                block = got[page, h, tile, 0].reshape(TILE, D)
                val = VALUES[block[t0:t0 + p1 - p0]] * 2.0 ** e
                assert np.all(np.abs(val - x) <= e_of + np.maximum(2.0 ** -4 * (np.abs(x) + e_of), 2.0 ** (e - 10)))
                before = s["pool"][page, h, tile, 0].reshape(TILE, D)
                moved = VALUES[before[:t0]] * 2.0 ** (old - e)
                was = VALUES[block[:t0]]
                assert np.array_equal(np.isnan(moved), np.isnan(was))
                assert np.all(np.nan_to_num(np.abs(was - moved)) <= 2.0 ** -10)
                assert np.array_equal(block[t0 + p1 - p0:], before[t0 + p1 - p0:])
                seen[page, h, tile, 0] = True
    alone = ~seen[..., 0, 0]
    assert np.array_equal(got[..., 0, :][alone], s["pool"][..., 0, :][alone])


def test_no_rotation_copies_queries():
    s = scene([3, 1], [0, 5], Hkv=2, ps=16, seed=3, Hq=8)
    got = run(s, "prefill", rope=(None, dict(rot_dim=0)))
    check(got, expected(s))
    assert torch.equal(got[3].cpu(), s["q"])


@pytest.mark.parametrize("layers", [1, 3])
def test_forks_and_moves_take_the_scales_along(layers):
    rng = np.random.default_rng(layers)
    Hkv, ps, P, tpp = 3, 48, 9, 3
    pool = torch.from_numpy(rng.integers(0, 256, layers * 2 * P * Hkv * ps * D, dtype=np.uint8)).to(DEV)
    scales = torch.from_numpy(rng.integers(0, 256, (layers, P, Hkv, tpp, 2), dtype=np.uint8)).to(DEV)
    live = torch.arange(100, 100 + P, dtype=torch.int32, device=DEV)
    table = torch.tensor([[4, 2, -1], [7, -1, -1], [-1, -1, -1]], dtype=torch.int32, device=DEV)
    tags = torch.where(table >= 0, live[table.clamp(min=0).long()], 0).to(torch.int32)
    lens = torch.tensor([ps + 17, 5, 0], dtype=torch.int32, device=DEV)
    mask = torch.zeros(3, dtype=torch.uint8, device=DEV)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    was = scales.clone()
    geo = dict(layers=layers, Hkv=Hkv, D=D, page_size=ps, num_pages=P)
    fpk_kv_fork_block(pool, scales, table, tags, lens, live, mask, i32(0), i32(2), i32(8), **geo)
    want = was.clone()
    want[:, 8, :, :2] = was[:, 2, :, :2]  # two tiles of the page in use hold tokens
    assert torch.equal(scales, want) and table[2].tolist() == [4, 8, -1] and not mask.any()
    x = pool.view(layers, P, Hkv, tpp, 2 * TILE * D)
    assert torch.equal(x[:, 8, :, :2], x[:, 2, :, :2])
    fpk_kv_compact_block(pool, scales, table, tags, lens, live, i32(7, 8), i32(0, 1), **geo)
    want[:, 0], want[:, 1] = want[:, 7], want[:, 8]
    assert torch.equal(scales, want) and table.tolist() == [[4, 2, -1], [0, -1, -1], [4, 1, -1]]
    assert torch.equal(x[:, 1], x[:, 8]) and torch.equal(tags[2], torch.tensor([104, 102, 0], dtype=torch.int32, device=DEV))
