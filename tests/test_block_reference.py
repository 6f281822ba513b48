"""The references of caches with block scales (CPU): codes against the oracle's
quantiser, the exponent rule by hand, and refusals of the calls."""
import numpy as np
import pytest
import torch

import fp8_paged_kv_gb300 as fpk
import oracle
from block_helpers import D, HIGH, LOW, NAN, TILE, VALUES, clamped, encode, exponent, write_tile

A = 1 << 20  # a 256-byte aligned address that is never followed
OK, EINVAL, EUNSUP, ENOSPC = fpk.FPK_OK, fpk.FPK_EINVAL, fpk.FPK_EUNSUPPORTED, fpk.FPK_ENOSPC
host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="run where no device is visible")


def test_codes_are_those_of_the_oracle():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(4000) * 10.0 ** rng.uniform(-4, 3, 4000), VALUES[:127], -VALUES[:127],
                        (VALUES[1:127] + VALUES[:126]) / 2, [0.0, -0.0, 449.0, 1e9, -1e9, np.inf, -np.inf, np.nan]])
    x = x.astype(np.float32)
    assert np.array_equal(encode(x.astype(np.float64)), oracle.e4m3_encode(x))


def test_exponent_rule():
    assert exponent(0.0) == LOW and exponent(448.0) == 0 and exponent(np.nextafter(448.0, 500)) == 1
    assert exponent(1.0) == -8 and exponent(1.75) == -8 and exponent(1.76) == -7  # 448 = 1.75 * 2^8
    assert exponent(1e30) == HIGH and exponent(1e-30) == LOW
    m, x = np.frexp(np.float64(3.3e5))
    assert exponent(3.3e5) == x - 9 + (m > 0.875)
    assert list(clamped(np.array([0, 255, 127, 77, 157], np.uint8))) == [LOW, HIGH, 0, LOW, HIGH]


def test_growth_keeps_normal_codes():
    """A block that grows by k binades holds the same values, but for codes below 2^-6."""
    pool, scales = np.full((1, 1, 1, 2, TILE * D), NAN, np.uint8), np.zeros((1, 1, 1, 2), np.uint8)
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, D))
    write_tile(pool, scales, 0, 0, 0, 0, x, 0)
    before, e0 = pool[0, 0, 0, 0, :3 * D].copy(), clamped(scales)[0, 0, 0, 0]
    write_tile(pool, scales, 0, 0, 0, 0, 8 * x[:1], 3)
    after, e1 = pool[0, 0, 0, 0, :3 * D], clamped(scales)[0, 0, 0, 0]
    assert e1 > e0
    was, now = VALUES[before] * 2.0 ** e0, VALUES[after] * 2.0 ** e1
    normal = np.abs(VALUES[after]) >= 2.0 ** -6
    assert np.array_equal(was[normal], now[normal]) and normal.mean() > 0.9
    assert np.all(np.abs(was - now) <= 2.0 ** (e1 - 10))
    assert np.all(pool[0, 0, 0, 0, 4 * D:] == NAN)


@pytest.fixture(scope="module")
def lib():
    from fp8_paged_kv_gb300 import build
    build.build()
    return fpk.load_library()


@host_only
@pytest.mark.parametrize("prefill", [True, False])
def test_rope_refusals(lib, prefill):
    def call(q=A, k=A, v=A, pos=A, n=5, f=A, qo=A, kv=A, sc=A, pt=A, mp=4, rot=64, B=2, Hq=16, Hkv=2, D=128, ps=16,
             pages=8):
        tail = (None, None, None, rot, 0, 1.0, B, Hq, Hkv, D, ps, pages, None)
        if prefill:
            return lib.fpk_rope_prefill_fp8_block(q, k, v, pos, n, None, f, qo, kv, sc, pt, mp, *tail)
        return lib.fpk_rope_append_fp8_block(q, k, v, f, qo, kv, sc, pt, mp, pos, *tail)

    assert call(B=0, n=0) == OK
    for bad in (dict(sc=None), dict(kv=None), dict(k=None), dict(v=None), dict(pos=None), dict(f=None), dict(q=None),
                dict(qo=None), dict(pt=None), dict(B=-1), dict(rot=-16), dict(Hkv=0), dict(Hq=-1), dict(ps=0),
                dict(mp=-1), dict(pages=-1), dict(k=A + 8), dict(q=A + 2), dict(kv=A + 1)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(D=64), dict(ps=24), dict(ps=272), dict(rot=8), dict(rot=144)):
        assert call(**bad) == EUNSUP, bad
    assert call(f=None, rot=0, sc=None) == EINVAL  # no frequencies are needed without a rotation: the scales are


@host_only
@pytest.mark.parametrize("prefill", [True, False])
def test_write_refusals(lib, prefill):
    def call(k=A, v=A, pos=A, n=5, kv=A, sc=A, pt=A, B=2, Hkv=2, D=128, ps=16):
        if prefill:
            return lib.fpk_kv_prefill_fp8_block(k, v, pos, n, None, kv, sc, pt, 4, None, None, None, B, Hkv, D, ps, 8, None)
        return lib.fpk_kv_append_fp8_block(k, v, kv, sc, pt, 4, pos, None, None, None, B, Hkv, D, ps, 8, None)

    for bad in (dict(sc=None), dict(kv=None), dict(k=None), dict(v=None), dict(pos=None), dict(pt=None), dict(B=-1),
                dict(Hkv=0), dict(v=A + 8)):
        assert call(**bad) == EINVAL, bad
    assert call(D=96) == EUNSUP and call(ps=20) == EUNSUP


@host_only
def test_decode_refusals(lib):
    def call(q=A, kv=A, sc=A, pt=A, mp=4, lens=A, out=A, ws=A, wsb=1 << 40, ns=0, B=2, Hq=16, Hkv=2, D=128, ps=16,
             pages=8):
        return lib.fpk_paged_decode_attn_fp8_block(q, kv, sc, pt, mp, lens, None, out, None, ws, wsb, ns, 0.1, B, Hq,
                                                   Hkv, D, ps, pages, None)

    assert call(B=0, q=None, kv=None, sc=None) == OK
    for bad in (dict(sc=None), dict(sc=A + 1), dict(kv=None), dict(q=None), dict(pt=None), dict(lens=None),
                dict(out=None), dict(ws=None), dict(B=-1), dict(Hq=15), dict(ns=-1), dict(q=A + 8), dict(ws=A + 16)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(D=64), dict(ps=24), dict(Hq=32)):
        assert call(**bad) == EUNSUP, bad


@host_only
def test_prefill_attention_refusals(lib):
    def call(q=A, cu=A, T=9, kv=A, sc=A, pt=A, mp=4, lens=A, out=A, ws=A, wsb=1 << 40, B=2, Hq=16, Hkv=2, D=128, ps=16,
             pages=8, causal=1):
        return lib.fpk_paged_prefill_attn_fp8_block(q, cu, T, kv, sc, pt, mp, lens, None, causal, out, None, ws, wsb, 0.1,
                                                    B, Hq, Hkv, D, ps, pages, None)

    assert call(B=0, q=None, out=None) == OK and call(T=0, q=None, out=None) == OK
    for bad in (dict(sc=None), dict(sc=A + 1), dict(cu=None), dict(kv=None), dict(q=None), dict(pt=None),
                dict(lens=None), dict(out=None), dict(ws=None), dict(B=-1), dict(T=-1), dict(Hq=15), dict(Hkv=0),
                dict(mp=-1), dict(pages=-1), dict(q=A + 8), dict(ws=A + 16), dict(out=A + 16), dict(kv=A + 8)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(D=64), dict(ps=24), dict(ps=272), dict(Hq=32)):
        assert call(**bad) == EUNSUP, bad
    for bad in ((2, 9, 15, 2, 128), (2, 9, 32, 2, 128), (-1, 9, 16, 2, 128), (2, -1, 16, 2, 128), (2, 9, 16, 2, 64)):
        assert lib.fpk_prefill_workspace_bytes(*bad) == 0, bad


@host_only
@pytest.mark.parametrize("fork", [True, False])
def test_move_refusals(lib, fork):
    def call(kv=A, layers=2, stride=1 << 20, sc=A, ss=1 << 10, pt=A, tags=A, lens=A, live=A, x=A, y=A, z=A, n=3, B=2,
             Hkv=2, D=128, ps=16, pages=8):
        if fork:
            return lib.fpk_kv_fork_block(kv, layers, stride, sc, ss, pt, 4, tags, lens, live, None, x, y, z, n, B, Hkv, D,
                                         ps, pages, None)
        return lib.fpk_kv_compact_block(kv, layers, stride, sc, ss, pt, 4, tags, lens, live, x, y, n, B, Hkv, D, ps, pages,
                                        None)

    assert call(n=0, sc=None) == OK
    # a layer's scales: 2 * 8 pages * 2 heads * 1 tile = 32 bytes
    for bad in (dict(sc=None), dict(sc=A + 1), dict(ss=31), dict(ss=30), dict(ss=-2), dict(kv=None), dict(x=None),
                dict(y=None), dict(live=None), dict(layers=-1), dict(stride=16)):
        assert call(**bad) == EINVAL, bad
    assert call(D=64) == EUNSUP


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    B, Hq, Hkv, ps, P, T = 2, 8, 2, 16, 4, 5
    pool, sc = torch.zeros(2 * P * Hkv * ps * D, dtype=torch.uint8), torch.zeros(P, Hkv, 1, 2, dtype=torch.uint8)
    kv, q = torch.zeros(B, Hkv, D, dtype=torch.bfloat16), torch.zeros(B, Hq, D, dtype=torch.bfloat16)
    pt, lens, tags = torch.zeros(B, 2, dtype=torch.int32), torch.ones(B, dtype=torch.int32), torch.zeros(P, dtype=torch.int32)
    cu, ws = torch.tensor([0, 2, T], dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    geo = dict(Hkv=Hkv, page_size=ps, num_pages=P)
    kt, qt = kv.repeat(3, 1, 1)[:T], q.repeat(3, 1, 1)[:T]
    calls = [
        lambda sc=sc: fpk.fpk_kv_append_fp8_block(kv, kv, pool, sc, pt, lens, D=D, **geo),
        lambda sc=sc: fpk.fpk_kv_prefill_fp8_block(kt, kt, cu, None, pool, sc, pt, D=D, **geo),
        lambda sc=sc: fpk.fpk_rope_append_fp8_block(None, kv, kv, None, None, pool, sc, pt, lens, rot_dim=0, **geo),
        lambda sc=sc: fpk.fpk_rope_prefill_fp8_block(qt, kt, kt, cu, None, None, qt, pool, sc, pt, rot_dim=0, **geo),
        lambda sc=sc: fpk.fpk_paged_decode_attn_fp8_block(q, pool, sc, pt, lens, None, q.float(), None, ws, sm_scale=0.1, **geo),
        lambda sc=sc: fpk.fpk_paged_prefill_attn_fp8_block(qt, cu, pool, sc, pt, lens, None, qt, None, ws, sm_scale=0.1, **geo),
        lambda sc=sc: fpk.fpk_kv_fork_block(pool, sc, pt, pt, lens, tags, None, lens, lens, lens, D=D, **geo),
        lambda sc=sc: fpk.fpk_kv_compact_block(pool, sc, pt, pt, lens, tags, lens, lens, D=D, **geo),
    ]
    for i, c in enumerate(calls):
        with pytest.raises(fpk.FpkError):
            c()
        with pytest.raises(fpk.FpkError, match="kv_scales"):
            c(sc[:2])
    assert fpk.block_scales(P, Hkv, 64, layers=3, device="cpu").shape == (3, P, Hkv, 4, 2)
