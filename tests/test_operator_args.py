"""Refusals of shared-prefix attention, rotary writes, forks and compactions (CPU):
bad sizes, missing and misaligned pointers return before any device call; the
binding refuses host tensors and shapes that do not belong together."""
import pytest
import torch

import fp8_paged_kv_gb300 as fpk

A = 1 << 20  # a 256-byte aligned address that is never followed
OK, EINVAL, EUNSUP = fpk.FPK_OK, fpk.FPK_EINVAL, fpk.FPK_EUNSUPPORTED

# every call below returns at a host-side check; where a device exists a
# regression in their order could launch on the addresses
host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="run where no device is visible")


@pytest.fixture(scope="module")
def lib():
    from fp8_paged_kv_gb300 import build
    build.build()
    return fpk.load_library()


@host_only
@pytest.mark.parametrize("fp8", [True, False])
def test_prefix(lib, fp8):
    def call(q=A, kv=A, ks=A, vs=A, pt=A, mp=4, lens=A, gs=A, pl=A, n=1, out=A, ws=A, wsb=1 << 40, B=2, Hq=16,
             Hkv=2, D=128, ps=16, pages=8):
        sc = (ks, vs) if fp8 else ()
        f = lib.fpk_paged_decode_attn_fp8_prefix if fp8 else lib.fpk_paged_decode_attn_bf16_prefix
        return f(q, kv, *sc, pt, mp, lens, None, gs, pl, n, out, None, ws, wsb, 0.1, B, Hq, Hkv, D, ps, pages, None)

    assert call(B=0, q=None, kv=None, out=None, ws=None, gs=None) == OK
    for bad in (dict(B=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=15), dict(n=-1), dict(n=3), dict(mp=-1), dict(pages=-1),
                dict(ps=0), dict(q=None), dict(kv=None), dict(pt=None), dict(lens=None), dict(out=None),
                dict(ws=None), dict(gs=None), dict(pl=None), dict(q=A + 2), dict(kv=A + 8), dict(out=A + 16),
                dict(ws=A + 128)) + ((dict(ks=None), dict(vs=None)) if fp8 else ()):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(D=64), dict(ps=24), dict(ps=272), dict(Hq=32)):
        assert call(**bad) == EUNSUP, bad


@host_only
def test_prefix_workspace(lib):
    for bad in ((2, 15, 2, 128), (2, 32, 2, 128), (-1, 16, 2, 128), (2, 16, 2, 64), (2, 0, 2, 128)):
        assert lib.fpk_prefix_workspace_bytes(*bad) == 0, bad


@host_only
@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("prefill", [True, False])
def test_rope(lib, fp8, prefill):
    def call(q=A, k=A, v=A, pos=A, n=5, f=A, qo=A, kv=A, ks=A, vs=A, pt=A, mp=4, rot=64, B=2, Hq=16, Hkv=2,
             D=128, ps=16, pages=8):
        sc = (ks, vs) if fp8 else ()
        tail = (None, None, None, rot, 0, 1.0, B, Hq, Hkv, D, ps, pages, None)
        name = f"fpk_rope_{'prefill' if prefill else 'append'}_{'fp8' if fp8 else 'bf16'}"
        if prefill:
            return getattr(lib, name)(q, k, v, pos, n, None, f, qo, kv, *sc, pt, mp, *tail)
        return getattr(lib, name)(q, k, v, f, qo, kv, *sc, pt, mp, pos, *tail)

    assert call(B=0, q=None, k=None, kv=None) == OK
    if prefill:
        assert call(n=0, k=None) == OK and call(n=-1) == EINVAL
    for bad in (dict(B=-1), dict(Hq=-1), dict(Hkv=0), dict(rot=0), dict(rot=-16), dict(mp=-1), dict(pages=-1),
                dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(pos=None), dict(f=None),
                dict(kv=None), dict(pt=None), dict(q=A + 8), dict(qo=A + 8), dict(k=A + 2), dict(v=A + 8),
                dict(kv=A + 8)) + ((dict(ks=None), dict(vs=None)) if fp8 else ()):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(D=64), dict(ps=24), dict(ps=272), dict(rot=8), dict(rot=144), dict(rot=72)):
        assert call(**bad) == EUNSUP, bad


@host_only
def test_moves(lib):
    def fork(kv=A, el=1, layers=2, stride=1 << 20, pt=A, mp=4, ex=A, lens=A, live=A, p=A, c=A, f=A, n=2, B=3,
             Hkv=2, D=128, ps=16, pages=8):
        return lib.fpk_kv_fork(kv, el, layers, stride, pt, mp, ex, lens, live, None, p, c, f, n, B, Hkv, D, ps,
                               pages, None)

    def compact(kv=A, el=1, layers=2, stride=1 << 20, pt=A, mp=4, ex=A, lens=A, live=A, s=A, d=A, n=2, B=3,
                Hkv=2, D=128, ps=16, pages=8):
        return lib.fpk_kv_compact(kv, el, layers, stride, pt, mp, ex, lens, live, s, d, n, B, Hkv, D, ps, pages,
                                  None)

    for call, own in ((fork, ("p", "c", "f")), (compact, ("s", "d"))):
        assert call(n=0, kv=None, pt=None) == OK and call(B=0, kv=None) == OK
        for name in ("kv", "pt", "ex", "lens", "live") + own:
            assert call(**{name: None}) == EINVAL, name
        # 2 layers of 8 pages of 8 KiB do not fit a stride below 64 KiB
        for bad in (dict(n=-1), dict(B=-1), dict(layers=-1), dict(stride=-16), dict(stride=(1 << 20) + 8),
                    dict(stride=65520), dict(kv=A + 8), dict(Hkv=0), dict(mp=-1), dict(pages=-1)):
            assert call(**bad) == EINVAL, bad
        for bad in (dict(D=64), dict(ps=24), dict(ps=272), dict(el=4), dict(el=0)):
            assert call(**bad) == EUNSUP, bad


def test_binding_refuses(lib):
    B, Hq, Hkv, D, ps, P = 2, 8, 2, 128, 16, 4
    z, i32, bf = torch.zeros, torch.int32, torch.bfloat16
    pool = z(2 * P * Hkv * ps * D, dtype=torch.uint8)
    kv, q, sc = z(B, Hkv, D, dtype=bf), z(B, Hq, D, dtype=bf), torch.ones(1)
    pt, ex, lens = z(B, 2, dtype=i32), z(B, 2, dtype=i32), torch.ones(B, dtype=i32)
    live, f, ws, lse = z(P, dtype=i32), z(32), z(4096, dtype=torch.uint8), z(B, Hq)
    cu, one = torch.tensor([0, 1, 2], dtype=i32), z(1, dtype=i32)
    geo = dict(Hkv=Hkv, page_size=ps, num_pages=P)

    def prefix(starts=torch.tensor([0, 2], dtype=i32), table=pt, out=None, pool_=pool):
        fpk.fpk_paged_decode_attn_fp8_prefix(q, pool_, sc, sc, table, lens, None, starts, one,
                                             q.clone() if out is None else out, lse, ws, sm_scale=0.1, **geo)

    def append(**k):
        a = dict(q=q, k=kv, v=kv, f=f, qo=q, pool=pool, pt=pt, lens=lens, rot=64) | k
        fpk.fpk_rope_append_fp8(a["q"], a["k"], a["v"], a["f"], a["qo"], a["pool"], sc, sc, a["pt"], a["lens"],
                                rot_dim=a["rot"], **geo)

    def prefill(start):
        fpk.fpk_rope_prefill_fp8(q, kv, kv, cu, start, f, q, pool, sc, sc, pt, rot_dim=64, **geo)

    def fork(child=one, layers=1, ex_=ex):
        fpk.fpk_kv_fork(pool, pt, ex_, lens, live, None, one, child, one, layers=layers, D=D, **geo)

    def compact(dst=one):
        fpk.fpk_kv_compact(pool, pt, ex, lens, live, one, dst, D=D, **geo)

    for call in (prefix, append, lambda: prefill(None), fork, compact):
        with pytest.raises(fpk.FpkError, match="CUDA"):
            call()
    bad = [lambda: prefix(starts=one), lambda: prefix(table=z(3, 2, dtype=i32)),
           lambda: prefix(out=z(B, Hq, 64, dtype=bf)), lambda: prefix(pool_=pool[16:]),
           lambda: append(k=z(B, 1, D, dtype=bf)), lambda: append(qo=z(B, 1, D, dtype=bf)),
           lambda: append(rot=128), lambda: append(lens=z(3, dtype=i32)),
           lambda: append(pt=z(3, 2, dtype=i32), lens=z(3, dtype=i32)), lambda: append(pool=pool[:-16]),
           lambda: prefill(one), lambda: fork(child=lens), lambda: fork(layers=2), lambda: fork(layers=0),
           lambda: fork(ex_=z(B, 1, dtype=i32)), lambda: compact(dst=lens)]
    for call in bad:
        with pytest.raises(fpk.FpkError, match="shape|elements|entries|rows"):
            call()
