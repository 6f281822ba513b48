"""How calls on caches with block scales may be made: captured and replayed, two graphs over one
workspace, two streams at once, behind work of another stream, past 32-bit offsets, in batches of
any number of requests.  Results are those of the plain call, bit for bit (a call's work is cut by
its units alone), or meet the bounds of test_gpu_block_attention."""
import numpy as np
import pytest
import torch

from block_helpers import D, bf16
from fp8_paged_kv_gb300 import (FpkError, block_scales, fpk_decode_status, fpk_decode_workspace_bytes, fpk_kv_compact_block, fpk_kv_fork_block,
                                fpk_paged_decode_attn_fp8_block, fpk_paged_prefill_attn_fp8_block,
                                fpk_prefill_workspace_bytes, fpk_rope_append_fp8_block, fpk_rope_prefill_fp8_block)
from fp8_paged_kv_gb300.rope import rope_inv_freq
from test_gpu_block_attention import SM, check, dev, run, scene

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


class Calls:
    """A chunk's write and attention and a decode step's append and attention, over buffers of its own."""

    def __init__(self, seed, ws=None, counts=(5, 40, 1), lens=(300, 40, 17), Hq=16, Hkv=2, ps=32):
        g = torch.Generator(device=DEV).manual_seed(seed)
        B, T, maxp = len(counts), sum(counts), -(-(max(lens) + 4) // ps)
        P = B * maxp + 1
        r = lambda n, h: torch.randn(n, h, D, device=DEV, generator=g).to(torch.bfloat16)  # noqa: E731
        self.inputs = [r(T, Hq), r(T, Hkv), r(T, Hkv), r(B, Hq), r(B, Hkv), r(B, Hkv)]
        self.geo = dict(Hkv=Hkv, page_size=ps, num_pages=P)
        self.table = torch.randperm(P, device=DEV, generator=g)[:B * maxp].view(B, maxp).to(torch.int32)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        self.cu, self.start = i32(np.concatenate([[0], np.cumsum(counts)])), i32([n - c for n, c in zip(lens, counts)])
        self.lens, self.lens1 = i32(lens), i32([n + 1 for n in lens])
        self.pool = torch.randint(0, 120, (2 * P * Hkv * ps * D,), dtype=torch.uint8, device=DEV, generator=g)
        self.scales = block_scales(P, Hkv, ps, device=DEV).fill_(120)
        self.freqs, _ = rope_inv_freq(D, 10000.0, device=DEV)
        self.q_out, self.q1_out = torch.zeros_like(self.inputs[0]), torch.zeros_like(self.inputs[3])
        self.out, self.lse = torch.zeros_like(self.inputs[0]), torch.zeros(T, Hq, device=DEV)
        self.out1, self.lse1 = torch.zeros(B, Hq, D, device=DEV), torch.zeros(B, Hq, device=DEV)
        self.ws = ws if ws is not None else [torch.zeros(n, dtype=torch.uint8, device=DEV) for n in (
            fpk_prefill_workspace_bytes(B, T, Hq, Hkv), fpk_decode_workspace_bytes(B, Hq, Hkv, D, 0))]

    def __call__(self, stream=None):
        q, k, v, q1, k1, v1 = self.inputs
        rope = dict(rot_dim=D, stream=stream, **self.geo)
        fpk_rope_prefill_fp8_block(q, k, v, self.cu, self.start, self.freqs, self.q_out, self.pool, self.scales, self.table, **rope)
        fpk_paged_prefill_attn_fp8_block(self.q_out, self.cu, self.pool, self.scales, self.table, self.lens, None, self.out,
                                         self.lse, self.ws[0], sm_scale=SM, stream=stream, **self.geo)
        fpk_rope_append_fp8_block(q1, k1, v1, self.freqs, self.q1_out, self.pool, self.scales, self.table, self.lens1, **rope)
        fpk_paged_decode_attn_fp8_block(self.q1_out, self.pool, self.scales, self.table, self.lens1, None, self.out1,
                                        self.lse1, self.ws[1], sm_scale=SM, stream=stream, **self.geo)

    def results(self):
        return [x.clone() for x in (self.q_out, self.out, self.lse, self.q1_out, self.out1, self.lse1, self.pool, self.scales)]

    def state(self):
        return self.pool.clone(), self.scales.clone()

    def back(self, state):
        self.pool.copy_(state[0])
        self.scales.copy_(state[1])


def test_captured_and_replayed():
    a = Calls(1)
    start = a.state()
    a()
    want = a.results()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a()
    for _ in range(3):
        a.back(start)
        a.out.zero_(), a.out1.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert same(a.results(), want)
    for x in a.inputs:          # new values, fewer tokens: a replay reads them
        x.copy_(x.flip(0))
    a.cu.copy_(torch.tensor([0, 5, 30, 30], device=DEV))
    a.lens.copy_(torch.tensor([300, 40, 0], device=DEV))
    a.back(start)
    g.replay()
    torch.cuda.synchronize()
    got = a.results()
    a.back(start)
    a()
    torch.cuda.synchronize()
    assert same(a.results(), got) and not same(got, want)


def test_two_graphs_over_one_workspace():
    a = Calls(2, counts=(300, 7), lens=(2000, 700))
    b = Calls(3, ws=a.ws, counts=(1, 1, 90), lens=(1500, 30, 400))
    pairs = []
    for x in (a, b):
        start = x.state()
        x()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        pairs.append((x, start, x.results(), g))
        with torch.cuda.graph(g):
            x()
    for x, start, want, g in (pairs[0], pairs[1], pairs[1], pairs[0], pairs[1]):
        x.back(start)
        g.replay()
    for x, start, want, g in pairs:
        assert same(x.results(), want)


def test_two_streams_at_once():
    pairs = []
    for seed, counts, lens in ((4, (300, 7), (2000, 700)), (5, (1, 1, 90), (1500, 30, 400))):
        x = Calls(seed, counts=counts, lens=lens)
        start = x.state()
        x()
        torch.cuda.synchronize()
        pairs.append((x, start, x.results(), torch.cuda.Stream()))
        x.back(start)
    torch.cuda.synchronize()
    for _ in range(4):
        for x, start, _, stream in pairs:
            with torch.cuda.stream(stream):
                x.back(start)
                x()                     # the current stream
                x.back(start)
            x(stream=stream)            # .. and the same one by name
    torch.cuda.synchronize()
    for x, _, want, _ in pairs:
        assert same(x.results(), want)


def test_behind_another_stream():
    """The call waits for its stream's work alone, and for all of that."""
    x = Calls(6)
    start = x.state()
    x()
    torch.cuda.synchronize()
    want = x.results()
    good = [t.clone() for t in x.inputs]
    busy, side = torch.randn(4096, 4096, device=DEV), torch.cuda.Stream()
    for t in x.inputs:
        t.fill_(3.0)
    x.back(start)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            busy = busy @ busy * 1e-3
        for t, y in zip(x.inputs, good):
            t.copy_(y)
    x(stream=side)
    side.synchronize()
    assert same(x.results(), want)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv", [(16, 2), (10, 2), (5, 5)])
def test_batches_that_need_a_plan(Hq, Hkv, causal):
    """Empty requests, a wide table or rows behind the last request change how the work list is made, not the bits."""
    lens, counts = [700, 0, 33, 2000, 129], [300, 5, 33, 4, 1]
    s = scene(lens, counts, Hq=Hq, Hkv=Hkv, ps=16, seed=Hq)
    want = run(s, causal=causal)
    check(s, want, causal=causal, rows=9)
    more = dict(s, counts=counts + [0] * 40, lens=np.array(lens + [7] * 40, np.int32),
                table=np.concatenate([s["table"], np.repeat(s["table"][2:3], 40, 0)]),
                cu=np.concatenate([s["cu"], np.full(40, s["cu"][-1])]).astype(np.int32))
    wide = dict(s, table=np.pad(s["table"], ((0, 0), (0, 32768 // 5)), constant_values=-1))
    for t, extra in ((more, 0), (wide, 0), (s, 16384 // (Hq // Hkv))):
        got = run(t, causal=causal, extra_rows=extra)
        assert np.array_equal(got[0], want[0], equal_nan=True) and np.array_equal(got[1], want[1])


@pytest.mark.parametrize("causal", [True, False])
def test_more_requests_than_the_plan_keeps_near(causal):
    rng = np.random.default_rng(3)
    lens, counts = [int(x) for x in rng.integers(0, 60, 4300)], [int(x) for x in rng.integers(0, 3, 4300)]
    s = scene(lens, counts, Hq=2, Hkv=1, ps=16, seed=1)
    check(s, run(s, causal=causal), causal=causal)


@pytest.mark.parametrize("seed", range(8))
def test_random_batches(seed):
    rng = np.random.default_rng(100 + seed)
    B, (Hq, Hkv) = int(rng.integers(1, 45)), [(16, 2), (6, 2), (8, 8), (7, 1)][seed % 4]
    counts = [int(rng.choice([0, 1, 3, rng.integers(1, 200)])) for _ in range(B)]
    lens = [int(n + rng.choice([0, 5, rng.integers(0, 1500)])) for n in counts]
    s = scene(lens, counts, Hq=Hq, Hkv=Hkv, ps=[16, 64, 48][seed % 3], seed=seed)
    got = run(s, causal=True)
    check(s, got, causal=True, rows=5)
    for _ in range(5):
        again = run(s, causal=True)
        assert np.array_equal(again[0], got[0]) and np.array_equal(again[1], got[1])


@pytest.mark.parametrize("what", [np.nan, np.inf, -np.inf])
def test_queries_that_are_not_finite(what):
    """They make NaN of their own row, and of no other."""
    s = scene([400, 20], [150, 3], Hq=16, Hkv=2, ps=16, seed=12)
    clean = run(s, causal=True)
    for row, head, dim in ((0, 0, 0), (37, 9, 100), (149, 15, 127), (151, 3, 64)):
        s["q"][row, head, dim] = what
    out, lse = run(s, causal=True)
    hit = np.zeros(lse.shape, bool)
    for row, head in ((0, 0), (37, 9), (149, 15), (151, 3)):
        hit[row, head] = True
    assert np.isnan(out[hit]).all() and np.isnan(lse[hit]).all()
    assert np.array_equal(out[~hit], clean[0][~hit]) and np.array_equal(lse[~hit], clean[1][~hit])


def test_pages_past_32_bit_offsets():
    """The same calls in a small pool and at the end of one of 5.4 GB, with forks and moves between pages there."""
    a = Calls(7, counts=(70, 3), lens=(130, 60), Hq=16, Hkv=8, ps=64)
    P, far = a.geo["num_pages"], 41000
    one = 2 * 8 * 64 * D
    assert (far - P) * one > 1 << 32
    pool, scales = torch.empty(far * one, dtype=torch.uint8, device=DEV), block_scales(far, 8, 64, device=DEV)
    pool[-P * one:].copy_(a.pool)
    scales[0, -P:].copy_(a.scales[0])
    b = Calls(7, counts=(70, 3), lens=(130, 60), Hq=16, Hkv=8, ps=64)
    b.pool, b.scales, b.table = pool, scales, a.table + (far - P)
    b.geo["num_pages"] = far
    a(), b()
    torch.cuda.synchronize()
    assert same(b.results()[:6], a.results()[:6])
    assert torch.equal(pool[-P * one:], a.pool) and torch.equal(scales[0, -P:], a.scales[0])
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    spare = next(p for p in range(P) if p not in a.table.tolist()[0] + a.table.tolist()[1])
    for x, base in ((a, 0), (b, far - P)):
        tags = torch.zeros(x.geo["num_pages"], dtype=torch.int32, device=DEV)
        # a third, empty request takes over the first, its page in use copied to the spare page
        x.table = torch.cat((x.table, torch.full((1, x.table.shape[1]), -1, dtype=torch.int32, device=DEV)))
        x.tags = torch.zeros(x.table.shape, dtype=torch.int32, device=DEV)
        lens = torch.cat((x.lens1, i32([0])))
        fpk_kv_fork_block(x.pool, x.scales, x.table, x.tags, lens, tags, None, i32([0]), i32([2]), i32([base + spare]), D=D, **x.geo)
        assert lens.tolist()[2] == 131 and x.table[2, 2].item() == base + spare
    torch.cuda.synchronize()
    assert torch.equal(pool[-P * one:], a.pool) and torch.equal(scales[0, -P:], a.scales[0])
    # .. and that page moves to the front of the large pool
    fpk_kv_compact_block(pool, scales, b.table, b.tags, i32([131, 61, 131]), tags, i32([far - P + spare]), i32([1]), D=D, **b.geo)
    torch.cuda.synchronize()
    assert b.table[2, 2].item() == 1
    assert torch.equal(pool[one:2 * one], a.pool[spare * one:][:one]) and torch.equal(scales[0, 1], a.scales[0, spare])


def test_small_workspace_and_wrong_buffers_are_refused():
    s = scene([40], [3], Hq=8, Hkv=2, ps=16, seed=1)
    with pytest.raises(FpkError, match="status 3"):
        run(s, causal=True, ws=torch.zeros(fpk_prefill_workspace_bytes(1, 3, 8, 2) - 1, dtype=torch.uint8, device=DEV))
    q, pool, scales, table = dev(s["q"]), dev(s["pool"]).reshape(-1), dev(s["scales"]), dev(s["table"])
    ws = torch.zeros(fpk_prefill_workspace_bytes(1, 3, 8, 2) + 256, dtype=torch.uint8, device=DEV)
    good = dict(q=q, cu_seqlens=dev(s["cu"]), kv_pool=pool, kv_scales=scales, page_table=table, seq_lens=dev(s["lens"]),
                abort_mask=None, out=torch.empty_like(q), lse=None, workspace=ws)
    odd = torch.empty(q.numel() + 8, dtype=torch.bfloat16, device=DEV)[8:].view(q.shape)       # 16 bytes on
    for name, bad in (("out", odd), ("workspace", ws[16:]), ("q", torch.empty(q.numel() + 1, dtype=torch.bfloat16, device=DEV)[1:].view(q.shape)),
                      ("kv_scales", scales.reshape(-1)[:-1]), ("out", good["out"].float()), ("seq_lens", torch.zeros(2, dtype=torch.int32, device=DEV)),
                      ("kv_pool", pool.cpu()), ("abort_mask", torch.zeros(1, device=DEV)), ("lse", torch.zeros(3, 7, device=DEV))):
        with pytest.raises(FpkError):
            fpk_paged_prefill_attn_fp8_block(**dict(good, **{name: bad}), Hkv=2, page_size=16, num_pages=s["P"], sm_scale=SM)
    fpk_paged_prefill_attn_fp8_block(**good, Hkv=2, page_size=16, num_pages=s["P"], sm_scale=SM)
    torch.cuda.synchronize()
    check(s, (bf16(good["out"]), run(s, causal=True)[1]), causal=True)


@pytest.mark.parametrize("B", [5, 41])
def test_query_starts_that_decrease(B):
    """More rows than there are: the status word says so, and no row is written."""
    n = 256       # tokens, 8 units; every second request has them all
    s = scene([40], [1], Hq=64, Hkv=8, ps=16, seed=3)
    cu = np.tile(np.array([0, n], np.int32), B)[:B + 1]
    q, out = dev(s["q"]).expand(n, -1, -1).contiguous(), torch.full((n, 64, D), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(fpk_prefill_workspace_bytes(B, n, 64, 8), dtype=torch.uint8, device=DEV)
    table, lens = dev(s["table"]).expand(B, -1).contiguous(), dev(s["lens"]).expand(B).contiguous()
    fpk_paged_prefill_attn_fp8_block(q, dev(cu), dev(s["pool"]).reshape(-1), dev(s["scales"]), table, lens, None, out, None, ws,
                                     Hkv=8, page_size=16, num_pages=s["P"], sm_scale=SM)
    torch.cuda.synchronize()
    assert fpk_decode_status(ws) != 0 and torch.all(out == 7)
