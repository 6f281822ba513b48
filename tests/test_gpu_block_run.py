"""A server's day over one cache with block scales, through DecodePool and PageLedger: prompts
written and attended chunk by chunk, decode steps, drafted tokens checked in one pass, forks, a
compaction and a stale mapping.  Every attention is checked against 64 bits over the pool's own
bytes; the bytes, where nothing rotates, against the definition of the writes."""
import numpy as np
import pytest
import torch

from block_helpers import D, NAN, bf16, write_tokens
from fp8_paged_kv_gb300 import fpk_decode_status
from fp8_paged_kv_gb300.ledger import PageLedger
from fp8_paged_kv_gb300.pool import DecodePool, HostPipeline, admission_cap, to_device
from fp8_paged_kv_gb300.rope import rope_inv_freq
from test_gpu_block_attention import check
from workloads import custom

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Server:
    def __init__(self, *, B, Hq, Hkv, ps, room, prompt_tokens, rope, seed):
        self.wl = custom(seed, B=B, Hq=Hq, Hkv=Hkv, ps=ps, prompt_lens=[0] * B, steps=0, pool_factor=1.0,
                         extra_pages=B * -(-room // ps) + 5, max_pages=-(-room // ps))
        self.pool = DecodePool(self.wl, fp8=True, device=DEV, block_scales=True, prompt_tokens=prompt_tokens)
        self.led = PageLedger(self.wl.num_pages, self.wl.page_table.shape[1], B, ps, self.wl.live_tags)
        self.rope = rope
        self.freqs, self.rot_scale = rope_inv_freq(96, 10000.0, scaling="yarn", factor=4.0, original_len=512, device=DEV)
        self.rng = np.random.default_rng(seed)
        self.host = np.full((self.wl.num_pages, Hkv, ps // 16, 2, 16 * D), NAN, np.uint8)
        self.host_scales = np.zeros((self.wl.num_pages, Hkv, ps // 16, 2), np.uint8)

    def values(self, n, H):
        x = self.rng.standard_normal((n, H, D)) * 2.0 ** self.rng.uniform(-3, 3, (n, H, 1))
        return torch.from_numpy(x).to(torch.bfloat16).to(DEV)

    def rotation(self):
        return dict(rot_dim=96, rot_scale=self.rot_scale) if self.rope else dict(rot_dim=0)

    def upload(self):
        self.pool.page_table.copy_(to_device(self.led.page_table, DEV))
        self.pool.expected_tags.copy_(to_device(self.led.expected, DEV))
        self.pool.seq_lens.copy_(i32(self.led.lens))

    def grow(self, counts):
        got = [p for r, n in enumerate(counts) for _ in range(n) for p in self.led.grow(r)]
        if got:
            self.pool.bump(i32(got))
        self.upload()

    def wrote(self, r, first, k, v):
        if not self.rope:
            write_tokens(self.host, self.host_scales, self.led.page_table[r], first, bf16(k), bf16(v), self.wl.page_size)

    def scene(self, q, counts):
        """The pool as it is, for test_gpu_block_attention.check."""
        w, p = self.wl, self.pool
        return dict(lens=self.led.lens.copy(), counts=list(counts), Hq=w.Hq, Hkv=w.Hkv, ps=w.page_size, P=w.num_pages,
                    T=sum(counts), table=self.led.page_table, q=q.cpu(),
                    pool=p.kv_pool.cpu().numpy().reshape(self.host.shape),
                    scales=p.kv_scales.cpu().numpy().reshape(self.host_scales.shape),
                    cu=np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))

    def chunk(self, counts, stale=()):
        """counts[r] further tokens of each request, written and attended."""
        first = self.led.lens.copy()
        self.grow(counts)
        T, w = sum(counts), self.wl
        q, k, v = self.values(T, w.Hq), self.values(T, w.Hkv), self.values(T, w.Hkv)
        cu = np.concatenate([[0], np.cumsum(counts)])
        for r, n in enumerate(counts):
            if r not in stale:
                self.wrote(r, int(first[r]), k[cu[r]:cu[r + 1]], v[cu[r]:cu[r + 1]])
        out = torch.full((T, w.Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((T, w.Hq), 7.0, device=DEV)
        self.pool.rope_prefill(q, k, v, i32(cu), i32(first), self.freqs, **self.rotation())
        self.pool.validate()
        self.pool.attend_prompt(q, i32(cu), out, lse)
        torch.cuda.synchronize()
        assert self.pool.abort_mask.tolist() == [int(r in stale) for r in range(w.B)]
        check(self.scene(q, counts), (bf16(out), bf16(lse)), causal=True, dead=stale, rows=24)

    def step(self, live=None, stale=()):
        """One token more of each live request (the others' contexts are empty)."""
        counts = [int(x) for x in (live if live is not None else np.ones(self.wl.B, int))]
        self.grow(counts)
        w, p = self.wl, self.pool
        for name, H in (("q", w.Hq), ("k_new", w.Hkv), ("v_new", w.Hkv)):
            getattr(p, name).copy_(self.values(w.B, H))
        for r in range(w.B):
            if counts[r] and r not in stale:
                self.wrote(r, int(self.led.lens[r]) - 1, p.k_new[r:r + 1], p.v_new[r:r + 1])
        if self.rope:
            p.rope_append(self.freqs, rot_dim=96, rot_scale=self.rot_scale)
            p.validate()
            p.attend()
        else:
            p.step()
        torch.cuda.synchronize()
        assert p.abort_mask.tolist() == [int(r in stale) for r in range(w.B)]
        check(self.scene(p.q, [1] * w.B), (bf16(p.out), bf16(p.lse)), dead=stale)

    def check_bytes(self):
        """Of every live request: its tokens' codes and their blocks' scales."""
        if self.rope:
            return
        ps = self.wl.page_size
        pool = self.pool.kv_pool.cpu().numpy().reshape(self.host.shape)
        scales = self.pool.kv_scales.cpu().numpy().reshape(self.host_scales.shape)
        for r, L in enumerate(self.led.lens):
            for j in range(-(-int(L) // ps)):
                page = self.led.page_table[r, j]
                for t in range(min(ps // 16, -(-(int(L) - j * ps) // 16))):
                    n = min(16, int(L) - j * ps - t * 16)
                    assert np.array_equal(scales[page, :, t], self.host_scales[page, :, t])
                    a, b = pool[page, :, t], self.host[page, :, t]
                    assert np.array_equal(a[:, 0].reshape(-1, 16, D)[:, :n], b[:, 0].reshape(-1, 16, D)[:, :n])
                    assert np.array_equal(a[:, 1].reshape(-1, D, 16)[..., :n], b[:, 1].reshape(-1, D, 16)[..., :n])

    def in_step(self):
        assert np.array_equal(self.pool.page_table.cpu().numpy(), self.led.page_table)
        assert np.array_equal(self.pool.expected_tags.cpu().numpy().view(np.uint32), self.led.expected)
        assert np.array_equal(self.pool.live_tags.cpu().numpy().view(np.uint32), self.led.tags)
        assert np.array_equal(self.pool.seq_lens.cpu().numpy(), self.led.lens)


@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("Hq,Hkv,ps", [(16, 2, 16), (12, 4, 64)])
def test_serving_run(Hq, Hkv, ps, rope):
    s = Server(B=7, Hq=Hq, Hkv=Hkv, ps=ps, room=420, prompt_tokens=640, rope=rope, seed=ps + rope)
    s.chunk([300, 0, 0, 33, 0, 1, 150])          # prompts, whole or their first chunks
    s.chunk([45, 0, 0, 0, 0, 129, 7])            # .. and the rest
    parent, child = [0, 0, 3], [1, 2, 4]
    fresh = [s.led.fork(p, c) for p, c in zip(parent, child)]
    before = s.led.lens[parent] % ps
    s.pool.fork(i32(parent), i32(child), i32(fresh))
    torch.cuda.synchronize()
    s.in_step()
    for p, c, f, part in zip(parent, child, fresh, before):
        if f >= 0:     # the page in use: the host's copy follows
            last = s.led.page_table[p, s.led.pages_of(p) - 1]
            s.host[f], s.host_scales[f] = s.host[last], s.host_scales[last]
            assert part
    for _ in range(3):
        s.step()
    s.chunk([4, 3, 0, 1, 5, 4, 2])               # drafts, checked in one pass
    s.check_bytes()
    s.led.release(0)                             # the prompt's first holder leaves, its pages stay
    s.upload()
    s.step([0, 1, 1, 1, 1, 1, 1])
    src, dst = s.led.compact()
    assert len(src)
    s.pool.compact(i32(src), i32(dst))
    s.host[dst], s.host_scales[dst] = s.host[src], s.host_scales[src]
    torch.cuda.synchronize()
    s.in_step()
    s.step([0, 1, 1, 1, 1, 1, 1])
    s.chunk([40, 3, 0, 1, 0, 0, 2])
    s.check_bytes()
    s.led.expected[2, 0] -= np.uint32(1)         # a stale mapping: that request alone is dead
    s.step([1, 1, 1, 1, 1, 1, 1], stale=(2,))
    s.chunk([1, 2, 3, 0, 1, 0, 2], stale=(2,))
    assert fpk_decode_status(s.pool.workspace) == 0 and fpk_decode_status(s.pool.prompt_workspace) == 0


def test_prompts_of_a_workload_and_cross_attention():
    """DecodePool.prefill writes a workload's prompts; rows that see all of a context read them."""
    wl = custom(71, B=3, Hq=16, Hkv=2, ps=32, prompt_lens=[200, 0, 33], steps=1)
    pool = DecodePool(wl, fp8=True, device=DEV, block_scales=True, prompt_tokens=40)
    pool.prefill(chunk_tokens=128)
    shape = (wl.num_pages, 2, 2, 2, 16 * D)
    host, scales = np.full(shape, NAN, np.uint8), np.zeros(shape[:-1], np.uint8)
    f64 = lambda x: torch.from_numpy(x.view(np.int16)).view(torch.bfloat16).to(torch.float64).numpy()  # noqa: E731
    for r in range(3):
        a, b = wl.cu_prompt[r], wl.cu_prompt[r + 1]
        write_tokens(host, scales, wl.page_table[r], 0, f64(wl.k_prompt[a:b]), f64(wl.v_prompt[a:b]), 32)
    for r, L in enumerate([200, 0, 33]):
        for t in range(-(-L // 16)):
            assert np.array_equal(pool.kv_scales.cpu().numpy().reshape(scales.shape)[wl.page_table[r, t // 2], :, t % 2],
                                  scales[wl.page_table[r, t // 2], :, t % 2])
    counts = [17, 3, 20]
    q = torch.randn(40, 16, D, device=DEV).to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty(40, 16, device=DEV)
    pool.attend_prompt(q, i32([0, 17, 20, 40]), out, lse, causal=False, use_mask=False)
    torch.cuda.synchronize()
    s = dict(lens=wl.prompt_lens.astype(np.int32), counts=counts, Hq=16, Hkv=2, ps=32, P=wl.num_pages, T=40, table=wl.page_table,
             q=q.cpu(), cu=np.array([0, 17, 20, 40]), pool=pool.kv_pool.cpu().numpy().reshape(shape),
             scales=pool.kv_scales.cpu().numpy().reshape(scales.shape))
    check(s, (bf16(out), bf16(lse)), causal=False)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("validate", [True, False])
def test_pipelined_steps(graph, validate):
    """HostPipeline's steps are those of each step alone, bit for bit, eagerly and replayed."""
    n = 5
    wl = custom(132, B=5, Hq=16, Hkv=2, ps=16, prompt_lens=[40, 0, 300, 17, 1000], steps=n)
    wl.expected_tags[2, 3] ^= np.uint32(1)
    pool = DecodePool(wl, fp8=True, device=DEV, block_scales=True)
    pool.count_aborts = False
    pool.prefill()
    kept = pool.kv_pool.clone(), pool.kv_scales.clone()
    host_in, ref = [], []
    for t in range(n):
        pool.set_step(t)
        host_in.append(pool.io_in.cpu().pin_memory())
        pool.step(validate=validate)
        torch.cuda.synchronize()
        ref.append((pool.out.cpu().clone(), pool.lse.cpu().clone()))
    end = pool.kv_pool.clone(), pool.kv_scales.clone()
    host_out = [torch.zeros(pool.io_out.numel(), dtype=torch.uint8).pin_memory() for _ in range(n)]
    pipe = HostPipeline(pool, host_in, host_out, validate=validate)
    g = torch.cuda.CUDAGraph()
    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            pipe.run(n)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            pipe.run(n)
    pool.kv_pool.copy_(kept[0])
    pool.kv_scales.copy_(kept[1])
    g.replay() if graph else pipe.run(n)
    torch.cuda.synchronize()
    out_bytes = ref[0][0].numel() * 4
    lse_at = pool._io[0][3]["lse"].data_ptr() - pool._io[0][2].data_ptr()
    for t in range(n):
        assert torch.equal(host_out[t][:out_bytes].view(torch.int32), ref[t][0].view(torch.int32).view(-1)), f"step {t}"
        assert torch.equal(host_out[t][lse_at:lse_at + ref[t][1].numel() * 4].view(torch.int32), ref[t][1].view(torch.int32).view(-1))
    assert torch.equal(pool.kv_pool, end[0]) and torch.equal(pool.kv_scales, end[1])


def test_what_such_a_pool_refuses():
    wl = custom(72, B=2, Hq=8, Hkv=2, ps=16, prompt_lens=[20, 30], steps=1)
    for kw in (dict(fp8=False), dict(tensor_cores=True)):
        with pytest.raises(ValueError, match="block scales"):
            DecodePool(wl, device=DEV, block_scales=True, **kw)
    with pytest.raises(ValueError, match="attend_prompt"):
        DecodePool(wl, device=DEV, prompt_tokens=8)
    pool = DecodePool(wl, device=DEV, block_scales=True, prompt_tokens=4)
    with pytest.raises(ValueError, match="append_check"):
        pool.append_check()
    with pytest.raises(ValueError, match="attend_shared"):
        pool.attend_shared(i32([0, 2]), i32([16]))
    q = torch.zeros(5, 8, D, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="prompt_tokens=4"):
        pool.attend_prompt(q, i32([0, 2, 5]), q.clone(), None)


def test_admission():
    # a page's codes and its scales: 2 * 2 * 64 * 128 and 2 * 2 * 4 bytes
    assert admission_cap(10 * (32768 + 16), 100, Hkv=2, D=128, page_size=64, fp8=True, block_scales=True) == (10, 2, 5)
    assert admission_cap(10 * (32768 + 16) - 1, 100, Hkv=2, D=128, page_size=64, fp8=True, block_scales=True) == (9, 2, 4)
