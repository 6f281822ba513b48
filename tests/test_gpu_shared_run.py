"""Forks, rotary writes, shared-prefix attention and a compaction together, as a
server samples several answers to one prompt: the ledger decides, the device
follows, and every step's attention equals the one over each request's own
table (fpk_paged_decode_attn_*), whose results the oracle tests pin."""
import numpy as np
import pytest
import torch

import oracle
from fp8_paged_kv_gb300.ledger import PageLedger
from fp8_paged_kv_gb300.pool import DecodePool, to_device
from fp8_paged_kv_gb300.rope import rope_inv_freq
from workloads import custom

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("ps", [16, 64])
def test_sampling_run(fp8, ps):
    lens = [600, 0, 0, 0, 333, 0, 0, 90]
    wl = custom(5, B=8, Hq=16, Hkv=2, ps=ps, prompt_lens=lens, steps=0, pool_factor=2.0, extra_pages=40,
                max_pages=-(-700 // ps))
    pool = DecodePool(wl, fp8=fp8, device=DEV)
    led = PageLedger(wl.num_pages, wl.page_table.shape[1], wl.B, ps, wl.live_tags,
                     np.where(np.arange(wl.page_table.shape[1]) < -(-wl.prompt_lens[:, None] // ps), wl.page_table, -1),
                     wl.prompt_lens)
    pool.page_table.copy_(to_device(led.page_table, DEV))
    pool.expected_tags.copy_(to_device(led.expected, DEV))
    pool.prefill()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    parent, child = [0, 0, 0, 4, 4], [1, 2, 3, 5, 6]
    fresh = [led.fork(p, c) for p, c in zip(parent, child)]
    pool.fork(i32(parent), i32(child), i32(fresh))
    torch.cuda.synchronize()

    def in_step():
        assert np.array_equal(pool.page_table.cpu().numpy(), led.page_table)
        assert np.array_equal(pool.expected_tags.cpu().numpy().view(np.uint32), led.expected)
        assert np.array_equal(pool.live_tags.cpu().numpy().view(np.uint32), led.tags)
        assert np.array_equal(pool.seq_lens.cpu().numpy(), led.lens)

    in_step()
    f, scale = rope_inv_freq(128, 10000.0, scaling="yarn", factor=4.0, original_len=512, device=DEV)
    starts, pre = i32([0, 4, 7]), i32([600, 333])
    rng = np.random.default_rng(1)
    for step in range(5):
        got = [p for r in range(wl.B) for p in led.grow(r)]
        if got:
            pool.bump(i32(got))
        pool.page_table.copy_(to_device(led.page_table, DEV))
        pool.expected_tags.copy_(to_device(led.expected, DEV))
        pool.seq_lens.copy_(i32(led.lens))
        for name, H in (("q", wl.Hq), ("k_new", wl.Hkv), ("v_new", wl.Hkv)):
            getattr(pool, name).copy_(torch.from_numpy(rng.standard_normal((wl.B, H, 128)).astype(np.float32)))
        pool.rope_append(f, rot_scale=scale)
        pool.validate()
        pool.attend_shared(starts, pre)
        torch.cuda.synchronize()
        assert not pool.abort_mask.any() and int(pool.abort_count) == 0
        out, lse = pool.out16.float().cpu().numpy(), pool.lse.cpu().numpy()
        pool.attend()
        torch.cuda.synchronize()
        ref, rl = pool.out.cpu().numpy(), pool.lse.cpu().numpy()
        # two kernels within the attention tests' bound of one reference, and a bf16 rounding
        assert (np.abs(out - ref) <= 4e-3 + (2e-2 + 2.0 ** -8) * np.abs(ref)).all()
        assert (np.abs(lse - rl) <= 2e-3 + 2.0 ** -15 * np.abs(rl)).all()
        host = pool.pool_bytes()
        o, l_ = oracle.paged_attention(pool.q.view(torch.int16).cpu().numpy().view(np.uint16), host, led.page_table,
                                       led.lens, fp8=fp8, k_scale=wl.k_scale, v_scale=wl.v_scale, sm_scale=wl.sm_scale,
                                       Hkv=wl.Hkv, page_size=ps, num_pages=wl.num_pages)
        assert (np.abs(out - o) <= 2e-3 + (1e-2 + 2.0 ** -8) * np.abs(o)).all()
        assert (np.abs(lse - l_) <= 1e-3 + 2.0 ** -16 * np.abs(l_)).all()
        if step == 1:
            led.release(0)                 # the prompt's first holder leaves, its pages stay
            pool.page_table.copy_(to_device(led.page_table, DEV))
            pool.expected_tags.copy_(to_device(led.expected, DEV))
            led.admit(0, 0)
            pool.seq_lens.copy_(i32(led.lens))
        if step == 2:
            src, dst = led.compact()
            assert len(src)
            pool.compact(i32(src), i32(dst))
            torch.cuda.synchronize()
            in_step()
    # a stale mapping in one fork: that request alone is aborted
    led.expected[2, 0] -= np.uint32(1)
    pool.expected_tags.copy_(to_device(led.expected, DEV))
    pool.validate()
    pool.attend_shared(starts, pre)
    torch.cuda.synchronize()
    assert pool.abort_mask.tolist() == [0, 0, 1, 0, 0, 0, 0, 0]
    out = pool.out16.float().cpu().numpy()
    live = np.arange(8) != 2
    assert not out[2].any() and (np.abs(out - o)[live] <= (2e-3 + (1e-2 + 2.0 ** -8) * np.abs(o))[live]).all()


@pytest.mark.parametrize("fp8", [True, False])
def test_first_shared_attention_on_another_stream(fp8):
    # its workspace is made, and zeroed, on the current stream, which is busy
    wl = custom(3, B=4, Hq=16, Hkv=2, ps=16, prompt_lens=[300, 310, 40, 7], steps=0)
    pool = DecodePool(wl, fp8=fp8, device=DEV)
    pool.prefill()
    pool.page_table[1, :10] = pool.page_table[0, :10]
    pool.q.copy_(torch.from_numpy(np.random.default_rng(2).standard_normal((4, 16, 128)).astype(np.float32)))
    starts, pre = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 2], [160]))
    busy = torch.zeros(1 << 27, device=DEV)
    side = torch.cuda.Stream(device=DEV)
    torch.cuda.synchronize()
    for _ in range(20):
        busy.add_(1.0)
    pool.attend_shared(starts, pre, use_mask=False, stream=side)
    torch.cuda.synchronize()
    first = pool.out16.clone(), pool.lse.clone()
    pool.attend_shared(starts, pre, use_mask=False)
    torch.cuda.synchronize()
    assert torch.equal(first[0], pool.out16) and torch.equal(first[1], pool.lse) and first[0].any()
