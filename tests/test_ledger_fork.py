"""Shared pages in the host ledger (CPU): forks count holders, a page is freed by
its last holder, compaction brings the pages in use to the front, and the tag
check accepts every mapping that the ledger made and none that it moved away."""
import numpy as np
import pytest

import oracle
from fp8_paged_kv_gb300.ledger import PageLedger


def make(num_pages=40, max_pages=8, B=6, ps=16, seed=0):
    tags = np.random.default_rng(seed).integers(0, 1 << 32, num_pages, dtype=np.uint64).astype(np.uint32)
    return PageLedger(num_pages, max_pages, B, ps, tags)


def aborts(led):
    return oracle.page_tags_validate(led.page_table, led.expected, led.lens, led.tags, led.num_pages,
                                     led.page_size)[0]


def consistent(led):
    refs = np.zeros(led.num_pages, int)
    for r in range(led.B):
        row = led.page_table[r]
        assert {int(p) for p in row[row >= 0]} == led.held[r]
        refs[list(led.held[r])] += 1
    assert np.array_equal(refs, led.refs)
    assert sorted(led.free) == np.flatnonzero(refs == 0).tolist()
    for p in np.flatnonzero(refs):
        assert int(p) in led.held[led.owner[p]]
    assert not aborts(led).any()


@pytest.mark.parametrize("L", [0, 1, 15, 16, 17, 64, 100])
def test_fork_shares_full_pages(L):
    led = make()
    led.admit(0, L)
    before = led.tags.copy()
    fresh = led.fork(0, 3)
    full = L // 16
    assert (fresh >= 0) == (L % 16 != 0)
    assert np.array_equal(led.page_table[3, :full], led.page_table[0, :full])
    if fresh >= 0:
        assert led.page_table[3, full] == fresh and fresh not in led.held[0]
        assert led.tags[fresh] == before[fresh] + np.uint32(1)
    assert led.lens[3] == L
    consistent(led)


def test_last_holder_frees():
    led = make()
    led.admit(0, 50)
    for c in (1, 2):
        led.fork(0, c)
    shared = set(led.page_table[0, :3].tolist())
    assert led.release(0) and not shared & set(led.free)     # only its own last page
    consistent(led)
    led.release(2)
    assert not shared & set(led.free)
    assert shared <= set(led.release(1)) and shared <= set(led.free)
    consistent(led)


def test_fork_refuses():
    led = make(num_pages=4)
    led.admit(0, 60)
    with pytest.raises(RuntimeError, match="exhausted"):
        led.fork(0, 1)
    assert led.refs.max() == 1 and led.pages_of_table(1) == 0
    led.page_table[0, 0] = -1
    with pytest.raises(RuntimeError, match="not its own"):
        led.fork(0, 1)


def test_compact_moves_to_the_front():
    led = make(num_pages=60)
    rng = np.random.default_rng(3)
    for step in range(60):
        r = int(rng.integers(0, led.B))
        if led.pages_of_table(r):
            if rng.random() < 0.4:
                led.release(r)
            elif led.lens[r] < 120 and led.free:
                led.grow(r)
        elif len(led.free) > 9:
            live = [i for i in range(led.B) if led.pages_of_table(i)]
            if live and rng.random() < 0.6:
                led.fork(int(rng.choice(live)), r)
            else:
                led.admit(r, int(rng.integers(1, 120)))
        if step % 7 == 6:
            table, tags = led.page_table.copy(), led.tags.copy()
            src, dst = led.compact()
            assert np.all(np.diff(src) > 0) and not set(src.tolist()) & set(dst.tolist())
            to = dict(zip(src.tolist(), dst.tolist()))
            assert np.array_equal(led.page_table, np.vectorize(lambda p: to.get(p, p))(table))
            assert np.array_equal(led.tags[dst], tags[dst] + np.uint32(1))
            used = np.flatnonzero(led.refs)
            assert np.array_equal(used, np.arange(used.size))
        consistent(led)


def test_compact_leaves_stale_entries():
    led = make()
    led.admit(0, 16)
    led.admit(1, 32)
    stale = int(led.page_table[1, 1])
    led.release(0)
    led.expected[1, 1] -= np.uint32(1)
    src, _ = led.compact()
    assert stale in src and led.page_table[1, 1] == stale
    assert aborts(led).tolist() == [0, 1, 0, 0, 0, 0]
