"""Shared pages in the host ledger where rows and holders differ (CPU): stale entries,
pages given ahead of the context, and forks of requests that the device would refuse."""
import numpy as np
import pytest

from fp8_paged_kv_gb300.ledger import PageLedger
from test_ledger_fork import consistent, make


def counted(led):
    """Holders, free list and owners agree, whatever the rows say."""
    refs = np.zeros(led.num_pages, int)
    for held in led.held:
        refs[list(held)] += 1
    assert np.array_equal(refs, led.refs)
    assert sorted(led.free) == np.flatnonzero(refs == 0).tolist()
    assert np.array_equal(led.owner >= 0, refs > 0)
    for p in np.flatnonzero(refs):
        assert int(p) in led.held[led.owner[p]]


class Draws:
    """Answers of a generator, in turn."""

    def __init__(self, entry, chance, other=0):
        self.ints, self.chance = [entry, other], chance

    def integers(self, lo, hi):
        return self.ints.pop(0)

    def random(self):
        return self.chance


def test_release_counts_a_page_named_twice_once():
    led = make()
    led.admit(0, 32)
    led.fork(0, 1)
    p, q = led.page_table[0, :2].tolist()
    # request 1 holds both pages; request 0 is the owner, so that a stale entry may name the other one
    assert led.corrupt(1, Draws(1, 0.9)) == (1, "reallocated page")
    assert led.page_table[1, :2].tolist() == [p, p]
    assert led.release(1) == [] and led.refs[[p, q]].tolist() == [1, 1]
    consistent(led)
    assert led.release(0) == [p, q]
    consistent(led)


def test_release_frees_a_page_that_a_stale_entry_displaced():
    led = make()
    led.admit(0, 16)
    mine = led.admit(1, 48)
    led.corrupt(1, Draws(1, 0.9))
    assert led.release(1) == [mine[0], mine[2], mine[1]]   # the row's order, then what it no longer names
    counted(led)
    led.release(0)
    consistent(led)


def test_rows_that_name_a_page_twice_at_the_start():
    table = np.array([[3, 5, 3], [5, -1, -1]], np.int32)
    led = PageLedger(8, 3, 2, 16, np.zeros(8, np.uint32), table, np.array([48, 16], np.int32))
    counted(led)
    assert led.release(0) == [3]
    counted(led)
    assert led.release(1) == [5] and not led.refs.any()


@pytest.mark.parametrize("seed", range(4))
def test_churn_with_stale_entries(seed):
    led = make(num_pages=80)
    rng = np.random.default_rng(seed)
    for _ in range(300):
        r = int(rng.integers(0, led.B))
        live = [i for i in range(led.B) if led.lens[i]]
        if not led.lens[r]:
            if live and rng.random() < 0.6:
                src = int(rng.choice(live))
                try:
                    led.fork(src, r)
                except RuntimeError:
                    assert not led.held[r]   # a stale parent
            else:
                led.admit(r, int(rng.integers(1, 100)))
        elif rng.random() < 0.3:
            led.corrupt(r, rng)
        elif rng.random() < 0.5 and led.lens[r] < 120:
            led.grow(r)
        else:
            led.release(r)
        counted(led)
    for r in range(led.B):
        led.release(r)
    assert len(led.free) == led.num_pages


@pytest.mark.parametrize("L", [32, 40])
@pytest.mark.parametrize("what", ["tag", "page", "range", "gone", "long"])
def test_fork_refuses_what_the_device_refuses(L, what):
    # the last entry is the page in use (40 tokens), which the child would copy
    led = make()
    led.admit(0, L)
    led.admit(1, 64)
    last = led.pages_of(0) - 1
    if what == "tag":
        led.expected[0, last] -= np.uint32(1)
    elif what == "page":
        led.page_table[0, last] = led.page_table[1, 0]
        led.expected[0, last] = led.tags[led.page_table[1, 0]]
    elif what == "long":
        led.lens[0] = 8 * 16 + 1
    else:
        led.page_table[0, last] = led.num_pages if what == "range" else -1
    state = [x.copy() for x in (led.tags, led.refs, led.owner, led.page_table, led.expected, led.lens)]
    free, held = list(led.free), [set(h) for h in led.held]
    with pytest.raises(RuntimeError, match="request 0"):
        led.fork(0, 3)
    after = led.tags, led.refs, led.owner, led.page_table, led.expected, led.lens
    assert all(np.array_equal(x, y) for x, y in zip(state, after))
    assert free == list(led.free) and held == led.held


def test_fork_of_itself():
    led = make()
    with pytest.raises(RuntimeError, match="request 2"):
        led.fork(2, 2)


def compacted(led):
    """compact() with its promises checked: rows follow, what is ahead stays, the rest is in front."""
    table, tags = led.page_table.copy(), led.tags.copy()
    ahead = {int(p) for r in range(led.B) for p in table[r, led.pages_of(r):] if p >= 0}
    src, dst = led.compact()
    assert np.all(np.diff(src) > 0) and not set(src.tolist()) & set(dst.tolist())
    to = dict(zip(src.tolist(), dst.tolist()))
    assert not ahead & (set(to) | set(to.values()))
    assert np.array_equal(led.page_table, np.vectorize(lambda p: to.get(p, p))(table))
    assert np.array_equal(led.tags[dst], tags[dst] + np.uint32(1))
    used = [p for p in np.flatnonzero(led.refs).tolist() if p not in ahead]
    assert used == [p for p in range(led.num_pages) if p not in ahead][:len(used)]
    consistent(led)
    return src, dst


def test_compact_leaves_pages_ahead_of_the_context():
    led = make(num_pages=20)
    led.admit(0, 64)
    led.admit(1, 16)
    ahead = led.allocate(1, 2)
    led.release(0)
    src, _ = compacted(led)
    assert src.size == 1 and led.page_table[1, 1:3].tolist() == ahead
    for _ in range(32):
        assert led.grow(1) == []
    consistent(led)
    led.admit(2, 120)
    assert not set(led.page_table[2].tolist()) & set(ahead)
    consistent(led)
    src, _ = compacted(led)      # the context has reached them: now they move
    assert led.refs[:11].all()
    led.release(1)
    led.release(2)
    assert len(led.free) == 20


@pytest.mark.parametrize("seed", range(4))
def test_compact_with_pages_ahead_in_a_churn(seed):
    led = make(num_pages=70)
    rng = np.random.default_rng(seed)
    for step in range(120):
        r = int(rng.integers(0, led.B))
        if not led.held[r]:
            live = [i for i in range(led.B) if led.lens[i]]
            if live and rng.random() < 0.5:
                led.fork(int(rng.choice(live)), r)
            else:
                led.admit(r, int(rng.integers(0, 100)))
            led.allocate(r, int(rng.integers(0, 2)))
        elif rng.random() < 0.3:
            led.release(r)
        elif led.lens[r] < 120:
            led.grow(r)
        if step % 5 == 4:
            compacted(led)
        consistent(led)
