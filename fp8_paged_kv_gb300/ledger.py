"""Host-side page ledger: the server's record of pages, owners and expected tags.

The Cloudflare write-up ("Cosa ha cambiato Cloudflare per Kimi e GLM" and "La
sicurezza della cache KV condivisa diventa una questione di produzione",
remio.ai) has the serving system keep, for every request, the physical pages
it maps and the tag it expects on each; a page's tag changes whenever the
page is reallocated, so a mapping that outlived a reallocation no longer
matches.  The ledger is that bookkeeping for one layer's pool:

* a free list of physical pages and, per request, its page list;
* a mirror of the live tags (the device holds the real ones; every tag bump
  the ledger orders is applied on the device by ``fpk_page_tags_bump``);
* per request, the table row (page ids) and the expected tags.

Requests may share pages: ``fork`` makes one request hold another's full pages
(``fpk_kv_fork`` applies it on the device) and ``release`` frees a page when its
last holder leaves.  ``compact`` plans the moves that bring the pages in use to
the front of the pool (``fpk_kv_compact`` applies them); pages given ahead of a
context stay where they are.

Every allocation is a reallocation and bumps the page's tag; the pages
returned by ``allocate`` are the bump list for that step.  The ledger does no
GPU work itself and holds none of the kernels' arithmetic beyond the +1 it
must mirror to know the tag a fresh mapping should expect.
"""
from __future__ import annotations

from collections import deque

import numpy as np


class PageLedger:
    def __init__(self, num_pages: int, max_pages: int, B: int, page_size: int,
                 live_tags: np.ndarray, page_table: np.ndarray | None = None,
                 seq_lens: np.ndarray | None = None):
        self.num_pages = num_pages
        self.max_pages = max_pages
        self.B = B
        self.page_size = page_size
        self.tags = np.asarray(live_tags, np.uint32).copy()
        self.page_table = np.full((B, max_pages), -1, np.int32)
        self.expected = np.zeros((B, max_pages), np.uint32)
        self.lens = np.zeros(B, np.int32)
        self.owner = np.full(num_pages, -1, np.int64)      # one of a page's holders, -1: free
        self.held = [set() for _ in range(B)]               # pages each request holds
        self.refs = np.zeros(num_pages, np.int64)           # holders of each page
        if page_table is not None:
            self.page_table[:] = page_table
            m = page_table >= 0
            self.expected[m] = self.tags[page_table[m]]
            rows, _ = np.nonzero(m)
            self.owner[page_table[m]] = rows
            for r, p in zip(rows, page_table[m]):
                self.held[r].add(int(p))
            for pages in self.held:
                self.refs[list(pages)] += 1
            self.lens[:] = seq_lens
        self.free = deque(int(p) for p in np.flatnonzero(self.owner < 0))

    # ----------------------------------------------------------- allocation
    def pages_of(self, r: int) -> int:
        return -(-int(self.lens[r]) // self.page_size)

    def allocate(self, r: int, n: int) -> list[int]:
        """Give request r `n` more pages; each is reallocated (its tag bumped)."""
        have = self.pages_of_table(r)
        if have + n > self.max_pages:
            raise RuntimeError(f"request {r}: page table full")
        if n > len(self.free):
            raise RuntimeError("pool exhausted")
        got = [self.free.popleft() for _ in range(n)]
        for i, p in enumerate(got):
            self.tags[p] = self.tags[p] + np.uint32(1)
            self.owner[p] = r
            self.refs[p] = 1
            self.held[r].add(p)
            self.page_table[r, have + i] = p
            self.expected[r, have + i] = self.tags[p]
        return got

    def pages_of_table(self, r: int) -> int:
        row = self.page_table[r]
        return int(np.count_nonzero(row >= 0))

    def release(self, r: int) -> list[int]:
        """Request r finished (or was aborted): its pages return to the free list, but
        for those that another request still holds.  Returns the pages freed."""
        # each page held counts once, whatever the row says of it (a stale entry may name one
        # twice, or have taken the place of another): in the row's order, then those it lacks
        held = self.held[r]
        named = dict.fromkeys(int(p) for p in self.page_table[r] if int(p) in held)
        mine = [*named, *sorted(held - named.keys())]
        held.clear()
        pages = []
        for p in mine:
            self.refs[p] -= 1
            if self.refs[p] == 0:
                self.owner[p] = -1
                self.free.append(p)
                pages.append(p)
            elif self.owner[p] == r:
                self.owner[p] = next(i for i in range(self.B) if p in self.held[i])
        self.page_table[r] = -1
        self.expected[r] = 0
        self.lens[r] = 0
        return pages

    def admit(self, r: int, prompt_len: int) -> list[int]:
        """Slot r takes a new request with `prompt_len` tokens already computed."""
        assert self.pages_of_table(r) == 0, "slot still holds pages"
        self.lens[r] = prompt_len
        return self.allocate(r, -(-prompt_len // self.page_size))

    def grow(self, r: int) -> list[int]:
        """One decode token for request r; a page is reallocated when it crosses a boundary."""
        self.lens[r] += 1
        need = self.pages_of(r) - self.pages_of_table(r)
        return self.allocate(r, need) if need > 0 else []

    # -------------------------------------------------- sharing and moving
    def fork(self, parent: int, child: int) -> int:
        """Empty slot `child` takes over request `parent`: its full pages are shared,
        and where its last page is not full the child gets a page of its own, to
        which fpk_kv_fork copies it.  Returns that page (-1: none was needed).
        Raises, and changes nothing, where fpk_kv_fork would refuse: a fork refused
        on the device alone leaves the fresh page's tag behind the ledger's for good."""
        assert self.pages_of_table(child) == 0, "slot still holds pages"
        if parent == child:
            raise RuntimeError(f"request {parent}: forked to itself")
        L = int(self.lens[parent])
        full = L // self.page_size
        row = self.page_table[parent, :self.pages_of(parent)]
        if row.size < self.pages_of(parent) or not all(int(p) in self.held[parent] for p in row):
            raise RuntimeError(f"request {parent}: a page it maps is not its own")
        if not np.array_equal(self.expected[parent, :row.size], self.tags[row]):
            raise RuntimeError(f"request {parent}: it expects a tag that its page no longer has")
        if L % self.page_size and not self.free:
            raise RuntimeError("pool exhausted")
        row = row[:full]
        self.page_table[child, :full] = row
        self.expected[child, :full] = self.expected[parent, :full]
        self.held[child].update(int(p) for p in row)
        self.refs[row] += 1
        self.lens[child] = L
        return self.allocate(child, 1)[0] if L % self.page_size else -1

    def compact(self) -> tuple[np.ndarray, np.ndarray]:
        """Moves (src ascending, dst) after which the pages in use are the pool's
        first ones, but for pages given ahead of a request's context: these stay
        where they are (fpk_kv_compact rewrites the entries of contexts alone).
        Tables, tags and holders follow, as fpk_kv_compact leaves them on the
        device; stale entries stay."""
        at = self.page_table
        held = np.arange(self.max_pages) < -(-self.lens[:, None] // self.page_size)
        known = held & (at >= 0) & (at < self.num_pages)
        stays = np.zeros(self.num_pages, bool)
        for r, j in np.argwhere(~held & (at >= 0)):
            if int(at[r, j]) in self.held[r]:
                stays[at[r, j]] = True
        used = np.flatnonzero((self.refs > 0) & ~stays)
        front = np.flatnonzero(~stays)[:used.size]
        src = np.setdiff1d(used, front).astype(np.int32)
        dst = np.setdiff1d(front, used).astype(np.int32)
        to = np.arange(self.num_pages, dtype=np.int32)
        to[src] = dst
        safe = np.where(known, at, 0)
        moved = known & (to[safe] != safe) & (self.expected == self.tags[safe])
        self.tags[dst] += np.uint32(1)
        at[moved] = to[safe[moved]]
        self.expected[moved] = self.tags[at[moved]]
        self.refs[dst], self.owner[dst] = self.refs[src], self.owner[src]
        self.refs[src], self.owner[src] = 0, -1
        self.held = [{int(to[p]) for p in h} for h in self.held]
        taken = set(dst.tolist())
        self.free = deque([p for p in self.free if p not in taken] + src.tolist())
        return src, dst

    # ------------------------------------------------------ stale mappings
    def corrupt(self, r: int, rng: np.random.Generator) -> tuple[int, str]:
        """Make one of request r's checked entries stale, as a bookkeeping bug would:
        either the expected tag of its page lags one reallocation behind, or the
        entry points at a page that has been reallocated to another request and
        carries that page's previous tag.  Returns (entry, kind)."""
        P = self.pages_of(r)
        i = int(rng.integers(0, P))
        others = np.flatnonzero((self.owner >= 0) & (self.owner != r))
        if rng.random() < 0.5 or others.size == 0:
            self.expected[r, i] = self.expected[r, i] - np.uint32(1)
            return i, "lagging tag"
        p = int(others[rng.integers(0, others.size)])
        self.page_table[r, i] = p
        self.expected[r, i] = self.tags[p] - np.uint32(1)
        return i, "reallocated page"
