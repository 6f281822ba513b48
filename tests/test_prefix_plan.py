"""CPU model of the shared-prefix attention's work list: every block of every unit
belongs to exactly one CTA, a CTA finds its first unit from the planner's request,
at most one of its pieces continues a unit, and the merge of a row visits exactly
the partials that the pieces wrote."""
import random

import pytest

PAIR, SOLO, START_PAIR, START_SOLO, ROWS, BLK = 6, 2, 12, 5, 256, 8


def prefix_shape(ptiles, gcount, G):
    rows = gcount * G
    blocks, units = -(-ptiles // BLK), -(-rows // ROWS)
    wlast = PAIR if rows - (units - 1) * ROWS > 128 else SOLO
    step = START_PAIR + PAIR * blocks
    return blocks, units, wlast, step, step * (units - 1) + start_cost(wlast) + wlast * blocks


def start_cost(w):
    return START_PAIR if w == PAIR else START_SOLO


def own_cost(stok):
    return START_SOLO + SOLO * own_blocks(stok) if stok > 0 else 0


def own_blocks(stok):
    return -(-stok // 128)


def owned(y, n, w, b0, b1):
    lo = 0 if b0 <= y else (b0 - y + w - 1) // w
    hi = 0 if b1 <= y else (b1 - y + w - 1) // w
    return min(lo, n), min(hi, n)


def begin(c, T, n):
    return c * (T // n) + min(c, T % n)


def owner(y, T, n):
    share, more = divmod(T, n)
    return y // (share + 1) if y < more * (share + 1) else more + (y - more * (share + 1)) // share


def plan(groups, G, Hkv, ctas):
    """groups: [(ptiles, [own tokens])]; requests as (y0, ptiles, stok, gfirst, gcount)."""
    reqs, y = [], 0
    for ptiles, own in groups:
        first = len(reqs)
        for i, stok in enumerate(own):
            cost = own_cost(stok)
            if ptiles and i == 0:
                cost += prefix_shape(ptiles, len(own), G)[4]
            reqs.append((y, ptiles, stok, first, len(own)))
            y += cost * Hkv
    T = y
    # the last request whose units start at or before the range
    start = [max(r for r, q in enumerate(reqs) if q[0] <= begin(c, T, ctas)) for c in range(ctas)]
    return reqs, T, start


def pieces(reqs, T, start, G, Hkv, ctas, c):
    b0, b1 = begin(c, T, ctas), begin(c + 1, T, ctas)
    if b0 >= b1:
        return
    r = start[c]

    def enter(r):
        y0, ptiles, _, gfirst, _ = reqs[r]
        return 0, (0 if ptiles and gfirst == r else -1), y0

    h, u, y = enter(r)
    at = b0 - y
    assert at >= 0
    skip_own = True
    if u == 0:
        blocks, units, wlast, step, head = prefix_shape(reqs[r][1], reqs[r][4], G)
        if at < head * Hkv:
            h = at // head
            u = min(at % head // step, units - 1)
            y += h * head + u * step
            skip_own = False
        else:
            u, y, at = -1, y + head * Hkv, at - head * Hkv
    if skip_own:
        cost = own_cost(reqs[r][2])
        if cost:
            h = min(at // cost, Hkv)
            y += h * cost
    while y < b1:
        y0, ptiles, stok, gfirst, gcount = reqs[r]
        if u >= 0:
            blocks, units, wlast, step, head = prefix_shape(ptiles, gcount, G)
            w = wlast if u == units - 1 else PAIR
            i0, i1 = owned(y + start_cost(w), blocks, w, b0, b1)
            unit = ("prefix", gfirst, h, u)
            pair = min(ROWS, gcount * G - u * ROWS) > 128
            assert pair == (w == PAIR)
            y += start_cost(w) + blocks * w
            u += 1
            if u == units:
                u, h = 0, h + 1
                if h == Hkv:
                    h, u = 0, -1
        else:
            n = own_blocks(stok)
            if n == 0 or h >= Hkv:
                r += 1
                if r >= len(reqs):
                    return
                h, u, y = enter(r)
                continue
            i0, i1 = owned(y + START_SOLO, n, SOLO, b0, b1)
            unit, pair = ("own", r, h, 0), False
            y += own_cost(stok)
            h += 1
        if i0 < i1:
            yield unit, i0, i1, pair


def merge(reqs, T, G, Hkv, ctas, r, h, g):
    """(unit, start slot or CTA slot, sub) of the partials that row (r, h, g) reads."""
    y0, ptiles, stok, gfirst, gcount = reqs[r]
    own = y0

    def unit(y, n, w, name, subs):
        for c in range(owner(y, T, ctas), owner(y + (n - 1) * w, T, ctas) + 1):
            i0, i1 = owned(y, n, w, begin(c, T, ctas), begin(c + 1, T, ctas))
            for sub in range(subs):
                if i0 < i1:
                    yield name, ("start" if i0 == 0 else c), sub

    if ptiles:
        blocks, units, wlast, step, head = prefix_shape(ptiles, gcount, G)
        i = (r - gfirst) * G + g
        u = i // ROWS
        w = wlast if u == units - 1 else PAIR
        yield from unit(reqs[gfirst][0] + h * head + u * step + start_cost(w), blocks, w, ("prefix", gfirst, h, u),
                        1 if w == PAIR else 2)
        if gfirst == r:
            own += head * Hkv
    n = own_blocks(stok)
    if n:
        yield from unit(own + h * own_cost(stok) + START_SOLO, n, SOLO, ("own", r, h, 0), 2)


@pytest.mark.parametrize("seed", range(60))
def test_work_list(seed):
    rng = random.Random(seed)
    G, Hkv, ctas = rng.randint(1, 8), rng.choice([1, 2, 5, 8]), rng.choice([1, 3, 152])
    groups = []
    for _ in range(rng.randint(1, 6)):
        n = rng.choice([1, 2, 3, 16, 40, 70])
        groups.append((rng.choice([0, 1, 7, 8, 9, 64, 500]) if n > 1 else 0,
                       [rng.choice([0, 0, 1, 128, 129, 700, 3000]) for _ in range(n)]))
    reqs, T, start = plan(groups, G, Hkv, ctas)
    if T == 0:
        return
    want = {}
    for r, (_, ptiles, stok, gfirst, gcount) in enumerate(reqs):
        for h in range(Hkv):
            if ptiles and gfirst == r:
                blocks, units, *_ = prefix_shape(ptiles, gcount, G)
                for u in range(units):
                    want["prefix", r, h, u] = set(range(blocks))
            if own_blocks(stok):
                want["own", r, h, 0] = set(range(own_blocks(stok)))
    wrote = set()
    for c in range(ctas):
        continuing = 0
        for unit, i0, i1, pair in pieces(reqs, T, start, G, Hkv, ctas, c):
            assert set(range(i0, i1)) <= want[unit]
            want[unit] -= set(range(i0, i1))
            continuing += i0 > 0
            for sub in range(1 if pair else 2):
                key = unit, ("start" if i0 == 0 else c), sub
                assert key not in wrote
                wrote.add(key)
        assert continuing <= 1
    assert not any(want.values())
    read = set()
    for r in range(len(reqs)):
        for h in range(Hkv):
            for g in range(G):
                mine = list(merge(reqs, T, G, Hkv, ctas, r, h, g))
                assert len(mine) == len(set(mine)) and set(mine) <= wrote
                read |= set(mine)
    assert read == wrote
