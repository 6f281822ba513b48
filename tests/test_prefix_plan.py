"""CPU model of the shared-prefix attention's work list: every block of every unit
belongs to exactly one CTA, a CTA finds its first unit from the planner's group,
at most one of its pieces continues a unit, and the merge of a row visits exactly
the partials that the pieces wrote."""
import random

import pytest

PAIR, SOLO, START_PAIR, START_SOLO, ROWS, BLK = 6, 2, 12, 5, 256, 8


def start_cost(w):
    return START_PAIR if w == PAIR else START_SOLO


def shape(ptiles, count, G):
    """blocks, units per kv head, cost of the last one's blocks, cost of a full unit, of a kv head"""
    rows = count * G
    blocks, units = -(-ptiles // BLK), -(-rows // ROWS)
    wlast = PAIR if rows - (units - 1) * ROWS > 128 else SOLO
    step = START_PAIR + PAIR * blocks
    return blocks, units, wlast, step, step * (units - 1) + start_cost(wlast) + wlast * blocks


def owned(y, n, w, b0, b1):
    return tuple(min(n, (max(b - y, 0) + w - 1) // w) for b in (b0, b1))


def begin(c, T, n):
    return c * (T // n) + min(c, T % n)


def owner(y, T, n):
    share, more = divmod(T, n)
    return y // (share + 1) if y < more * (share + 1) else more + (y - more * (share + 1)) // share


def plan(groups, G, Hkv, ctas):
    """groups: [(ptiles, requests)]; every group's place, the list's length, every CTA's first group"""
    places, T = [], 0
    for ptiles, count in groups:
        places.append(T)
        T += shape(ptiles, count, G)[4] * Hkv if ptiles else 0
    start = [max(g for g, y in enumerate(places) if y <= begin(c, T, ctas)) for c in range(ctas)]
    return places, T, start


def pieces(groups, places, T, g, G, Hkv, ctas, c):
    b0, b1 = begin(c, T, ctas), begin(c + 1, T, ctas)
    if b0 >= b1:
        return
    *_, step, head = shape(*groups[g], G)
    units = shape(*groups[g], G)[1]
    h = (b0 - places[g]) // head
    u = min((b0 - places[g] - h * head) // step, units - 1)
    y = places[g] + h * head + u * step
    assert h < Hkv
    while y < b1:
        if groups[g][0] == 0 or h == Hkv:
            g += 1
            if g >= len(groups):
                return
            h, u, y = 0, 0, places[g]
            continue
        blocks, units, wlast, step, head = shape(*groups[g], G)
        w = wlast if u == units - 1 else PAIR
        i0, i1 = owned(y + start_cost(w), blocks, w, b0, b1)
        pair = min(ROWS, groups[g][1] * G - u * ROWS) > 128
        assert pair == (w == PAIR)
        if i0 < i1:
            yield (g, h, u), i0, i1, pair
        y += start_cost(w) + blocks * w
        u += 1
        if u == units:
            u, h = 0, h + 1


def merge(groups, places, T, G, ctas, g, h, i):
    """(unit, start slot or CTA slot, sub) of the partials that row i of a group's kv head reads."""
    blocks, units, wlast, step, head = shape(*groups[g], G)
    u = i // ROWS
    w = wlast if u == units - 1 else PAIR
    y = places[g] + h * head + u * step + start_cost(w)
    for c in range(owner(y, T, ctas), owner(y + (blocks - 1) * w, T, ctas) + 1):
        i0, i1 = owned(y, blocks, w, begin(c, T, ctas), begin(c + 1, T, ctas))
        for sub in range(1 if w == PAIR else 2):
            if i0 < i1:
                yield (g, h, u), ("start" if i0 == 0 else c), sub


@pytest.mark.parametrize("seed", range(80))
def test_work_list(seed):
    rng = random.Random(seed)
    G, Hkv, ctas = rng.randint(1, 8), rng.choice([1, 2, 5, 8]), rng.choice([1, 3, 152])
    groups = [(rng.choice([0, 1, 7, 8, 9, 64, 500]), rng.choice([2, 3, 16, 17, 40, 70])) for _ in range(rng.randint(1, 7))]
    places, T, start = plan(groups, G, Hkv, ctas)
    if T == 0:
        return
    want = {}
    for g, (ptiles, count) in enumerate(groups):
        if ptiles:
            blocks, units, *_ = shape(ptiles, count, G)
            for h in range(Hkv):
                for u in range(units):
                    want[g, h, u] = set(range(blocks))
    wrote = set()
    for c in range(ctas):
        continuing = 0
        for unit, i0, i1, pair in pieces(groups, places, T, start[c], G, Hkv, ctas, c):
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
    for g, (ptiles, count) in enumerate(groups):
        for h in range(Hkv if ptiles else 0):
            for i in range(count * G):
                mine = list(merge(groups, places, T, G, ctas, g, h, i))
                assert len(mine) == len(set(mine)) and set(mine) <= wrote
                read |= set(mine)
    assert read == wrote
