"""CPU model of the prompt attention's work list: every block of every unit belongs to exactly
one CTA, a unit without tokens to the one that holds its place, at most one of a CTA's pieces
continues a unit and at most one leaves its end to others, and the merge of a unit visits
exactly the partials that the pieces wrote, in slots of their own; or the units are dealt out whole."""
import random

import pytest

PAIR, SOLO, START_PAIR, START_SOLO, CUT, ROWS, BLK = 6, 4, 20, 16, 48, 256, 128


def units_of(requests, G, causal):
    """requests: [(query tokens, context, alive)]; a kv head's units (place, request, rows, blocks) and their length"""
    units, y = [], 0
    for r, (n, L, alive) in enumerate(requests):
        L = L if alive else 0
        for row0 in range(0, n * G, ROWS):
            rows = min(ROWS, n * G - row0)
            last = (row0 + rows - 1) // G
            tokens = min(L, max(0, (L - n if causal else L) + last + 1))
            blocks = -(-tokens // BLK)
            units.append((y, r, rows, blocks))
            y += start(rows) + cost(rows) * blocks
    return units, y


def cost(rows):
    return PAIR if rows > 128 else SOLO


def start(rows):
    return START_PAIR if rows > 128 else START_SOLO


def begin(c, line, n):
    return c * (line // n) + min(c, line % n)


def owner(y, line, n):
    share, more = divmod(line, n)
    return y // (share + 1) if y < more * (share + 1) else more + (y - more * (share + 1)) // share


def owned(rows, blocks, y, b0, b1):
    at, w = y + start(rows), cost(rows)
    return tuple(min(blocks, (max(b - at, 0) + w - 1) // w) for b in (b0, b1))


def ranges(units, T, Hkv, ctas):
    """Where the CTAs' ranges of the line begin, and its end; whether they end with units."""
    every = len(units) * Hkv
    top = max((start(u[2]) + cost(u[2]) * u[3] for u in units), default=0)
    if -(-every // ctas) * top <= T * Hkv // ctas + CUT:
        places = [h * T + u[0] for h in range(Hkv) for u in units] + [T * Hkv]
        return [places[begin(c, every, ctas)] for c in range(ctas + 1)], True
    return [begin(c, T * Hkv, ctas) for c in range(ctas + 1)], False


def unit_at(units, T, Hkv, place):
    h = min(place // T, Hkv - 1)
    return max(x for x, u in enumerate(units) if u[0] <= place - h * T), h


def pieces(units, T, Hkv, b0, b1):
    if b0 >= b1:
        return
    x, h = unit_at(units, T, Hkv, b0)
    while True:
        if x == len(units):
            x, h = 0, h + 1
            if h == Hkv:
                return
        y0, _, rows, blocks = units[x]
        y = h * T + y0
        if y >= b1:
            return
        i0, i1 = owned(rows, blocks, y, b0, b1)
        if i0 < i1 or (blocks == 0 and y >= b0):
            yield x, h, i0, i1
        x += 1


def check(requests, G, Hkv, ctas, causal):
    units, T = units_of(requests, G, causal)
    line, done, slots, cuts = T * Hkv, {}, {}, []
    at, uncut = ranges(units, T, Hkv, ctas)
    for c in range(ctas):
        b0, b1 = at[c], at[c + 1]
        whole = []
        for x, h, i0, i1 in pieces(units, T, Hkv, b0, b1):
            blocks = units[x][3]
            assert done.get((x, h), 0) == i0, "blocks in order, none twice"
            assert blocks or (x, h) not in done
            done[x, h] = i1
            whole.append((i0 == 0, i1 == blocks))
            if not (i0 == 0 and i1 == blocks):
                slot = 2 * c + (0 if i0 == 0 else 1)
                assert slot not in slots, "one partial per slot"
                slots[slot] = (x, h)
        assert sum(not first for first, _ in whole) <= 1 and sum(not last for _, last in whole) <= 1
        assert not uncut or all(x == (True, True) for x in whole)
        if b0 < b1 < line and not uncut:
            x, h = unit_at(units, T, Hkv, b1)
            y0, _, rows, blocks = units[x]
            y = h * T + y0
            i0, i1 = owned(rows, blocks, y, b0, b1)
            if i0 == 0 and 0 < i1 < blocks:
                cuts.append((c, owner(y + start(rows) + (blocks - 1) * cost(rows), line, ctas), x, h))
    assert done == {(x, h): u[3] for h in range(Hkv) for x, u in enumerate(units)}
    merged = {}
    for c, to, x, h in cuts:
        y0, _, rows, blocks = units[x]
        for k in range(c, to + 1):
            i0, i1 = owned(rows, blocks, h * T + y0, begin(k, line, ctas), begin(k + 1, line, ctas))
            if i0 < i1:
                merged[2 * k + (0 if k == c else 1)] = (x, h)
    assert merged == slots


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("G,Hkv", [(8, 8), (5, 2), (1, 7), (7, 1)])
@pytest.mark.parametrize("requests", [
    [(1, 1, True)], [(4, 131072, True)], [(8192, 8192, True)], [(512, 512, True)] * 16, [(4, 2048, True)] * 16,
    [(0, 5, True), (300, 10, True), (3, 0, True), (0, 0, True), (40, 4000, False), (700, 3000, True)],
])
def test_shapes(requests, G, Hkv, causal):
    for ctas in (152, 148, 3, 1):
        check(requests, G, Hkv, ctas, causal)


@pytest.mark.parametrize("seed", range(150))
def test_random_shapes(seed):
    rng = random.Random(seed)
    requests = [(rng.choice([0, 1, 2, rng.randrange(600)]), rng.choice([0, 1, rng.randrange(300), rng.randrange(20000)]),
                 rng.random() < 0.9) for _ in range(rng.randrange(1, 40))]
    check(requests, rng.randrange(1, 9), rng.randrange(1, 9), rng.choice([152, 152, 7, 1]), rng.random() < 0.7)
