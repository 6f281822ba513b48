"""CPU model of what the prompt attention kernel keeps in its query buffers: queries, put there some
pieces ahead, read by the score products of every block, and a piece's results, staged there behind
its last product and read late.  Pieces take the two pairs of buffers in turn, those without blocks
(dead requests, rows that see nothing) too, but these hold none: nothing waits for them."""
import random

import pytest

from test_prefill_plan import pieces, ranges, units_of

RING, V_AHEAD = 4, 2  # pieces known ahead, V blocks converted ahead of their product


def simulate(blocks_of, seed, empty_stages):
    """blocks_of: blocks of each piece of a CTA.  empty_stages: whether pieces without blocks stage their zeroes."""
    rng = random.Random(seed)
    n = len(blocks_of)
    holds, filled, freed = [None, None], [0] * n, [0] * n  # of the buffers; pieces whose queries are there, are read
    taken = dict(convert=0, softmax=0)
    asked, scored, converted, multiplied = 0, 0, 0, 0
    late = []  # reads of staged results, in order
    first = [sum(blocks_of[:k]) for k in range(n + 1)]

    def known(k):  # the piece ring: a slot is written again once everybody has taken it
        return k < RING + min(taken.values())

    def convert():
        nonlocal converted
        last = [None, None]  # piece that has a buffer
        done = 0             # V blocks of the pieces before
        for k in range(n):
            while not known(k):
                yield
            taken["convert"] = k + 1
            if blocks_of[k]:
                b = k & 1
                while last[b] is not None and not freed[last[b]]:
                    # V of the piece before goes on meanwhile
                    if converted < done and converted < multiplied + V_AHEAD:
                        converted += 1
                    yield
                assert holds[b] is None or holds[b][0] == "read", f"piece {k}'s queries over {holds[b]}"
                holds[b], last[b] = ("queries", k), k
                yield
                filled[k] = 1
            while converted < done:  # the piece before is over before the next is known to be this one's
                if converted < multiplied + V_AHEAD:
                    converted += 1
                yield
            done += blocks_of[k]
        while converted < done:
            if converted < multiplied + V_AHEAD:
                converted += 1
            yield

    def products():
        nonlocal scored
        for k in range(n):
            for i in range(blocks_of[k]):
                while not filled[k] or asked < first[k] + i:
                    yield
                assert holds[k & 1] == ("queries", k), f"scores of piece {k}'s block {i} read {holds[k & 1]}"
                scored += 1
                yield

    def softmax():
        nonlocal asked, multiplied
        for k in range(n):
            while not known(k):
                yield
            for i in range(blocks_of[k]):
                while scored <= first[k] + i or converted <= first[k] + i:
                    yield
                asked += 1
                multiplied += 1
                yield
            taken["softmax"] = k + 1
            b = k & 1
            if blocks_of[k] or empty_stages:
                if blocks_of[k] == 0:
                    assert holds[b] is None or holds[b][0] == "read", f"piece {k}'s zeroes over {holds[b]}"
                holds[b] = ("results", k)
                yield
                late.append(k)
                while k in late:
                    yield
                assert holds[b] == ("results", k), f"results of piece {k} are {holds[b]}"
                holds[b] = ("read", k)
                freed[k] = 1
            yield

    def store():
        while True:
            if late:
                assert holds[late[0] & 1] == ("results", late[0]), "results read by their store"
                late.pop(0)
            yield

    tasks = [convert(), products(), softmax(), store()]
    weight = [rng.choice([1, 1, 4, 20]) for _ in tasks]
    live = [True] * 3
    for _ in range(100000):
        i = rng.choices(range(4), weight)[0]
        if i == 3 or live[i]:
            try:
                next(tasks[i])
            except StopIteration:
                live[i] = False
        if not any(live):
            return
    raise AssertionError("a warp waits for ever")


SCENES = [[2, 0, 0, 3], [2, 0, 0, 3, 0, 0, 0, 2], [2, 0, 2, 2], [0, 0, 3, 1], [4, 4, 0, 4, 4], [1, 0, 1, 0, 1, 0, 0, 0, 0, 1]]


@pytest.mark.parametrize("scene", SCENES)
def test_buffers_hold_what_is_read(scene):
    for seed in range(200):
        simulate(scene, seed, empty_stages=False)


def test_random_scenes():
    for seed in range(400):
        rng = random.Random(seed)
        simulate([rng.choice([0, 0, 1, 2, 3]) for _ in range(rng.randint(3, 14))], seed, empty_stages=False)


@pytest.mark.parametrize("scene", SCENES[:2])
def test_zeroes_have_no_place_there(scene):
    """What staging the zeroes too would come to: they meet queries of the piece two behind."""
    met = 0
    for seed in range(50):
        try:
            simulate(scene, seed, empty_stages=True)
        except AssertionError as e:
            met += "zeroes over" in str(e)
    assert met > 25


@pytest.mark.parametrize("requests", [
    [(1024, 1024, r != 3) for r in range(8)], [(1024, 1024, r != 0) for r in range(8)],
    [(512, 512, r != 4) for r in range(16)], [(4, 4 + 37 * r % 600, r % 7 not in (1, 2)) for r in range(64)],
])
def test_batches_that_come_to_it(requests):
    """One dead request, or two neighbours, give some CTAs a piece without blocks two before one with blocks."""
    units, T = units_of(requests, 8, True)
    at, _ = ranges(units, T, 8, 152)
    met = 0
    for c in range(152):
        blocks = [i1 - i0 for _, _, i0, i1 in pieces(units, T, 8, at[c], at[c + 1])]
        met += any(a == 0 and b > 0 for a, b in zip(blocks, blocks[2:]))
        simulate(blocks, c, empty_stages=False)
    assert met
