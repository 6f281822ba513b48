"""CPU model of the barriers inside the prompt attention kernel: its warps as coroutines that run
in a random order, products and copies that finish late, and barriers that tell a waiter no more
than a phase's parity.  Every run has to end, and every read has to find what it waits for: the
piece, its queries, the block, its scales, its product."""
import random

import pytest

PIECES, SCALES, KST, V16 = 4, 8, 2, 2


class Bar:
    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self, n=1):
        for _ in range(n):
            self.left -= 1
            if self.left == 0:
                self.left, self.phase = self.count, self.phase + 1

    def done(self, phase):
        return (self.phase & 1) != (phase & 1)


def simulate(pieces, seed, slow=None):
    """pieces: [(pair, blocks, halves of the last block, steps of its queries)]; slow: a warp that hardly ever gets its turn"""
    rng = random.Random(seed)
    B = dict(kfull=[Bar(1) for _ in range(KST)], kfree=[Bar(2) for _ in range(KST)],
             ready=[Bar(4) for _ in range(V16)], used=[Bar(2) for _ in range(V16)],
             S=[Bar(1), Bar(1)], P=[[Bar(4), Bar(4)], [Bar(4), Bar(4)]], O=[Bar(1), Bar(1)], half=[Bar(1), Bar(1)],
             ofree=[Bar(4), Bar(4)], Q=[Bar(4) for _ in range(4)], qfree=[Bar(10) for _ in range(4)],
             piece=[Bar(1) for _ in range(PIECES)], piecefree=[Bar(15) for _ in range(PIECES)],
             scale=[Bar(1) for _ in range(SCALES)], scalefree=[Bar(12) for _ in range(SCALES)], join=[Bar(4)])
    queues = {}
    slots, scales = [None] * PIECES, [None] * SCALES
    qof = [[None] * 4 for _ in range(4)]          # piece whose rows each converting warp left in a buffer
    kof, cof = [None] * KST, [[None] * 4 for _ in range(V16)]
    sof, oof, hof, joined = [None, None], [None, None], [None, None], [None] * 4
    turned = [0, 0]
    count = len(pieces)

    def later(queue, effect):
        queues.setdefault(queue, []).append(effect)

    def wait(bar, phase):
        while not bar.done(phase):
            yield

    def take(pn, keep=False):
        yield from wait(B["piece"][pn % PIECES], pn // PIECES)
        p = slots[pn % PIECES]
        assert p is not None and p[0] == pn, "piece slot"
        yield
        if not keep:
            B["piecefree"][pn % PIECES].arrive()
        return p

    def plan():
        j = qset = t0 = 0
        for n in range(count + 1):
            pair, blocks, tail, steps = pieces[n] if n < count else (0, 0, 0, 0)
            if n >= PIECES:
                yield from wait(B["piecefree"][n % PIECES], n // PIECES - 1)
            slots[n % PIECES] = (n, qset, t0, pair, blocks, tail, steps, n == count)
            qset ^= 1
            t0 ^= blocks & 1
            yield
            B["piece"][n % PIECES].arrive()
            for i in range(blocks):
                if j >= SCALES:
                    yield from wait(B["scalefree"][j % SCALES], j // SCALES - 1)
                scales[j % SCALES] = (n, i)
                yield
                B["scale"][j % SCALES].arrive()
                j += 1

    def loader():
        j = pn = 0
        while True:
            k, _, _, _, blocks, _, _, last = yield from take(pn)
            pn += 1
            if last:
                return
            for i in range(blocks):
                s = j % KST
                if j >= KST:
                    yield from wait(B["kfree"][s], j // KST - 1)

                def land(s=s, at=(k, i)):
                    kof[s] = at
                    B["kfull"][s].arrive()
                later(("k", s), land)
                j += 1
                yield

    def vwarp(w):
        j = pn = i = blocks = at = n = 0
        known, k, nxt = False, -1, None
        used, phases = set(), [0] * 4

        def first_of(key):
            yield from wait(B["scale"][j % SCALES], j // SCALES)
            assert scales[j % SCALES] == key, "scales of a piece's first block"
            yield
            B["scalefree"][j % SCALES].arrive()

        while True:
            queries = known and at < n
            if i < blocks and (not queries or j < V16 or B["used"][j % V16].done(j // V16 - 1)):
                if i + 1 < blocks:
                    yield from wait(B["scale"][(j + 1) % SCALES], (j + 1) // SCALES)
                    assert scales[(j + 1) % SCALES] == (k, i + 1), "scales"
                if j >= V16:
                    yield from wait(B["used"][j % V16], j // V16 - 1)
                cof[j % V16][w] = (k, i)
                yield
                if i + 1 < blocks:
                    B["scalefree"][(j + 1) % SCALES].arrive()
                B["ready"][j % V16].arrive()
                i += 1
                j += 1
            elif queries:
                end = n if i == blocks else at + 2
                while at < end:
                    buf = 2 * nxt[1] + (at >> 3)
                    if at & 7 == 0:
                        if buf in used:
                            yield from wait(B["qfree"][buf], phases[buf])
                            phases[buf] += 1
                        used.add(buf)
                    qof[buf][w] = nxt[0]
                    yield
                    at += 2
                    if at & 7 == 0 or at == n:
                        B["Q"][buf].arrive()
            if not known and blocks - i <= SCALES and (i == blocks or B["piece"][pn % PIECES].done(pn // PIECES)):
                nxt = yield from take(pn)
                pn += 1
                known, at = True, 0
                n = 0 if nxt[7] or nxt[4] == 0 else nxt[6]
            if i == blocks and known and at >= n:
                if nxt[7]:
                    return
                k, _, _, _, blocks, _, _, _ = nxt
                known, i = False, 0
                if blocks:
                    yield from first_of((k, 0))
            yield

    def mma(t):
        j0 = begun = pn = 0
        n = [0, 0]
        phases = [0] * 4
        q = ("mma", t)
        while True:
            k, qset, t0, pair, blocks, tail, _, last = yield from take(pn)
            pn += 1
            if last:
                return
            if blocks == 0:
                continue
            assert t0 == j0 % 2
            mine, begins, step = 2 * qset + (t if pair else 0), True, 1 if pair else 2
            yield from wait(B["Q"][mine], phases[mine])
            for b in (2 * qset, 2 * qset + 1)[:1 + pair]:
                phases[b] += 1
            i = 0 if pair else (j0 ^ t) & 1
            while i < blocks + step:
                m, ks = i - step, (j0 + i) % KST
                vs = (j0 + m) % V16
                if i < blocks:
                    yield from wait(B["kfull"][ks], (j0 + i) // KST)
                if i >= step:
                    yield from wait(B["ready"][vs], (j0 + m) // V16)
                    if begins and begun > 0:
                        yield from wait(B["ofree"][t], begun - 1)
                    yield from wait(B["P"][t][0], n[0])
                    n[0] += 1
                for _ in range(rng.randint(0, 5)):  # (a turn is waited for a while, then gone without)
                    if pair and turned[t ^ 1] - turned[t] < t:
                        yield
                if i >= step:
                    def first(at=(k, m), vs=vs):
                        assert cof[vs] == [at] * 4, "V under the first half's product"
                        hof[t] = at
                        B["half"][t].arrive()
                    later(q, first)
                    if m < blocks - 1 or tail == 2:
                        yield from wait(B["P"][t][1], n[1])
                        n[1] += 1

                    def both(at=(k, m), vs=vs):
                        assert cof[vs] == [at] * 4, "V under a product"
                        oof[t] = at
                        B["O"][t].arrive()
                    later(q, both)
                    begun += begins
                    begins = False
                if i < blocks:
                    def s(at=(k, i), ks=ks, b=mine, c=1 if pair else 2):
                        assert kof[ks] == at and qof[b] == [at[0]] * 4, "operands of S"
                        sof[t] = at
                        B["S"][t].arrive()
                        B["kfree"][ks].arrive(c)
                    later(q, s)
                turned[t] += pair
                if i >= step:
                    later(q, lambda vs=vs, c=1 if pair else 2: B["used"][vs].arrive(c))
                yield
                i += step
            j0 += blocks
            later(q, lambda b=mine, c=1 + pair: B["qfree"][b].arrive(c))

    def softmax(t, w):
        ns = pn = joins = j0 = 0
        phases = [0] * 4
        while True:
            k, qset, t0, pair, blocks, tail, _, last = yield from take(pn, keep=True)
            pn += 1
            if last:
                return
            buf = 2 * qset + (t if pair else 0)
            some = False
            if blocks:
                yield from wait(B["Q"][buf], phases[buf])
                assert qof[buf] == [k] * 4, "queries"
                for b in (2 * qset, 2 * qset + 1)[:1 + pair]:
                    phases[b] += 1
                for i in range(0 if pair else t ^ t0, blocks, 1 if pair else 2):
                    st = (j0 + i) % SCALES
                    yield from wait(B["scale"][st], (j0 + i) // SCALES)
                    assert scales[st] == (k, i), "scales of S"
                    yield from wait(B["S"][t], ns)
                    assert sof[t] == (k, i), "S"
                    assert not some or oof[t][0] == k, "O grows while it belongs to the piece"
                    for h in range(tail if i == blocks - 1 else 2):
                        yield
                        if h and rng.random() < 0.3:      # a maximum that grows in the second half
                            yield from wait(B["half"][t], ns)
                            assert hof[t] == (k, i), "first half's product"
                        B["P"][t][h].arrive()
                    assert scales[st] == (k, i), "scales kept"
                    B["scalefree"][st].arrive(1 if pair else 2)
                    ns += 1
                    some = True
                if some:
                    yield from wait(B["O"][t], ns - 1)
                    assert oof[t][0] == k, "O"
            j0 += blocks
            assert slots[(pn - 1) % PIECES][0] == k, "piece slot, read again"
            yield
            B["piecefree"][(pn - 1) % PIECES].arrive()
            if not pair and t == 1:
                if blocks:
                    if some:
                        joined[w] = k
                        yield
                        B["join"][0].arrive()
                    B["qfree"][buf].arrive()
                continue
            other = not pair and blocks > 0 and (1 ^ t0) < blocks
            if other:
                yield from wait(B["join"][0], joins)
                joins += 1
                assert joined[w] == k and oof[1][0] == k, "the other tile's part"
            yield
            if some:
                assert oof[t][0] == k, "O read"
                B["ofree"][t].arrive()
            if other:
                assert joined[w] == k and oof[1][0] == k, "the other tile's O read"
                B["ofree"][1].arrive()
            yield
            if blocks:
                assert qof[buf] == [k] * 4, "results staged over its own queries"
                B["qfree"][buf].arrive(2 if pair else 1)

    tasks = [plan(), loader(), mma(0), mma(1)] + [vwarp(w) for w in range(4)] + [softmax(t, w) for t in (0, 1) for w in range(4)]
    weight = [0.002 if i == slow else rng.choice([1, 1, 3, 20]) for i in range(len(tasks))]

    def state():
        return [b.phase * 1000 + b.left for v in B.values() for x in v for b in (x if isinstance(x, list) else [x])]

    def step(i):
        try:
            next(tasks[i])
        except StopIteration:
            tasks[i] = None

    def finish_one():
        key = rng.choice(list(queues))
        queues[key].pop(0)()
        if not queues[key]:
            del queues[key]

    while any(tasks):
        before = state()
        for _ in range(300):
            if queues and rng.random() < 0.3:
                finish_one()
                continue
            i = rng.choices(range(len(tasks)), weight)[0]
            if tasks[i]:
                step(i)
        if state() == before:
            # everybody has its turn: something has to move
            for i in list(range(len(tasks))) * 8:
                if tasks[i]:
                    step(i)
            assert queues or state() != before or not any(tasks), f"{sum(map(bool, tasks))} warps wait for ever"
    while queues:
        finish_one()


@pytest.mark.parametrize("kind", ["pairs", "solo", "mixed", "long", "empty"])
def test_every_run_ends(kind):
    for seed in range(20):
        rng = random.Random(seed * 7 + len(kind))
        if kind == "long":
            shapes = [(rng.randint(0, 1), 19), (rng.randint(0, 1), 18), (rng.randint(0, 1), 11)]
        else:
            blocks = [0, 0, 1, 2] if kind == "empty" else [1, 1, 2, 3, 4]
            shapes = [({"pairs": 1, "solo": 0}.get(kind, rng.randint(0, 1)), rng.choice(blocks)) for _ in range(rng.randint(5, 11))]
        # each warp held back in turn
        simulate([(pair, n, rng.randint(1, 2), (8 if pair else 0) + 2 * rng.randint(1, 4)) for pair, n in shapes], seed, slow=seed - 1)
