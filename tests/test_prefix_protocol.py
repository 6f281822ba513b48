"""CPU model of the barriers inside the shared-prefix attention kernel: its warps as
coroutines that run in a random order, products and copies that finish late, and
barriers that tell a waiter no more than a phase's parity.  Every run has to end,
and every read has to find what it waits for: the block, the piece and the queries
that the reader is at."""
import random

import pytest

PIECES = 4


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


def simulate(pieces, fp8, seed, slow=None, pieces_ring=PIECES):
    """pieces: [(pair, blocks, halves of the last block)]; slow: a warp that hardly ever gets its turn"""
    rng = random.Random(seed)
    KST, VST, V16 = (4, 2, 2) if fp8 else (2, 3, 0)
    kst, ready_n = KST, V16 if fp8 else VST
    B = dict(kfull=[Bar(1) for _ in range(kst)], kfree=[Bar(2) for _ in range(kst)],
             vfull=[Bar(1) for _ in range(VST)], vfree=[Bar(4 if fp8 else 2) for _ in range(VST)],
             ready=[Bar(4) for _ in range(ready_n)], used=[Bar(2) for _ in range(V16)],
             S=[Bar(1), Bar(1)], P=[[Bar(4), Bar(4)], [Bar(4), Bar(4)]], O=[Bar(1), Bar(1)],
             ofree=[Bar(4), Bar(4)], Q=[Bar(1), Bar(1)], qfree=[Bar(10), Bar(10)],
             piece=[Bar(1) for _ in range(pieces_ring)], piecefree=[Bar(16) for _ in range(pieces_ring)])
    late = []                       # (order in its queue, effect)
    queues = {}
    slots = [None] * pieces_ring
    qof = [None, None]              # piece whose queries a buffer holds
    kof, vof, cof = [None] * kst, [None] * VST, [None] * ready_n
    sof, oof = [None, None], [None, None]
    nb = len(pieces)
    turned = [0, 0]

    def later(queue, effect):
        queues.setdefault(queue, []).append(effect)

    def wait(bar, phase):
        while not bar.done(phase):
            yield

    def take(pn):
        yield from wait(B["piece"][pn % pieces_ring], pn // pieces_ring)
        assert slots[pn % pieces_ring] is not None and slots[pn % pieces_ring][0] == pn, "piece slot"
        p = slots[pn % pieces_ring]
        yield
        B["piecefree"][pn % pieces_ring].arrive()
        return p

    def plan():
        qbuf = tile = 0
        for n in range(nb + 1):
            slot = (n, qbuf, tile) + (pieces[n] if n < nb else (0, 0, 0))
            qbuf ^= 1
            tile ^= slot[4] & 1
            if n >= pieces_ring:
                yield from wait(B["piecefree"][n % pieces_ring], n // pieces_ring - 1)
            slots[n % pieces_ring] = slot
            yield
            B["piece"][n % pieces_ring].arrive()
            yield

    def loader(full, free, stages, hold, name):
        j = pn = 0
        while True:
            k, qb, t0, pair, blocks, tail = yield from take(pn)
            pn += 1
            if not blocks:
                return
            for i in range(blocks):
                s, r = j % stages, j // stages
                if r > 0:
                    yield from wait(free[s], r - 1)

                def land(s=s, at=(k, i)):
                    hold[s] = at
                    full[s].arrive()
                later((name, s), land)
                j += 1
                yield

    def vwarp():
        j = pn = 0
        while True:
            k, qb, t0, pair, blocks, tail = yield from take(pn)
            pn += 1
            if not blocks:
                return
            for i in range(blocks):
                vs = j % VST
                yield from wait(B["vfull"][vs], j // VST)
                assert vof[vs] == (k, i), "V block"
                if fp8:
                    buf = j % V16
                    if j >= V16:
                        yield from wait(B["used"][buf], j // V16 - 1)
                    cof[buf] = (k, i)
                    yield
                    B["ready"][buf].arrive()
                    B["vfree"][vs].arrive()
                else:
                    cof[vs] = (k, i)
                    B["ready"][vs].arrive()
                j += 1
                yield

    def mma(t):
        j0 = v3 = v3r = begun = pn = 0
        n = [0, 0]
        uses = [0, 0]
        q = ("mma", t)
        while True:
            k, qb, t0, pair, blocks, tail = yield from take(pn)
            pn += 1
            if not blocks:
                return
            assert t0 == j0 % 2
            for b in (0, 1):
                if pair or qb == b:
                    yield from wait(B["Q"][b], uses[b])
                    uses[b] += 1
            mine_buf = t if pair else qb
            begins, step, passed = True, 1 if pair else 2, 0

            def pass_v(m):
                nonlocal passed, v3, v3r
                while not fp8 and passed < m:
                    yield from wait(B["ready"][v3], v3r)
                    assert cof[v3] == (k, passed), "V block passed"
                    yield
                    B["vfree"][v3].arrive()
                    passed += 1
                    v3 += 1
                    if v3 == VST:
                        v3, v3r = 0, v3r + 1

            i = 0 if pair else (j0 ^ t) & 1
            while i < blocks + step:
                m, ks = i - step, (j0 + i) % kst
                if i < blocks:
                    yield from wait(B["kfull"][ks], (j0 + i) // kst)
                    assert kof[ks] == (k, i), "K block"
                if i >= step:
                    yield from pass_v(m)
                    vs, vr = ((j0 + m) % V16, (j0 + m) // V16) if fp8 else (v3, v3r)
                    yield from wait(B["ready"][vs], vr)
                    assert cof[vs] == (k, m), "converted block"
                    if begins and begun > 0:
                        yield from wait(B["ofree"][t], begun - 1)
                    yield from wait(B["P"][t][0], n[0])
                    n[0] += 1
                # (a turn is waited for a while, then gone without: nothing depends on it)
                for _ in range(rng.randint(0, 5)):
                    if turned[t ^ 1] - turned[t] < t:
                        yield
                effects = []
                if i >= step:
                    if m < blocks - 1 or tail == 2:
                        yield from wait(B["P"][t][1], n[1])
                        n[1] += 1
                    begun += begins
                    begins = False

                    def pv(at=(k, m), vs=vs, freed=(B["used"] if fp8 else B["vfree"])[vs], c=2 if fp8 and not pair else 1):
                        assert cof[vs] == at, "V under a product"
                        oof[t] = at
                        B["O"][t].arrive()
                        freed.arrive(c)
                    effects.append(pv)
                    if not fp8:
                        passed += 1
                        v3 += 1
                        if v3 == VST:
                            v3, v3r = 0, v3r + 1
                if i < blocks:
                    def s(at=(k, i), ks=ks, b=mine_buf, c=1 if pair else 2):
                        assert kof[ks] == at and qof[b] == at[0], "operands of S"
                        sof[t] = at
                        B["S"][t].arrive()
                        B["kfree"][ks].arrive(c)
                    effects.insert(0, s)  # (its arrivals are asked for first, and come with the products')
                for e in effects:
                    later(q, e)
                turned[t] += pair
                yield
                i += step
            yield from pass_v(blocks)
            j0 += blocks
            for b in (0, 1):
                if pair or qb == b:
                    later(q, lambda b=b: B["qfree"][b].arrive())

    def softmax(t, w):
        ns = pn = 0
        uses = [0, 0]
        while True:
            k, qb, t0, pair, blocks, tail = yield from take(pn)
            pn += 1
            if not blocks:
                return
            b = t if pair else qb
            if (pair or t == 0) and w == 0:
                if uses[b] > 0:
                    yield from wait(B["qfree"][b], uses[b] - 1)

                def landed(b=b, k=k):
                    qof[b] = k
                    B["Q"][b].arrive()
                later(("q", b), landed)
            yield from wait(B["Q"][b], uses[b])
            assert qof[b] == k, "queries"
            yield
            for x in (0, 1):
                if pair or qb == x:
                    uses[x] += 1
            B["qfree"][b].arrive(2 if pair else 1)
            some = False
            for i in range(0 if pair else t ^ t0, blocks, 1 if pair else 2):
                yield from wait(B["S"][t], ns)
                if ns > 0:
                    yield from wait(B["O"][t], ns - 1)
                assert sof[t] == (k, i), "S"
                for h in range(tail if i == blocks - 1 else 2):
                    yield
                    B["P"][t][h].arrive()
                ns += 1
                some = True
            if some:
                yield from wait(B["O"][t], ns - 1)
                assert oof[t][0] == k, "O"
                yield
                B["ofree"][t].arrive()

    tasks = [plan(), loader(B["kfull"], B["kfree"], kst, kof, "k"), loader(B["vfull"], B["vfree"], VST, vof, "v"),
             mma(0), mma(1)] + [vwarp() for _ in range(4)] + [softmax(t, w) for t in (0, 1) for w in range(4)]
    weight = [0.002 if i == slow else rng.choice([1, 1, 3, 20]) for i in range(len(tasks))]
    def state():
        return [b.phase * 1000 + b.left for v in B.values() for x in v for b in (x if isinstance(x, list) else [x])]

    def step(i):
        try:
            next(tasks[i])
        except StopIteration:
            tasks[i] = None

    while any(tasks):
        before = state()
        for _ in range(300):
            if queues and rng.random() < 0.3:
                key = rng.choice(list(queues))
                queues[key].pop(0)()
                if not queues[key]:
                    del queues[key]
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
        key = next(iter(queues))
        queues[key].pop(0)()
        if not queues[key]:
            del queues[key]


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("kind", ["pairs", "solo", "mixed", "long"])
def test_every_run_ends(fp8, kind):
    for seed in range(18):
        rng = random.Random(seed * 7 + len(kind))
        many = rng.randint(5, 9)
        if kind == "long":
            pieces = [(rng.randint(0, 1), 9), (rng.randint(0, 1), 8)]
        else:
            pieces = [({"pairs": 1, "solo": 0}.get(kind, rng.randint(0, 1)), rng.choice([1, 1, 2, 3, 4])) for _ in range(many)]
        # each warp held back in turn
        simulate([p + (rng.randint(1, 2),) for p in pieces], fp8, seed, slow=seed - 1)
