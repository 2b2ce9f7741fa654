"""Model of the tree decode's row warps: the hand-offs between a segment's queries,
its tiles and its finished row, under random schedules of one CTA.

The roles are the kernel's (producer, QK^T issue, P.V issue, two softmax
warpgroups on alternate tiles, the row warps), the barriers count arrivals and
are waited on by parity, the tensor pipe completes what it is given in order.
Each buffer carries what it holds, and each reader states what it must find.
The score exchange between the two CTAs is the other model's
(test_decode_model.py) and is left out.
"""
import random

import pytest


class Bar:
    def __init__(self, count=1):
        self.count, self.arrived, self.phase = count, 0, 0

    def arrive(self):
        self.arrived += 1
        assert self.arrived <= self.count
        if self.arrived == self.count:
            self.arrived, self.phase = 0, self.phase + 1

    def done(self, parity):
        """What a parity wait sees: the phase of that parity is complete."""
        return self.phase & 1 != parity


class Model:
    STAGES = 4

    def __init__(self, segments, seed, mistake=None):
        self.r, self.mistake = random.Random(seed), mistake
        self.tiles = [(s, i == 0, i == n - 1) for s, n in enumerate(segments) for i in range(n)]
        self.segments = segments
        self.pipe = []                                       # (reads, writes) in the order of issue
        b = Bar
        self.kv_full, self.kv_empty = [b() for _ in range(4)], [b() for _ in range(4)]
        self.s_full, self.o_done = [b(), b()], [b(), b()]
        self.s_free, self.p_full, self.q_ready, self.o_free, self.q_free, self.row_done = b(), b(), b(), b(), b(), b()
        self.page = [None] * 4
        self.q = self.s = self.p = None
        self.o = []                                          # the tiles added to O since its segment began
        self.slot = [None] * 4
        self.stored = []

    # ---- roles: generators that yield conditions to wait for
    def producer(self):
        for t in range(len(self.tiles)):
            if t >= 4:
                yield lambda t=t: self.kv_empty[t % 4].done((t // 4 - 1) & 1)
            yield None
            self.page[t % 4] = t
            self.kv_full[t % 4].arrive()

    def qk(self):
        for t, (s, first, last) in enumerate(self.tiles):
            yield lambda: self.kv_full[t % 4].done((t // 4) & 1)
            if t:
                yield lambda: self.s_free.done((t - 1) & 1)
            if first:
                yield lambda: self.q_ready.done(s & 1)

            def run(t=t, s=s):
                assert self.page[t % 4] == t and self.q == s, ("QK", t, self.page, self.q)
                assert self.s is None, ("S overwritten", t, self.s)
                self.s = t
            commits = [self.s_full[t & 1]] + ([self.q_free] if last else [])
            self.pipe.append((run, commits))
            yield None

    def pv(self):
        for t, (s, first, last) in enumerate(self.tiles):
            yield lambda: self.p_full.done(t & 1)
            if first and self.mistake != "O not waited for":
                yield lambda: self.o_free.done(s & 1)

            def run(t=t, s=s, first=first):
                assert self.p == t and self.page[t % 4] == t, ("PV", t, self.p)
                if first:
                    assert not self.o, ("O overwritten", t, self.o)
                self.o.append(t)
            self.pipe.append((run, [self.kv_empty[t % 4], self.o_done[t & 1]] + ([self.row_done] if last else [])))
            yield None

    def softmax(self, wg):
        for t in range(wg, len(self.tiles), 2):
            s, first, last = self.tiles[t]
            yield lambda: self.s_full[t & 1].done((t >> 1) & 1)
            assert self.s == t, ("scores", t, self.s)
            self.s = None
            self.s_free.arrive()
            if not first:                                    # tagged slot of the tile before
                yield lambda: self.slot[(t - 1) & 3] is not None and self.slot[(t - 1) & 3][0] == t - 1
            self.slot[t & 3] = (t, s)
            yield None
            if t:
                yield lambda: self.o_done[(t - 1) & 1].done(((t - 1) >> 1) & 1)
            assert t == 0 or (self.o and self.o[-1] == t - 1) or (not self.o and first), ("P overwritten", t, self.o)
            self.p = t
            self.p_full.arrive()
            yield None

    def rows(self):
        self.o_free.arrive()

        def finish(s, g):
            yield lambda: self.row_done.done(s & 1)
            if self.mistake == "O freed before the maximum is read":
                tiles, self.o = self.o, []
                self.o_free.arrive()
                yield None
                yield None
                assert self.slot[g & 3] == (g, s), ("maximum", g, self.slot)
            else:
                assert self.slot[g & 3] == (g, s), ("maximum", g, self.slot)
                yield None
                tiles, self.o = self.o, []
                self.o_free.arrive()
            assert tiles == [t for t, x in enumerate(self.tiles) if x[0] == s], (s, tiles)
            self.stored.append(s)

        g = 0
        for s, n in enumerate(self.segments):
            if s and self.mistake != "Q not waited for":
                yield lambda: self.q_free.done((s - 1) & 1)
            yield None
            self.q = s
            self.q_ready.arrive()
            if s:
                yield from finish(s - 1, g - 1)
            g += n
        yield from finish(len(self.segments) - 1, g - 1)

    def run(self):
        roles = [self.producer(), self.qk(), self.pv(), self.softmax(0), self.softmax(1), self.rows()]
        waits = {r: next(r, StopIteration) for r in roles}
        waits = {r: w for r, w in waits.items() if w is not StopIteration}
        slow = self.r.choice([None, *roles])                 # one role may lag far behind
        while waits or self.pipe:
            ready = [r for r, w in waits.items() if w is None or w()]
            if slow in ready and len(ready) > 1 and self.r.random() < 0.9:
                ready.remove(slow)
            if self.pipe and (not ready or self.r.random() < 0.3):
                run, commits = self.pipe.pop(0)
                run()
                for c in commits:
                    c.arrive()
                continue
            assert ready, "deadlock"
            r = self.r.choice(ready)
            w = next(r, StopIteration)
            if w is StopIteration:
                del waits[r]
            else:
                waits[r] = w
        assert self.stored == list(range(len(self.segments)))


def _shapes(seed):
    r = random.Random(seed)
    return [r.choice([1, 1, 2, 3, 4, 5, 9]) for _ in range(r.randint(1, 9))]


@pytest.mark.parametrize("block", range(8))
def test_every_row_is_stored_whole(block):
    for seed in range(100 * block, 100 * block + 100):
        Model(_shapes(seed), seed).run()


@pytest.mark.parametrize("mistake", ["Q not waited for", "O not waited for", "O freed before the maximum is read"])
def test_planted_mistakes_are_seen(mistake):
    caught = 0
    for seed in range(300):
        try:
            Model(_shapes(seed), seed, mistake).run()
        except AssertionError:
            caught += 1
    assert caught > 0
