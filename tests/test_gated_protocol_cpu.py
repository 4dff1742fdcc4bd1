"""Discrete-event check of the gated feed-forward kernel's mbarrier protocol (CPU only).

k_gated (smc_gated.cu) runs on pairs of CTAs: each CTA's producer loads its own
operands into its own ring, the leader's MMA warp multiplies from both rings into
both CTAs' tensor memory, and sixteen epilogue warps per CTA take the sums.  The
barriers are waited on by phase parity, across the two CTAs:

* full (leader's): the leader's announcement, and the bytes of both CTAs' loads,
  which may land before the announcement;
* empty, tfull (one in each CTA): the leader's commits arrive on both;
* tempty (leader's): one arrival from each of the 32 epilogue warps;
* dh (per epilogue warp, two): the copy of the gradient's chunk for a tile, asked
  for one tile ahead, only for tiles in which the warp has rows and columns.

This test runs the roles of a pair as coroutines over random tiles with random
latencies and checks that every wait is for the phase it means, that no ring slot,
accumulator or staging slot is written while it is read, that every consumer finds
what it expects, and that all roles end.  Long sums come in pieces, an accumulator
each.  Mistakes planted in the model have to be caught.
"""
import random

import pytest

from test_protocol_cpu import Bar, Cta

WARPS = 16


class RemoteBar(Bar):
    """Bytes of the other CTA may land before they are announced."""

    def complete_tx(self, b):
        self.tx -= b
        self._check()


class Pair(Cta):
    """One pair of CTAs over its list of segments (numbers of stages)."""

    def __init__(self, rng, segs, stages, piece, dh, mistake=None):
        self.rng, self.segs, self.stages, self.piece, self.dh = rng, segs, stages, piece, dh
        self.mistake = mistake
        self.t = self.seq = 0
        self.events = []
        self.full = [RemoteBar(f"full{s}", 1) for s in range(stages)]
        self.empty = [[Bar(f"empty{r}.{s}", 1) for s in range(stages)] for r in range(2)]
        self.tfull = [[Bar(f"tfull{r}.{a}", 1) for a in range(2)] for r in range(2)]
        count = WARPS if mistake == "half of the hand-backs" else 2 * WARPS
        self.tempty = [Bar(f"tempty{a}", count) for a in range(2)]
        self.ring = [[None] * stages for _ in range(2)]
        self.ring_reading = [[0] * stages for _ in range(2)]
        self.acc = [None, None]
        self.acc_reading = [0, 0]
        self.tensor_tail = 0
        self.done = 0
        self.taken = []
        # which warps have rows and columns of a segment's tile
        self.live = [[[rng.random() < 0.7 for _ in segs] for _ in range(WARPS)] for _ in range(2)]

    def pieces(self, k):
        """(first stage, last stage) of each accumulation of a segment."""
        step = self.piece or k
        return [(a, min(a + step, k)) for a in range(0, k, step)]

    def producer(self, rank):
        n = 0
        for seg, k in enumerate(self.segs):
            for it in range(k):
                st, use = n % self.stages, n // self.stages
                if self.mistake != "no wait for an empty slot":
                    yield ("wait", self.empty[rank][st], (use & 1) ^ 1, use - 1)
                assert not self.ring_reading[rank][st], ("ring slot written while read", rank, st)
                self.ring[rank][st] = None
                b = self.full[st]
                if rank == 0:
                    b.expect_tx(2)
                    b.arrive()

                def land(b=b, st=st, rank=rank, what=(seg, it)):
                    self.ring[rank][st] = what
                    b.complete_tx(1)
                self.at(self.t + self.delay(50, 1500), land)
                n += 1
                yield ("sleep", self.delay(1, 30))

    def commit(self, fn):
        """fn at the end of all MMAs issued so far."""
        self.at(max(self.t, self.tensor_tail) + self.delay(10, 100), fn)

    def mma(self):
        n = acc_use = 0
        for seg, k in enumerate(self.segs):
            for first, last in self.pieces(k):
                a, use = acc_use % 2, acc_use // 2
                yield ("wait", self.tempty[a], (use & 1) ^ 1, use - 1)
                acc_use += 1
                self.acc[a] = (seg, first, [])
                for it in range(first, last):
                    st = n % self.stages
                    yield ("wait", self.full[st], (n // self.stages) & 1, n // self.stages)
                    for r in range(2):
                        assert self.ring[r][st] == (seg, it), ("ring", r, st, self.ring[r][st], seg, it)
                        self.ring_reading[r][st] += 1
                    assert not self.acc_reading[a], ("accumulator written while read", a)
                    self.acc[a][2].append(it)
                    self.tensor_tail = max(self.tensor_tail, self.t) + self.delay(64, 500)

                    def release(st=st):
                        for r in range(2):
                            self.ring_reading[r][st] -= 1
                            self.empty[r][st].arrive()
                    self.commit(release)
                    n += 1
                    yield ("sleep", self.delay(1, 20))

                def ready(a=a):
                    for r in range(2):
                        self.tfull[r][a].arrive()
                if not (self.mistake == "no commit of inner pieces" and last < k):
                    self.commit(ready)

    def epilogue(self, rank, warp):
        bars = [Bar(f"dh{rank}.{warp}.{s}", 1) for s in range(2)]
        phases = [0, 0]                # of each dh barrier: the next to wait for
        slots = [None, None, None]     # dh of two tiles, then du
        stores = []                    # (end of the store's read, slot)
        live = self.live[rank][warp]

        def free(slot):
            assert all(end <= self.t or s != slot for end, s in stores), "staging written while read"

        def stores_read():
            return ("sleep", max([0] + [end - self.t for end, _ in stores]))

        def prefetch(seg, slot):
            if not live[seg]:
                return
            if self.mistake != "no wait for the last store":
                yield stores_read()
            free(slot)
            slots[slot] = None
            bars[slot].expect_tx(1)
            bars[slot].arrive()

            def land():
                slots[slot] = ("dh", seg)
                bars[slot].complete_tx(1)
            self.at(self.t + self.delay(50, 1500), land)

        use = 0
        if self.dh and self.segs:
            yield from prefetch(0, 0)
        for seg, k in enumerate(self.segs):
            slot = seg % 2
            if self.dh and seg + 1 < len(self.segs):
                yield from prefetch(seg + 1, slot ^ 1)
            for first, last in self.pieces(k):
                a = use % 2
                yield ("wait", self.tfull[rank][a], (use // 2) & 1, use // 2)
                use += 1
                if live[seg]:
                    assert self.acc[a] == (seg, first, list(range(first, last))), (self.acc[a], seg)
                    self.acc_reading[a] += 1
                    yield ("sleep", self.delay(20, 400))
                    self.acc_reading[a] -= 1
                elif self.mistake == "no hand-back without rows":
                    continue
                self.at(self.t + self.delay(1, 200), self.tempty[a].arrive)
                if not self.dh and live[seg]:
                    self.taken.append((rank, warp, seg, first))
            if not self.dh or not live[seg]:
                if self.mistake == "a phase for every tile":
                    phases[slot] += 1
                continue
            yield ("wait", bars[slot], phases[slot] & 1, phases[slot])
            phases[slot] += 1
            assert slots[slot] == ("dh", seg), (slots[slot], seg)
            yield stores_read()
            free(slot), free(2)
            slots[slot], slots[2] = ("dg", seg), ("du", seg)
            yield ("sleep", self.delay(20, 300))
            end = self.t + self.delay(10, 900)
            stores = [(end, slot), (end, 2)]
            self.taken += [(rank, warp, seg, f) for f, _ in self.pieces(k)]

    def go(self):
        roles = [self.producer(0), self.producer(1), self.mma()]
        roles += [self.epilogue(r, w) for r in range(2) for w in range(WARPS)]
        self.run(roles)
        want = sorted((r, w, s, f) for r in range(2) for w in range(WARPS)
                      for s, k in enumerate(self.segs) if self.live[r][w][s]
                      for f, _ in self.pieces(k))
        assert sorted(self.taken) == want


def _segments(rng, longest):
    return [rng.randint(1, longest) for _ in range(rng.randint(1, 7))]


# stages of the ring, stages of a piece (0: the whole sum), copies of dh
CONFIGS = [(2, 1, False), (2, 0, True), (4, 0, True), (6, 0, False), (8, 0, False), (4, 5, False),
           (8, 7, False), (3, 4, True), (2, 64, False)]


@pytest.mark.parametrize("stages,piece,dh", CONFIGS)
def test_pair_protocol(stages, piece, dh):
    for seed in range(6):
        rng = random.Random(1000 * stages + 10 * piece + seed)
        Pair(rng, _segments(rng, 20), stages, piece, dh).go()


@pytest.mark.parametrize("mistake,stages,piece,dh", [
    ("half of the hand-backs", 4, 0, False), ("no wait for an empty slot", 3, 0, False),
    ("no commit of inner pieces", 4, 3, False), ("no hand-back without rows", 4, 0, False),
    ("a phase for every tile", 4, 0, True), ("no wait for the last store", 4, 0, True),
])
def test_planted_mistakes_are_caught(mistake, stages, piece, dh):
    caught = 0
    for seed in range(8):
        rng = random.Random(seed)
        try:
            Pair(rng, [rng.randint(1, 12) for _ in range(7)], stages, piece, dh, mistake).go()
        except (AssertionError, RuntimeError):
            caught += 1
    assert caught >= 6, (mistake, caught)
