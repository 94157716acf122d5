"""The barrier protocol of the sliding-window kernel (window_kernel) once more, with each
softmax warp's steps in the kernel's own order and every wait left out in turn.

Per tile a softmax warp waits for S, takes it (s_free), waits for the P.V of two tiles
before, writes P, and only then, where its maximum moved, waits for the P.V of the tile
before and rescales O; then p_full.  A tile that none of a warp's rows sees gets a P of
zeros without its scores being read.  After an item's last S the warp stores the next
item's Q, waits for the last P.V and reads O.  The other actors are the TMA producer (K,
then V of each tile), the S issuer and the PV issuer; copies complete in any order, the
products of one issuer in issue order.

Checked under random schedules: every wait passes on the phase it means, nothing is read
before it is there or written over before it has been read, O is rescaled and read only
between products, and every schedule ends.  Each wait, left out alone, has to show in some
schedule."""
import random

import pytest

WARPS = 4
WAITS = ["k_full", "v_full", "k_empty", "v_empty", "s_full", "s_free", "p_full", "q_full", "p_slot", "rescale", "epilogue"]


class Violation(Exception):
    pass


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.done = count, 0, 0

    def arrive(self):
        self.pending += 1
        if self.pending == self.count:
            self.pending, self.done = 0, self.done + 1


class Model:
    def __init__(self, items, ns, nsv, seed, without=None):
        self.items, self.stages, self.without = items, {"k": ns, "v": nsv}, without
        self.rng = random.Random(seed)
        self.bars, self.inflight = {}, []
        self.ring = {"k": {}, "v": {}}   # stage -> tile that landed there
        self.q = {}                      # warp -> item whose rows it stored
        self.s, self.s_read = None, {}   # tile whose scores are there; tile -> warps that are through with them
        self.p = {}                      # (slot, warp) -> [tile, its P.V is done]
        self.pv_done, self.pv_flying = 0, 0
        self.o_read = {}                 # item -> warps that have read O

    def bar(self, *name):
        if name not in self.bars:
            self.bars[name] = Bar(WARPS if name[0] in ("s_free", "p_full", "q_full") else 1)
        return self.bars[name]

    def wait(self, what, phase, *name):
        """Waits on the barrier `name` for the end of `phase` as hardware does, by parity; `what` names the wait."""
        if what == self.without:
            return
        b = self.bar(*name)
        while b.done % 2 == phase % 2:
            yield
        self.need(b.done == phase + 1, f"{what}: waited for phase {phase} of {name}, passed at {b.done}")

    @staticmethod
    def need(holds, otherwise):
        if not holds:
            raise Violation(otherwise)

    def tiles(self):
        T = 0
        for j, n in enumerate(self.items):
            for i in range(n):
                yield T, j, i
                T += 1

    def producer(self):
        for T, _, _ in self.tiles():
            for r in "kv":
                st = T % self.stages[r]
                if T >= self.stages[r]:
                    yield from self.wait(r + "_empty", T // self.stages[r] - 1, r + "_empty", st)
                self.ring[r][st] = None

                def land(r=r, st=st, T=T):
                    self.ring[r][st] = T
                    self.bar(r + "_full", st).arrive()
                self.inflight.append((None, land))
                yield

    def s_issuer(self):
        for T, j, i in self.tiles():
            st = T % self.stages["k"]
            if i == 0:
                yield from self.wait("q_full", j, "q_full")
            yield from self.wait("k_full", T // self.stages["k"], "k_full", st)
            if T >= 1:
                yield from self.wait("s_free", T - 1, "s_free")

            def check(T=T, j=j, st=st):
                self.need(self.ring["k"].get(st) == T, f"S({T}) reads K of {self.ring['k'].get(st)}")
                self.need(all(self.q.get(w) == j for w in range(WARPS)), f"S({T}) of item {j} reads Q of {self.q}")
            check()
            self.need(T == 0 or self.s_read.get(T - 1) == WARPS, f"S({T}) written over scores not taken")
            self.s = None

            def done(T=T, st=st, check=check):
                check()
                self.s = T
                self.bar("s_full").arrive()
                self.bar("k_empty", st).arrive()
            self.inflight.append(("s", done))
            yield

    def pv_issuer(self):
        for T, j, i in self.tiles():
            st, slot = T % self.stages["v"], T & 1
            yield from self.wait("p_full", T >> 1, "p_full", slot)
            yield from self.wait("v_full", T // self.stages["v"], "v_full", st)
            self.need(i or not j or self.o_read.get(j - 1) == WARPS, f"P.V({T}) written over an O not read")

            def check(T=T, st=st, slot=slot):
                self.need(self.ring["v"].get(st) == T, f"P.V({T}) reads V of {self.ring['v'].get(st)}")
                self.need(all(self.p.get((slot, w), [None])[0] == T for w in range(WARPS)), f"P.V({T}) reads P of {self.p}")
            check()
            self.pv_flying += 1

            def done(slot=slot, st=st, check=check):
                check()
                self.pv_flying -= 1
                self.pv_done += 1
                for w in range(WARPS):
                    self.p[(slot, w)][1] = True
                self.bar("pv_done", slot).arrive()
                self.bar("v_empty", st).arrive()
            self.inflight.append(("pv", done))
            yield

    def softmax(self, w):
        self.q[w] = 0
        self.bar("q_full").arrive()
        yield
        for T, j, i in self.tiles():
            slot = T & 1
            yield from self.wait("s_full", T, "s_full")
            blank = self.rng.random() < 0.2  # no row of this warp sees the tile
            self.need(blank or self.s == T, f"warp {w} reads S of {self.s} for {T}")
            self.s_read[T] = self.s_read.get(T, 0) + 1
            self.bar("s_free").arrive()
            yield
            if T >= 2:
                yield from self.wait("p_slot", (T >> 1) - 1, "pv_done", slot)
                self.need(self.p[(slot, w)][1], f"warp {w} writes P of {T} over one not read")
            self.p[(slot, w)] = [T, False]
            yield
            if i and not blank and self.rng.random() < 0.3:  # the maximum moved
                yield from self.wait("rescale", (T - 1) >> 1, "pv_done", (T - 1) & 1)
                self.need(not self.pv_flying and self.pv_done == T, f"warp {w} rescales O before P.V({T - 1}) is done")
                yield
            self.bar("p_full", slot).arrive()
            yield
            if i + 1 < self.items[j]:
                continue
            if j + 1 < len(self.items):
                self.q[w] = j + 1
                self.bar("q_full").arrive()
                yield
            yield from self.wait("epilogue", T >> 1, "pv_done", slot)
            self.need(not self.pv_flying and self.pv_done == T + 1, f"warp {w} reads O before P.V({T}) is done")
            self.o_read[j] = self.o_read.get(j, 0) + 1
            yield

    def run(self):
        rng = self.rng
        live = [self.producer(), self.s_issuer(), self.pv_issuer()] + [self.softmax(w) for w in range(WARPS)]
        speed = {id(a): 10 ** rng.uniform(-2, 0) for a in live}
        rate = {None: 10 ** rng.uniform(-2, 0), "s": 10 ** rng.uniform(-2, 0), "pv": 10 ** rng.uniform(-2, 0)}
        for _ in range(200000):
            if not live and not self.inflight:
                return
            ready, seen = [], set()
            for at, (key, _cb) in enumerate(self.inflight):
                if key is None or key not in seen:
                    ready.append(at)
                    seen.add(key)
            choices = [(a, None) for a in live] + [(None, at) for at in ready]
            weights = [speed[id(a)] for a in live] + [rate[self.inflight[at][0]] for at in ready]
            actor, at = rng.choices(choices, weights)[0]
            if actor is None:
                self.inflight.pop(at)[1]()
                continue
            try:
                next(actor)
            except StopIteration:
                live.remove(actor)
        raise Violation("no progress: deadlock")


@pytest.mark.parametrize("items", [[1], [7], [1, 1, 1, 1], [3, 1, 2], [2, 2, 1], [5, 4, 1, 6]])
@pytest.mark.parametrize("ns,nsv", [(2, 3), (3, 3), (2, 2)])  # d = 128, 64, 256
def test_every_schedule_is_safe(items, ns, nsv):
    for seed in range(12):
        Model(items, ns, nsv, seed).run()


@pytest.mark.parametrize("without", WAITS)
@pytest.mark.parametrize("ns,nsv", [(2, 3), (3, 3), (2, 2)])
def test_each_wait_left_out_is_caught(without, ns, nsv):
    for seed in range(400):
        try:
            Model([5, 4, 1, 6], ns, nsv, seed, without).run()
        except Violation:
            return
    pytest.fail("no schedule shows it")
