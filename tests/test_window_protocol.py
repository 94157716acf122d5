"""The barrier protocol of the sliding-window kernel (window_kernel), run as a model under
random schedules on the CPU, as tests/test_pass2_protocol.py does for the pass-2 kernels.

A CTA takes several items (row blocks) in turn; T counts the tiles of all of them.  Actors:
the TMA producer (K, then V of each tile), the S issuer, the PV issuer and four softmax
warps.  Copies complete in any order, the products of one issuer in issue order.  Checked:
every wait passes on the phase it means; S reads its item's Q and its tile's K, and is
not written before all warps hold the scores of the tile before; P is not written over
one that its P.V has not read; P.V reads its tile's V and P and does not write an O that the
epilogue has yet to read; O is rescaled and read with no P.V in flight; every schedule ends.
A planted mistake (one wait left out) has to be caught by some schedule."""
import random

import pytest

WARPS = 4


class Violation(Exception):
    pass


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.done = count, 0, 0

    def arrive(self):
        self.pending += 1
        if self.pending == self.count:
            self.pending, self.done = 0, self.done + 1


def run(items, ns, nsv, seed, without=()):
    rng = random.Random(seed)
    per_warp = ("s_free", "p_full", "q_full")
    bars = {}

    def bar(*name):
        if name not in bars:
            bars[name] = Bar(WARPS if name[0] in per_warp else 1)
        return bars[name]

    def wait(phase, *name):
        if name[0] in without:
            return
        b = bar(*name)
        while b.done % 2 == phase % 2:  # hardware parity test
            yield
        if b.done != phase + 1:
            raise Violation(f"wait on {name} for phase {phase} passed at {b.done}")

    kst, vst, q = {}, {}, {}              # stage -> tile that landed; warp -> item whose Q rows are there
    score = [None]                        # tile whose S is in TMEM
    pbuf = {}                             # (slot, warp) -> [tile, read by its P.V]
    oread = {}                            # item -> warps whose epilogue has read O
    pv_running = [0]
    inflight = []

    def producer():
        T = 0
        for n in items:
            for _ in range(n):
                for ring, store, stages in (("k", kst, ns), ("v", vst, nsv)):
                    st = T % stages
                    if T >= stages:
                        yield from wait(T // stages - 1, ring + "_empty", st)
                    store[st] = None

                    def land(ring=ring, store=store, st=st, T=T):
                        store[st] = T
                        bar(ring + "_full", st).arrive()
                    inflight.append((None, land))
                    yield
                T += 1

    def s_issuer():
        T = 0
        for j, n in enumerate(items):
            yield from wait(j, "q_full")
            for _ in range(n):
                st = T % ns
                yield from wait(T // ns, "k_full", st)
                if T >= 1:
                    yield from wait(T - 1, "s_free")

                def check(T=T, st=st, j=j):
                    if kst.get(st) != T or any(q.get(w) != j for w in range(WARPS)):
                        raise Violation(f"S({T}) reads K of {kst.get(st)}, Q of {q}")
                check()
                score[0] = None  # being written

                def done(T=T, st=st, check=check):
                    check()
                    score[0] = T
                    bar("s_full").arrive()
                    bar("k_empty", st).arrive()
                inflight.append(("s", done))
                yield
                T += 1

    def pv_issuer():
        T = 0
        for j, n in enumerate(items):
            for i in range(n):
                st = T % nsv
                yield from wait(T >> 1, "p_full", T & 1)
                yield from wait(T // nsv, "v_full", st)
                if i == 0 and j and oread.get(j - 1, 0) != WARPS:
                    raise Violation(f"P.V({T}) writes O before it has been read")

                def check(T=T, st=st):
                    if vst.get(st) != T or any(pbuf.get((T & 1, w), [None])[0] != T for w in range(WARPS)):
                        raise Violation(f"P.V({T}) reads V of {vst.get(st)}, P of {pbuf}")
                check()
                pv_running[0] += 1

                def done(T=T, st=st, check=check):
                    check()
                    pv_running[0] -= 1
                    for w in range(WARPS):
                        pbuf[(T & 1, w)][1] = True
                    bar("pv_done", T & 1).arrive()
                    bar("v_empty", st).arrive()
                inflight.append(("pv", done))
                yield
                T += 1

    def softmax(w):
        T = 0
        q[w] = 0
        bar("q_full").arrive()
        yield
        for j, n in enumerate(items):
            for i in range(n):
                yield from wait(T, "s_full")
                if score[0] != T:
                    raise Violation(f"warp {w} reads S of {score[0]} for {T}")
                bar("s_free").arrive()
                yield
                if i and rng.random() < 0.2:  # the maximum moved: rescale O
                    yield from wait((T - 1) >> 1, "pv_done", (T - 1) & 1)
                    if pv_running[0]:
                        raise Violation(f"warp {w} rescales O with a P.V in flight")
                if T >= 2:
                    if "p_free" not in without:
                        yield from wait((T >> 1) - 1, "pv_done", T & 1)
                    if not pbuf[(T & 1, w)][1]:
                        raise Violation(f"warp {w} writes P of {T} over one not read")
                pbuf[(T & 1, w)] = [T, False]
                bar("p_full", T & 1).arrive()
                yield
                T += 1
            if j + 1 < len(items):
                q[w] = j + 1
                bar("q_full").arrive()
                yield
            yield from wait((T - 1) >> 1, "pv_done", (T - 1) & 1)
            if "pv_done" not in without and pv_running[0]:
                raise Violation(f"warp {w} reads O with a P.V in flight")
            oread[j] = oread.get(j, 0) + 1
            yield

    live = [producer(), s_issuer(), pv_issuer()] + [softmax(w) for w in range(WARPS)]
    speed = {id(a): 10 ** rng.uniform(-2, 0) for a in live}
    rate = {"copy": 10 ** rng.uniform(-2, 0), "mma": 10 ** rng.uniform(-2, 0)}
    for _ in range(200000):
        if not live and not inflight:
            return
        heads, seen = [], set()
        for k, (key, _cb) in enumerate(inflight):
            if key is None or key not in seen:
                heads.append(k)
                seen.add(key)
        choices = [("a", a) for a in live] + [("c", k) for k in heads]
        weights = [speed[id(a)] for a in live] + [rate["copy" if inflight[k][0] is None else "mma"] for k in heads]
        kind, what = rng.choices(choices, weights)[0]
        if kind == "c":
            inflight.pop(what)[1]()
            continue
        try:
            next(what)
        except StopIteration:
            live.remove(what)
    raise Violation("no progress: deadlock")


@pytest.mark.parametrize("items", [[1], [7], [1, 1, 1, 1], [3, 1, 2], [5, 4, 1, 6]])
@pytest.mark.parametrize("ns,nsv", [(2, 3), (3, 3), (2, 2)])  # d = 128, 64, 256
def test_every_schedule_is_safe(items, ns, nsv):
    for seed in range(8):
        run(items, ns, nsv, seed)


@pytest.mark.parametrize("without", ["s_free", "p_free", "q_full", "k_empty", "v_empty"])
def test_a_wait_left_out_is_caught(without):
    for seed in range(200):
        try:
            run([5, 4, 1, 6], 2, 3, seed, without=(without,))
        except (Violation, KeyError):
            return
    pytest.fail("no schedule shows it")
