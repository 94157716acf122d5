"""The barrier protocol of rows_kernel (csrc/rows.cuh) and the cutting of its list of uses, as models in the
kernel's own order (CPU).

The protocol: groups of four softmax warps with an issuer each (two groups for items of two blocks, else one) and
producers of K and V, run as coroutines under a random scheduler; an issuer's products execute in the order of their
issue, some time after it, and a commit arrives when all before it are done.  Every value carries a tag (which use, tile or segment it belongs to), so a
missing wait shows as a wrong tag, a surplus one as a deadlock."""
import random

import pytest


class Bar:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        assert self.left >= 0
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def done(self, parity):  # mbarrier.test_wait.parity
        return (self.phase & 1) != parity


class Machine:
    def __init__(self, segs, NG, NB, NK, NV, rng, drop=None):
        """segs: (tiles, blocks of the item) of each segment."""
        self.segs, self.NG, self.NB, self.NK, self.NV, self.rng, self.drop = segs, NG, NB, NK, NV, rng, drop
        W = self.W = 4 * NG
        self.kf, self.ke = [Bar(1) for _ in range(NK)], [Bar(NG) for _ in range(NK)]
        self.vf, self.ve = [Bar(1) for _ in range(NV)], [Bar(NG) for _ in range(NV)]
        self.s, self.p = ([[Bar(c) for _ in range(NB)] for _ in range(NG)] for c in (1, 4))
        self.pv, self.pv2 = [Bar(1) for _ in range(NG)], [Bar(1) for _ in range(NG)]
        self.q, self.qfree, self.x, self.xd = Bar(W), Bar(2 * NG), Bar(W), Bar(W)
        self.bars = [*self.kf, *self.ke, *self.vf, *self.ve, *sum(self.s, []), *sum(self.p, []), *self.pv, *self.pv2, self.q,
                     self.qfree, self.x, self.xd]
        self.K, self.V = [None] * NK, [None] * NV
        self.S = [[None] * NB for _ in range(NG)]               # the group's use whose scores are there
        self.P = [[[None] * 4 for _ in range(NB)] for _ in range(NG)]  # per warp of a group: use
        self.Q = [[None] * W, [None] * W]                       # per block: the segment that each warp stored
        self.O = [[] for _ in range(NG)]                        # per group: the uses summed up in it
        self.queue = [[] for _ in range(NG)]                    # products and commits in flight, per issuer
        self.X = [[None] * 4, [None] * 4]
        self.seen = []                                          # what the epilogues read

    def share(self, w, tiles, g, T):
        return range((g ^ T) & 1, tiles, 2) if self.NG == 2 and w == 1 else range(tiles)

    # ---- an issuer's products, executed in its order
    def execute(self, g):
        kind, *a = self.queue[g].pop(0)
        if kind == "commit":
            a[0].arrive()
        elif kind == "S":
            use, T, seg, blk, warps = a
            assert self.K[T % self.NK] == T, "S reads another tile's K"
            for w in warps:
                assert self.Q[blk][w] == seg, "S reads another segment's Q"
            self.S[g][use % self.NB] = use
            self.P[g][use % self.NB] = [None] * 4               # they share columns
        else:
            use, T, first = a
            assert self.P[g][use % self.NB] == [use] * 4, "P V reads another use's P"
            assert self.V[T % self.NV] == T, "P V reads another tile's V"
            self.O[g] = [use] if first else self.O[g] + [use]

    def wait(self, name, bar, parity):
        if self.drop == name:
            yield
            return
        while not bar.done(parity):
            yield

    # ---- roles
    def producer(self, full, empty, data, n, name):
        T = 0
        for tiles, _ in self.segs:
            for _ in range(tiles):
                if T >= n:
                    yield from self.wait(name, empty[T % n], (T // n + 1) & 1)
                data[T % n] = None
                yield
                data[T % n] = T
                full[T % n].arrive()
                T += 1

    def issuer(self, g):
        NB = self.NB
        n = T = 0
        for seg, (tiles, w) in enumerate(self.segs):
            mine = self.share(w, tiles, g, T)
            yield from self.wait("q", self.q, seg & 1)
            if self.NG == 2:
                self.qfree.arrive()
            count = 2 if self.NG == 2 and w == 1 else 1
            # the warps that store a block's rows: of the group whose uses it is, or (one block) all
            warps = range(self.W) if w == 1 else range(4 * g, 4 * g + 4)
            for i in range(-NB, len(mine)):
                j = i + NB
                buf = (n + j) % NB
                if i >= 0:
                    t = T + mine[i]
                    yield from self.wait("p", self.p[g][buf], ((n + i) // NB) & 1)
                    yield from self.wait("v", self.vf[t % self.NV], (t // self.NV) & 1)
                    self.queue[g].append(("PV", n + i, t, i == 0))
                    if j >= len(mine):
                        self.queue[g].append(("commit", (self.pv if i + 1 == len(mine) else self.pv2)[g]))
                if j < len(mine):
                    t = T + mine[j]
                    yield from self.wait("k", self.kf[t % self.NK], (t // self.NK) & 1)
                    self.queue[g].append(("S", n + j, t, seg, g if w == 2 else 0, warps))
                    self.queue[g].append(("commit", self.s[g][buf]))
                if NB == 2:  # (with one buffer the softmax group hands the stages back)
                    if i >= 0:
                        self.queue[g] += [("commit", self.ve[(T + mine[i]) % self.NV])] * count
                    if j < len(mine):
                        self.queue[g] += [("commit", self.ke[(T + mine[j]) % self.NK])] * count
            T += tiles
            n += len(mine)

    def softmax(self, warp):
        segs, NG, NB = self.segs, self.NG, self.NB
        g, wi = warp >> 2, warp & 3

        def put_q(seg):
            self.Q[g if segs[seg][1] == 2 else 0][warp] = seg
            yield
            self.q.arrive()

        def hand(bar, w):
            for _ in range(2 if NG == 2 and w == 1 else 1):
                bar.arrive()

        T = nx = npv2 = 0
        n, npv = [0] * NG, [0] * NG
        yield from put_q(0)
        for seg, (tiles, w) in enumerate(segs):
            share = self.share(w, tiles, g, T)
            joint = NG == 2 and w == 1
            mine = []
            for i, t in enumerate(share):
                v = n[g] + i
                buf = v % NB
                yield from self.wait("s", self.s[g][buf], (v // NB) & 1)
                assert self.S[g][buf] == v, "softmax reads another use's scores"
                if NB == 1 and wi == 0:
                    hand(self.ke[(T + t) % self.NK], w)
                    if i:
                        hand(self.ve[(T + share[i - 1]) % self.NV], w)
                if self.rng.random() < 0.3 and i:  # O is scaled
                    if NB == 2 and i + 1 < len(share):
                        yield from self.wait("rescale", self.s[g][buf ^ 1], ((v + 1) // NB) & 1)
                    elif NB == 2:
                        yield from self.wait("rescale", self.pv2[g], npv2 & 1)
                    assert self.O[g] == mine, "O is scaled before its last product"
                    yield
                    assert self.O[g] == mine, "O changes while it is scaled"
                yield
                assert self.S[g][buf] == v
                self.P[g][buf][wi] = v
                mine.append(v)
                self.p[g][buf].arrive()
            if NG == 2:
                if wi == 0:
                    self.qfree.arrive()
                yield from self.wait("qfree", self.qfree, seg & 1)
            if seg + 1 < len(segs):
                yield from put_q(seg + 1)
            if joint:
                self.X[g][wi] = seg
                self.x.arrive()
                yield from self.wait("x", self.x, nx & 1)
                assert self.X[g ^ 1][wi] == seg, "the other group's sums are of another segment"
            want = [list(range(n[k], n[k] + len(self.share(w, tiles, k, T)))) for k in range(NG)]
            for k in range(NG):
                if want[k] and (joint or k == g):
                    yield from self.wait("pv", self.pv[k], npv[k] & 1)
                npv[k] += len(want[k]) > 0
                n[k] += len(want[k])
            npv2 += NB == 2 and len(share) > 1
            if NB == 1 and wi == 0 and len(share):
                hand(self.ve[(T + share[-1]) % self.NV], w)
            reads = [k for k in range(NG) if want[k] and (joint or k == g)]
            for _ in range(2):
                for k in reads:
                    assert self.O[k] == want[k], "the epilogue reads O too early or too late"
                yield
            if joint:
                self.xd.arrive()
                yield from self.wait("xd", self.xd, nx & 1)
                nx += 1
            self.seen.append((seg, warp, tuple(mine)))
            T += tiles

    def run(self):
        roles = [self.producer(self.kf, self.ke, self.K, self.NK, "k_empty"),
                 self.producer(self.vf, self.ve, self.V, self.NV, "v_empty")]
        roles += [self.issuer(g) for g in range(self.NG)]
        roles += [self.softmax(w) for w in range(self.W)]
        pace = {r: self.rng.choice([0.05, 0.6, 0.9]) for r in roles}
        drain = [self.rng.choice([0.1, 0.5, 0.9]) for _ in self.queue]
        state = lambda: (sum(b.phase for b in self.bars), len(roles), sum(map(len, self.queue)))  # noqa: E731
        idle = 0
        while roles or any(self.queue):
            before = state()
            for r in self.rng.sample(roles, len(roles)):
                if self.rng.random() < pace[r]:
                    if next(r, "end") == "end":
                        roles.remove(r)
            for g, q in enumerate(self.queue):
                while q and self.rng.random() < drain[g]:
                    self.execute(g)
            idle = idle + 1 if state() == before else 0
            assert idle < 1000, "deadlock"
        for g in range(self.NG):
            done = [x for _, w, m in self.seen if w == 4 * g for x in m]
            before = [sum(t for t, _ in self.segs[:i]) for i in range(len(self.segs))]
            assert done == list(range(sum(len(self.share(w, t, g, T)) for (t, w), T in zip(self.segs, before))))


def _segs(rng, NG):
    return [(rng.choice([1, 1, 2, 3, 4, 7]), rng.randint(1, 2) if NG == 2 else 1) for _ in range(rng.randint(1, 7))]


# (two groups need rings of an even length, two buffers of S a second stage of V)
@pytest.mark.parametrize("NG,NB,NK,NV", [(1, 1, 2, 3), (1, 1, 2, 2), (1, 2, 2, 2), (1, 2, 3, 3), (1, 2, 5, 5), (2, 1, 2, 2),
                                         (2, 1, 4, 4), (2, 2, 2, 4), (2, 2, 4, 4), (2, 2, 8, 8)])
def test_protocol_keeps_every_value_for_its_reader(NG, NB, NK, NV):
    for seed in range(120):
        rng = random.Random(1000 * NG + seed)
        Machine(_segs(rng, NG), NG, NB, NK, NV, rng).run()


WAITS = ["k", "v", "q", "s", "p", "k_empty", "v_empty", "pv", "x", "xd", "qfree"]


@pytest.mark.parametrize("NB,drop", [(1, w) for w in WAITS] + [(2, w) for w in WAITS + ["rescale"]])
def test_protocol_model_sees_a_wait_left_out(drop, NB):
    """Without one of the waits some schedule goes wrong: the model can tell."""
    for seed in range(600):
        rng = random.Random(seed)
        try:
            Machine(_segs(rng, 2), 2, NB, 4, 4, rng, drop=drop).run()
        except AssertionError:
            return
    raise AssertionError(f"no schedule shows that the wait {drop} is needed")


# ------------------------------------------------------------------ the list
def _first(n, k):
    q, r = divmod(n, k)
    return lambda i: n if i >= k else q * i + min(i, r)


def _check_list(seqs, H, KB, grid, least, E):
    """seqs: (blocks, tiles) of each sequence; E: units that beginning an item counts as.  Every (sequence, head, block,
    tile) falls to one CTA once, a CTA keeps at most one part of an item that ends in it and one of an item that goes on,
    and the joining finds them all."""
    per_of = lambda blocks: -(-blocks // KB)  # noqa: E731
    cost = [b * t + E * per_of(b) if b and t else 0 for b, t in seqs]
    total = sum(cost) * H
    f = _first(total, max(1, min(grid, -(-total // least))))

    def place(x):
        before = 0
        for b, u in enumerate(cost):
            if u and before * H <= x < (before + u) * H:
                break
            before += u
        blocks, tiles = seqs[b]
        h, z = divmod(x - before * H, u)
        k = z // (KB * tiles + E)
        return b, h * per_of(blocks) + k, z - k * (KB * tiles + E)

    def item_of(b, item):
        per = per_of(seqs[b][0])
        return item // per, item % per * KB, min(KB, seqs[b][0] - item % per * KB), per

    seen, parts, recs = set(), {}, []
    for c in range(grid):
        x0, x1, rec, slots = f(c), f(c + 1), None, []
        if x1 > x0:
            b, item, pos = place(x1 - 1)
            h, rb, w, _ = item_of(b, item)
            if x1 - 1 - pos >= x0 and x1 - 1 - pos + E + seqs[b][1] * w > x1:
                rec = (x1 - 1 - pos, b, h, rb, seqs[b][1], w)
            b, item, pos = place(x0)
            left = x1 - x0
            while left > 0:
                h, rb, w, per = item_of(b, item)
                if pos == E + seqs[b][1] * w:
                    pos, item = 0, item + 1
                    if item == per * H:
                        item, b = 0, next(i for i in range(b + 1, len(seqs)) if cost[i])
                    h, rb, w, per = item_of(b, item)
                n = seqs[b][1]
                end = min(E + n * w, pos + left)
                t0, t1, left, pos = max(0, pos - E) // w, max(0, end - E) // w, left - (end - pos), end
                for t in range(t0, t1):
                    for k in range(w):
                        assert (b, h, rb + k, t) not in seen
                        seen.add((b, h, rb + k, t))
                if t1 > t0 and (t0, t1) != (0, n):
                    slots.append(t1 == n)
                    parts[c, b, h, rb] = (t0, t1)
        assert len(set(slots)) == len(slots)
        recs.append(rec)
    assert seen == {(b, h, r, t) for b, (bl, ti) in enumerate(seqs) for h in range(H) for r in range(bl) for t in range(ti)}
    for c, rec in enumerate(recs):
        if rec is None:
            continue
        first, b, h, rb, n, w = rec
        got = []
        for d in range(c, grid):
            if f(d) >= first + E + n * w:
                break
            got.append((d, *(max(0, min(x - first - E, n * w)) // w for x in (f(d), f(d + 1)))))
        if any((t0, t1) == (0, n) for _, t0, t1 in got):
            continue
        for d, t0, t1 in got:
            if t1 > t0:
                assert parts.pop((d, b, h, rb)) == (t0, t1)
    assert not parts


def test_list_is_cut_without_gaps_and_joined_whole():
    rng = random.Random(5)
    for _ in range(1500):
        seqs = [(rng.choice([0, 1, 2, 3, 5]), rng.choice([0, 1, 2, 7, 30])) for _ in range(rng.randint(1, 6))]
        _check_list(seqs, rng.randint(1, 3), rng.choice([1, 2]), rng.choice([1, 2, 5, 16, 152, 304]), rng.choice([1, 2, 4, 8]),
                    rng.choice([0, 1, 7, 20]))
