"""The barrier protocol of rows_kernel (csrc/rows.cuh) and the cutting of its list of uses, as models in the
kernel's own order (CPU).

The protocol: one issuer, two groups of four softmax warps (one group at d = 256), producers of K and V, run as
coroutines under a random scheduler; products execute in the order of their issue, some time after it, and a commit
arrives when all before it are done.  Every value carries a tag (which use, tile or segment it belongs to), so a
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
    def __init__(self, segs, NG, NK, NV, rng, drop=None):
        """segs: (tiles, blocks of the item) of each segment."""
        self.segs, self.NG, self.NK, self.NV, self.rng, self.drop = segs, NG, NK, NV, rng, drop
        W = self.W = 4 * NG
        self.kf, self.ke = [Bar(1) for _ in range(NK)], [Bar(1) for _ in range(NK)]
        self.vf, self.ve = [Bar(1) for _ in range(NV)], [Bar(1) for _ in range(NV)]
        self.s, self.p, self.pv = [Bar(1), Bar(1)], [Bar(4), Bar(4)], [Bar(1), Bar(1)]
        self.q, self.x, self.xd = Bar(W), Bar(W), Bar(W)
        self.K, self.V = [None] * NK, [None] * NV
        self.S = [None, None]                       # use whose scores are there
        self.P = [[None] * 4, [None] * 4]           # per warp of a group: use
        self.Q = [[None] * W, [None] * W]           # per block: the segment that each warp stored
        self.O = [[], []]                           # per group: the uses summed up in it
        self.queue = []                             # products and commits in flight
        self.seen = []                              # what the epilogues read

    # ---- products, executed in order
    def execute(self):
        kind, *a = self.queue.pop(0)
        if kind == "commit":
            a[0].arrive()
        elif kind == "S":
            use, T, seg, blk, warps = a
            assert self.K[T % self.NK] == T, "S reads another tile's K"
            for w in warps:
                assert self.Q[blk][w] == seg, "S reads another segment's Q"
            self.S[use & 1] = use
            self.P[use & 1] = [None] * 4            # they share columns
        else:
            use, T, g, first = a
            assert self.P[use & 1] == [use] * 4, "P V reads another use's P"
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

    def issuer(self):
        segs, NG = self.segs, self.NG
        st = dict(su=0, sT=0, si=0, sj=0, sn=0, fresh=True)

        def issue_s():
            tiles, w = segs[st["sn"]]
            if st["fresh"]:
                yield from self.wait("q", self.q, st["sn"] & 1)
                st["fresh"] = False
            if st["sj"] == 0:
                yield from self.wait("k", self.kf[st["sT"] % self.NK], (st["sT"] // self.NK) & 1)
            # the warps that store the block's rows: of the group whose uses it is, or (one block) all
            warps = range(self.W) if w == 1 else range(4 * (st["su"] & 1), 4 * (st["su"] & 1) + 4)
            self.queue.append(("S", st["su"], st["sT"], st["sn"], st["sj"], warps))
            self.queue.append(("commit", self.s[st["su"] & 1]))
            st["su"] += 1
            st["sj"] += 1
            if st["sj"] == w:
                self.queue.append(("commit", self.ke[st["sT"] % self.NK]))
                st["sj"] = 0
                st["sT"] += 1
                st["si"] += 1
                if st["si"] == tiles:
                    st["si"], st["fresh"] = 0, True
                    st["sn"] += 1

        u = T = 0
        for n, (tiles, w) in enumerate(segs):
            uses = tiles * w
            while st["sn"] == n and st["su"] < u + 2:
                yield from issue_s()
            for i in range(uses):
                yield from self.wait("p", self.p[u & 1], (u >> 1) & 1)
                if w == 1 or not i & 1:
                    yield from self.wait("v", self.vf[T % self.NV], (T // self.NV) & 1)
                self.queue.append(("PV", u, T, (u & 1) if NG == 2 else 0, i < NG))
                self.queue.append(("commit", self.pv[u & 1]))
                if w == 1 or i & 1:
                    self.queue.append(("commit", self.ve[T % self.NV]))
                    T += 1
                upto = n + 1 if i + 1 == uses else n
                while st["sn"] < len(segs) and st["sn"] <= upto and st["su"] <= u + 2:
                    yield from issue_s()
                u += 1

    def softmax(self, warp):
        segs, NG = self.segs, self.NG
        g, wi = warp >> 2, warp & 3

        def put_q(n, u0):
            w = segs[n][1]
            self.Q[(g ^ u0) & 1 if w == 2 else 0][warp] = n
            yield
            self.q.arrive()

        u = nx = 0
        yield from put_q(0, 0)
        for n, (tiles, w) in enumerate(segs):
            uses = tiles * w
            mine, began = [], False
            for i in range((g ^ (u & 1)) if NG == 2 else 0, uses, NG):
                use = u + i
                buf = use & 1
                yield from self.wait("s", self.s[buf], (use >> 1) & 1)
                assert self.S[buf] == use, "softmax reads another use's scores"
                if self.rng.random() < 0.3 and began:  # O is scaled
                    if NG == 1:
                        yield from self.wait("rescale", self.pv[(use - 1) & 1], ((use - 1) >> 1) & 1)
                    assert self.O[g] == mine, "O is scaled before its last product"
                    yield
                    assert self.O[g] == mine, "O changes while it is scaled"
                began = True
                yield
                assert self.S[buf] == use
                self.P[buf][wi] = use
                mine.append(use)
                self.p[buf].arrive()
            end = u + uses
            last = [end - 1 if (end - 1) & 1 == k else end - 2 for k in range(2)]
            have = [x >= u for x in last]
            for k in range(2):
                if have[k]:
                    yield from self.wait("s_end", self.s[k], (last[k] >> 1) & 1)
            if n + 1 < len(segs):
                yield from put_q(n + 1, end)
            joint = NG == 2 and w == 1
            if joint:
                self.x.arrive()
                yield from self.wait("x", self.x, nx & 1)
            for k in range(2):
                if have[k] and (joint or NG == 1 or k == g):
                    yield from self.wait("pv", self.pv[k], (last[k] >> 1) & 1)
            if joint:
                for h in range(2):
                    if have[h]:
                        want = [x for x in range(u, end) if x & 1 == h]
                        assert self.O[h] == want, "the epilogue reads O too early or too late"
                        yield
                        assert self.O[h] == want
                self.xd.arrive()
                yield from self.wait("xd", self.xd, nx & 1)
                nx += 1
            else:
                assert self.O[g] == mine, "the epilogue reads O too early or too late"
                yield
                assert self.O[g] == mine
            self.seen.append((n, warp, tuple(mine)))
            u = end

    def run(self):
        roles = [self.issuer(), self.producer(self.kf, self.ke, self.K, self.NK, "k_empty"),
                 self.producer(self.vf, self.ve, self.V, self.NV, "v_empty")]
        roles += [self.softmax(w) for w in range(self.W)]
        pace = {r: self.rng.choice([0.05, 0.6, 0.9]) for r in roles}
        idle = 0
        while roles or self.queue:
            state = (sum(b.phase for b in [*self.kf, *self.ke, *self.vf, *self.ve, *self.s, *self.p, *self.pv, self.q,
                                           self.x, self.xd]), len(roles), len(self.queue))
            for r in self.rng.sample(roles, len(roles)):
                if self.rng.random() < pace[r]:
                    if next(r, "end") == "end":
                        roles.remove(r)
            while self.queue and self.rng.random() < 0.5:
                self.execute()
            now = (sum(b.phase for b in [*self.kf, *self.ke, *self.vf, *self.ve, *self.s, *self.p, *self.pv, self.q, self.x,
                                         self.xd]), len(roles), len(self.queue))
            idle = idle + 1 if now == state else 0
            assert idle < 400, "deadlock"
        total = sum(t * w for t, w in self.segs)
        done = [x for _, w, m in self.seen if w % 4 == 0 for x in m]
        assert sorted(done) == list(range(total))


def _segs(rng, NG):
    return [(rng.choice([1, 1, 2, 3, 4, 7]), rng.randint(1, 2) if NG == 2 else 1) for _ in range(rng.randint(1, 7))]


@pytest.mark.parametrize("NG", [1, 2])
@pytest.mark.parametrize("rings", [(2, 2), (3, 2), (5, 5)])
def test_protocol_keeps_every_value_for_its_reader(NG, rings):
    for seed in range(120):
        rng = random.Random(1000 * NG + seed)
        Machine(_segs(rng, NG), NG, *rings, rng).run()


@pytest.mark.parametrize("drop", ["k", "v", "q", "s", "p", "k_empty", "v_empty", "pv", "xd", "s_end", "rescale"])
def test_protocol_model_sees_a_wait_left_out(drop):
    """Without one of the waits some schedule goes wrong: the model can tell."""
    for seed in range(400):
        NG = 1 if drop == "rescale" else 2
        rng = random.Random(seed)
        try:
            Machine(_segs(rng, NG), NG, 2, 2, rng, drop=drop).run()
        except AssertionError:
            return
    raise AssertionError(f"no schedule shows that the wait {drop} is needed")


# ------------------------------------------------------------------ the list
def _first(n, k):
    q, r = divmod(n, k)
    return lambda i: n if i >= k else q * i + min(i, r)


def _check_list(seqs, H, KB, grid, least=4):
    """seqs: (blocks, tiles) of each sequence.  Every (sequence, head, block, tile) falls to one CTA once, a CTA
    keeps at most one part of an item that ends in it and one of an item that goes on, and the joining finds them all."""
    uses = [b * t for b, t in seqs]
    total = sum(uses) * H
    f = _first(total, max(1, min(grid, -(-total // least))))

    def place(x):
        before = 0
        for b, u in enumerate(uses):
            if u and before * H <= x < (before + u) * H:
                break
            before += u
        blocks, tiles = seqs[b]
        h, z = divmod(x - before * H, u)
        k = z // (KB * tiles)
        return b, h * -(-blocks // KB) + k, z - k * KB * tiles

    def item_of(b, item):
        blocks = seqs[b][0]
        per = -(-blocks // KB)
        return item // per, item % per * KB, min(KB, blocks - item % per * KB), per

    seen, parts, recs = set(), {}, []
    for c in range(grid):
        x0, x1, rec, slots = f(c), f(c + 1), None, []
        if x1 > x0:
            b, item, pos = place(x1 - 1)
            h, rb, w, _ = item_of(b, item)
            if x1 - 1 - pos >= x0 and x1 - 1 - pos + seqs[b][1] * w > x1:
                rec = (x1 - 1 - pos, b, h, rb, seqs[b][1], w)
            b, item, pos = place(x0)
            left = x1 - x0
            while left > 0:
                h, rb, w, per = item_of(b, item)
                if pos == seqs[b][1] * w:
                    pos, item = 0, item + 1
                    if item == per * H:
                        item, b = 0, next(i for i in range(b + 1, len(seqs)) if uses[i])
                    h, rb, w, per = item_of(b, item)
                n = seqs[b][1]
                end = min(n * w, pos + left)
                t0, t1, left, pos = pos // w, end // w, left - (end - pos), end
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
            if f(d) >= first + n * w:
                break
            got.append((d, max(0, min(f(d) - first, n * w)) // w, min(f(d + 1) - first, n * w) // w))
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
        _check_list(seqs, rng.randint(1, 3), rng.choice([1, 2]), rng.choice([1, 2, 5, 16, 152]))
