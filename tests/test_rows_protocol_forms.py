"""The barrier protocol of rows_kernel in the forms that its sources have (csrc/apa_tree.cu, csrc/apa_cross.cu), with their
producers: the tree's pages, that go through a ring of their own to two warps for K and two for V, and the encoder's tiles,
both of whose copies one thread issues, and whose last one per sequence another warp clears behind the end (CPU; the core's
model is test_rows_protocol's, whose softmax groups and issuers are used here as they are).  Every wait of every form is left
out in turn."""
import os
import random
import re

import pytest

from mixed_precision_attention_gb300 import build

from .test_rows_protocol import Bar, Machine, _check_list, _segs

CORE = ["k", "v", "q", "s", "p", "pv", "rescale", "x", "xd", "qfree"]
BOTH = {"x", "xd", "qfree"}  # waits of two groups for one another


def _waits(NG, NB, own):
    return [w for w in CORE if (NG == 2 or w not in BOTH) and (NB == 2 or w != "rescale")] + own


class Halves(list):
    """A stage that several warps fill: it holds tile T when all of its parts do."""

    def __eq__(self, T):
        return all(x == T for x in self)

    __hash__ = None


def together(m, roles):
    """Several roles as one that the machine runs: a random one goes on each time, and copies land in any order."""
    m.flying = flying = []
    roles = list(roles)
    while roles or flying:
        if flying and (not roles or m.rng.random() < 0.4):
            m.land(flying.pop(m.rng.randrange(len(flying))))
        else:
            r = m.rng.choice(roles)
            if next(r, "end") == "end":
                roles.remove(r)
        yield


def both(rng, roles):
    while roles:
        r = rng.choice(roles)
        if next(r, "end") == "end":
            roles.remove(r)
        yield


class Tree(Machine):
    def __init__(self, segs, NG, NB, NK, NV, raw, rng, drop=None):
        super().__init__(segs, NG, NB, NK, NV, rng, drop)
        self.raw_full, self.raw_empty, self.raw = [Bar(1) for _ in range(raw)], [Bar(4) for _ in range(raw)], [None] * raw
        self.kf, self.vf = [Bar(2) for _ in range(NK)], [Bar(2) for _ in range(NV)]  # both warps of each
        self.bars += self.kf + self.vf + self.raw_full + self.raw_empty
        self.K, self.V = [Halves([None, None]) for _ in range(NK)], [Halves([None, None]) for _ in range(NV)]

    def tiles(self):
        return range(sum(t for t, _ in self.segs))

    def pages(self):
        n = len(self.raw)
        for T in self.tiles():
            if T >= n:
                yield from self.wait("raw_empty", self.raw_empty[T % n], (T // n + 1) & 1)
            self.raw[T % n] = None
            self.flying.append(T)
            yield

    def land(self, T):
        self.raw[T % len(self.raw)] = T
        self.raw_full[T % len(self.raw)].arrive()

    def decoder(self, full, empty, data, n, name, half):
        for T in self.tiles():
            raw = T % len(self.raw)
            yield from self.wait("raw_full", self.raw_full[raw], (T // len(self.raw)) & 1)
            if T >= n:
                yield from self.wait(name, empty[T % n], (T // n + 1) & 1)
            data[T % n][half] = None
            yield
            assert self.raw[raw] == T, "another tile's page is decoded"
            yield
            assert self.raw[raw] == T, "a page is written over while it is decoded"
            data[T % n][half] = T
            self.raw_empty[raw].arrive()
            full[T % n].arrive()
            yield

    def producer(self, full, empty, data, n, name):
        mine = [self.decoder(full, empty, data, n, name, h) for h in range(2)]
        return together(self, mine + [self.pages()]) if name == "k_empty" else both(self.rng, mine)


class Cross(Machine):
    """`ragged`: per segment, whether it ends with a tile whose values behind the end are to be cleared."""

    def __init__(self, segs, NG, NB, NK, NV, rng, drop=None):
        super().__init__(segs, NG, NB, NK, NV, rng, drop)
        self.landed = [Bar(1) for _ in range(NV)]
        self.bars += self.landed
        self.ragged = [rng.random() < 0.6 for _ in segs]

    def copies(self):
        """One thread issues K and V of each tile and, at the end, waits for all that is in flight."""
        NK, NV = self.NK, self.NV
        flying, T = self.flying, 0
        last, last_par = [False] * NV, [0] * NV
        for seg, (tiles, _) in enumerate(self.segs):
            for t in range(tiles):
                if T >= NK:
                    yield from self.wait("k_empty", self.ke[T % NK], (T // NK + 1) & 1)
                self.K[T % NK] = None
                flying.append(("K", T, self.kf[T % NK]))
                yield
                if T >= NV:
                    yield from self.wait("v_empty", self.ve[T % NV], (T // NV + 1) & 1)
                self.V[T % NV] = None
                fix = self.ragged[seg] and t == tiles - 1
                if last[T % NV]:
                    last_par[T % NV] ^= 1
                last[T % NV] = fix
                flying.append(("V", T, self.landed[T % NV] if fix else self.vf[T % NV]))
                T += 1
                yield
        # what it waits for at the end: the last copy into each stage.  It must not be past that already.
        ends = [(self.kf[x % NK], (x // NK) & 1, ("K", x)) for x in range(max(0, T - NK), T)]
        ends += [(self.landed[x % NV], last_par[x % NV], ("V", x)) if last[x % NV] else (self.vf[x % NV], (x // NV) & 1, ("V", x))
                 for x in range(max(0, T - NV), T)]
        for bar, par, copy in ends:
            while not bar.done(par):
                yield
            assert copy not in [f[:2] for f in flying], "a copy is in flight where the kernel thinks that all have landed"
        assert not flying

    def land(self, copy):
        kind, T, bar = copy
        if kind == "K":
            self.K[T % self.NK] = T
        else:
            self.V[T % self.NV] = ("as it came", T) if bar in self.landed else T
        bar.arrive()

    def clearer(self):
        T, par = 0, [0] * self.NV
        for seg, (tiles, _) in enumerate(self.segs):
            T += tiles
            if not self.ragged[seg]:
                continue
            st = (T - 1) % self.NV
            yield from self.wait("landed", self.landed[st], par[st])
            par[st] ^= 1
            assert self.V[st] == ("as it came", T - 1), "another tile is cleared"
            yield
            assert self.V[st] == ("as it came", T - 1)
            self.V[st] = T - 1
            self.vf[st].arrive()

    def producer(self, full, empty, data, n, name):
        return together(self, [self.copies()]) if name == "k_empty" else self.clearer()


# (form, NG, NB, NK, NV and, of trees, stages of pages)
FORMS = [(Tree, 1, 2, 3, 3, 8), (Tree, 2, 2, 2, 4, 4), (Tree, 1, 1, 2, 2, 3), (Tree, 1, 2, 2, 2, 4),
         (Cross, 1, 2, 5, 5), (Cross, 2, 2, 4, 4), (Cross, 1, 1, 2, 3), (Cross, 1, 2, 3, 3)]
OWN = {Tree: ["k_empty", "v_empty", "raw_full", "raw_empty"], Cross: ["k_empty", "v_empty", "landed"]}
# One buffer, K ring of 2, V ring of 3, one thread that issues K, then V of each tile: K of tile T waits for the scores of T - 2,
# and they come behind P V of T - 3, whose V is the one that T's goes over.  So that wait for V never waits.
IMPLIED = {((Cross, 1, 1, 2, 3), "v_empty")}
NAME = lambda f: f"{f[0].__name__}-{'-'.join(map(str, f[1:]))}"  # noqa: E731


def test_the_forms_are_the_kernels():
    """RowCfg<D, KT, NG, NB, QT, NK, NV, F16> of every pick, and the tree's stages of pages."""
    for kind, path in ((Tree, "apa_tree.cu"), (Cross, "apa_cross.cu")):
        with open(os.path.join(build.CSRC, path)) as f:
            text = f.read()
        found = set()
        for cfg, rest in re.findall(r"using Cfg = RowCfg<([^>]*)>;([^}]*)}", text):
            _, kt, ng, nb, _, nk, nv, _ = cfg.split(", ")
            raw = re.search(r"kRaw = (\d+)", rest)
            found.add((kind, int(ng), int(nb), int(nk), int(nv), *([int(raw.group(1))] if raw else [])))
            assert kt == "64"
        assert found == {f for f in FORMS if f[0] is kind}


@pytest.mark.parametrize("form", FORMS, ids=NAME)
def test_every_schedule_is_safe(form):
    for seed in range(80):
        rng = random.Random(seed)
        form[0](_segs(rng, form[1]), *form[1:], rng).run()


def test_the_implied_wait_is_not_missed():
    for form, drop in IMPLIED:
        for seed in range(150):
            rng = random.Random(seed)
            form[0](_segs(rng, form[1]), *form[1:], rng, drop=drop).run()


@pytest.mark.parametrize("form,drop", [(f, w) for f in FORMS for w in _waits(f[1], f[2], OWN[f[0]]) if (f, w) not in IMPLIED],
                         ids=lambda x: NAME(x) if isinstance(x, tuple) else x)
def test_each_wait_left_out_is_seen(form, drop):
    for seed in range(600):
        rng = random.Random(seed)
        try:
            form[0](_segs(rng, form[1]), *form[1:], rng, drop=drop).run()
        except AssertionError:
            return
    raise AssertionError(f"no schedule shows that the wait {drop} is needed")


# ------------------------------------------------------------------ the list, by the kernel's own rule
def _least(units, items):  # cut_ctas
    k = 1
    while k < 8 and 20 * k * k * items < units:
        k *= 2
    return k


@pytest.mark.parametrize("KB,grid,cost", [(1, 304, 7), (1, 152, 12), (2, 152, 20)])  # one block, d = 256, two blocks
def test_list_by_the_kernels_rule(KB, grid, cost):
    """Short lists, in which CTAs get the beginning of an item and no tile of it, and long ones."""
    with open(os.path.join(build.CSRC, "rows.cuh")) as f:
        text = f.read()
    assert "while (k < 8 && 20 * k * k * items < total) k *= 2;" in text
    assert "kItemCost = NG == 2 ? 20 : D == 256 ? 12 : 7;" in text
    rng = random.Random(KB + cost)
    lists = [([(1, 17)], 8), ([(2, 24)], 8), ([(1, 1)], 1), ([(3, 11)], 8), ([(1, 129)], 2), ([(0, 0), (1, 3), (0, 9), (5, 0)], 3)]
    lists += [([(rng.randint(0, 5), rng.choice([0, 1, 2, 9, 40])) for _ in range(rng.randint(1, 12))], rng.randint(1, 8))
              for _ in range(150)]
    idle = 0
    for seqs, H in lists:
        units = H * sum(b * t + cost * -(-b // KB) for b, t in seqs if b and t)
        if not units:
            continue
        least = _least(units, len(seqs) * H * max(b for b, _ in seqs))
        _check_list(seqs, H, KB, grid, least, cost)
        ctas = max(1, min(grid, -(-units // least)))
        idle += ctas > H * sum(b * t for b, t in seqs)
    assert idle > 5  # lists with CTAs that have nothing but beginnings
