"""Drafted trees over the 4-bit cache: masks and depths from parents, attention over them, and the accepted path's keys
moved, against plain implementations from the formulas in include/apa.h (attention in 64 bits; the tolerances are those
derived in test_gpu_cache.py: the numerics are the same)."""
import math

import numpy as np
import pytest

from .test_gpu_cache import _cache, _near, _torch, _types

pytestmark = pytest.mark.gpu


def _i32(a):
    return _torch(np.asarray(a, np.int32))


def _tree(parents, nodes):
    """(sees [B, Nq, Nq] bool, depths [B, Nq]) one ancestor at a time."""
    B, n = parents.shape
    sees, depths = np.zeros((B, n, n), bool), np.zeros((B, n), int)
    for b in range(B):
        for i in range(nodes[b]):
            at = i
            while at >= 0:
                sees[b, i, at] = True
                at = parents[b, at]
            depths[b, i] = sees[b, i].sum() - 1
    return sees, depths


def _words(sees):
    B, n, _ = sees.shape
    w = (n + 31) // 32
    bits = np.zeros((B, n, 32 * w), np.uint8)
    bits[:, :, :n] = sees
    return np.packbits(bits, axis=-1, bitorder="little").view(np.uint32).view(np.int32).reshape(B, n, w)


def _parents(rng, B, n, kind):
    p = np.full((B, n), -1)
    for i in range(1, n):
        p[:, i] = {"chain": i - 1, "star": 0, "roots": -1}.get(kind, 0)
        if kind == "tree":
            p[:, i] = rng.integers(max(-1, (i - 1) // 4 - 1), i, B)
    return p


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 100, 128, 250, 1000, 1024])
@pytest.mark.parametrize("kind", ["chain", "star", "roots", "tree"])
def test_draft_tree(n, kind):
    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(n)
    B = 5 if n < 300 else 2
    parents = _parents(rng, B, n, kind)
    nodes = rng.integers(0, n + 1, B)
    nodes[0] = n
    for given in (nodes, None):
        count = nodes if given is not None else np.full(B, n)
        sees, depths = _tree(parents, count)
        r = apa.draft_tree(_i32(parents), None if given is None else _i32(given))
        apa.check_error()
        assert np.array_equal(r["mask"].cpu().numpy(), _words(sees)) and np.array_equal(r["depths"].cpu().numpy(), depths)


def test_draft_tree_reports_what_is_no_tree():
    import mixed_precision_attention_gb300 as apa
    good = np.array([[-1, 0, 1, 1]])
    for bad, as_if in (([[-1, 1, 1, 1]], [[-1, -1, 1, 1]]), ([[-1, 0, 3, 1]], [[-1, 0, -1, 1]]),
                       ([[-2, 0, 1, 1]], good), ([[-1, 0, 1, 2 ** 30]], [[-1, 0, 1, -1]])):
        r = apa.draft_tree(_i32(bad))
        with pytest.raises(apa.ApaError):
            apa.check_error()
        assert np.array_equal(r["mask"].cpu().numpy(), _words(_tree(np.array(as_if), [4])[0]))
    for nodes, count in ((5, 4), (-1, 0)):
        r = apa.draft_tree(_i32(good), _i32([nodes]))
        with pytest.raises(apa.ApaError):
            apa.check_error()
        assert np.array_equal(r["mask"].cpu().numpy(), _words(_tree(good, [count])[0]))
    r = apa.draft_tree(_i32([[-1, 0, 9, 9]]), _i32([2]))  # rows from nodes on are not looked at
    apa.check_error()
    assert not r["mask"][0, 2:].any()


# ------------------------------------------------------------------ attention
def _attend(q, kv, lens, nodes, sees, depths, window, sinks):
    """64-bit attention, and sum_j w_j |v_j| of each output."""
    B, Hq, Nq, d = q.shape
    out, lse, mag = np.zeros(q.shape), np.full((B, Hq, Nq), -np.inf), np.zeros(q.shape)
    for b, n in enumerate(lens):
        k, v = kv[b]
        G, base = Hq // k.shape[0], n - nodes[b]
        pos = np.arange(n)
        pos[base:] = base + depths[b, :nodes[b]]
        for i in range(nodes[b]):
            vis = np.ones(n, bool)
            vis[base:] = sees[b, i, :nodes[b]]
            if window:
                vis &= (pos > base + depths[b, i] - window) | (pos < sinks)
            j = np.nonzero(vis)[0]
            if not len(j):
                continue
            for hq in range(Hq):
                s = k[hq // G][j] @ q[b, hq, i] / math.sqrt(d)
                m = s.max()
                w = np.exp(s - m)
                lse[b, hq, i] = m + np.log(w.sum())
                w /= w.sum()
                out[b, hq, i], mag[b, hq, i] = w @ v[hq // G][j], w @ np.abs(v[hq // G][j])
    return out, lse, mag


SHAPES = [  # B, Hq, Hkv, Nq, d, base, nodes, window, sinks, kind
    (1, 1, 1, 1, 64, [0], [1], 0, 0, "tree"),
    (1, 1, 1, 1, 128, [63], [1], 0, 0, "tree"),
    (2, 6, 2, 5, 128, [0, 17], [5, 0], 0, 0, "tree"),
    (4, 8, 2, 7, 64, [57, 64, 60, 1000], [7, 7, 6, 3], 0, 0, "tree"),   # trees that end with, and cross, a page
    (3, 8, 1, 33, 256, [31, 0, 700], [33, 20, 32], 0, 0, "tree"),
    (2, 5, 1, 64, 128, [0, 129], [64, 50], 0, 0, "chain"),
    (2, 8, 2, 70, 128, [300, 5], [70, 1], 0, 0, "star"),                # 280 rows: three blocks of one head
    (1, 24, 2, 40, 64, [777], [40], 0, 0, "tree"),
    (1, 4, 4, 130, 128, [100], [130], 0, 0, "tree"),                    # a tree over three pages
    (1, 2, 1, 100, 256, [333], [100], 0, 0, "roots"),
    (1, 40, 1, 9, 128, [4100], [9], 0, 0, "tree"),
    (2, 4, 2, 9, 64, [1000, 90], [9, 9], 1, 0, "tree"),                 # only itself
    (2, 4, 2, 20, 64, [1000, 90], [20, 18], 3, 2, "chain"),             # the window is shorter than the tree
    (2, 4, 2, 12, 128, [1000, 90], [12, 12], 32, 0, "tree"),
    (2, 4, 1, 15, 128, [1500, 3], [15, 9], 100, 4, "chain"),
    (3, 4, 1, 8, 128, [1500, 200, 50], [8, 8, 8], 129, 70, "tree"),
    (1, 6, 2, 30, 256, [900], [30], 200, 33, "tree"),
    (1, 2, 1, 11, 128, [640], [11], 5000, 3, "tree"),
    (1, 2, 1, 24, 64, [3000], [24], 7, 2999, "tree"),                   # the sinks reach into the window
    (1, 2, 1, 24, 64, [30], [24], 5, 40, "chain"),                      # and into the tree
    (200, 2, 1, 6, 64, None, None, 0, 0, "tree"),
]


def _case(rng, shape, dtype):
    B, Hq, H, Nq, d, base, nodes, window, sinks, kind = shape
    base = rng.integers(0, 150, B) if base is None else np.array(base)
    nodes = rng.integers(0, Nq + 1, B) if nodes is None else np.array(nodes)
    lens = base + nodes
    pages, table, ks, vs, kv = _cache(rng, B, H, d, lens, int(max(lens)) // 64 + 2)
    parents = _parents(rng, B, Nq, kind)
    q = _torch(rng.standard_normal((B, Nq, Hq, d)) * 2, _types()[dtype]).transpose(1, 2)
    return pages, table, ks, vs, kv, lens, nodes, parents, q


@pytest.mark.parametrize("case", range(len(SHAPES)))
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_attention_tree(case, dtype):
    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(case)
    pages, table, ks, vs, kv, lens, nodes, parents, q = _case(rng, SHAPES[case], dtype)
    window, sinks = SHAPES[case][7:9]
    sees, depths = _tree(parents, nodes)
    t = apa.draft_tree(_i32(parents), _i32(nodes))
    out, lse = apa.attention_tree(q, pages, table, _i32(lens), _i32(nodes), t["mask"], _torch(ks), _torch(vs),
                                  depths=t["depths"], window=window, sinks=sinks)
    apa.check_error()
    ref = _attend(q.double().cpu().numpy(), kv, lens, nodes, sees, depths, window, sinks)
    _near(out, lse, ref, dtype)


# ------------------------------------------------------------------ the accepted path
def _key_bytes(d):
    """Bytes of key i (of its 16-key block) in a head's block: [16, bytes of a key]."""
    i, n = np.arange(16)[:, None], d // 16
    t, g = np.arange(n)[None, :, None], np.arange(8)[None, None, :]
    v = 8 * d + 512 * (t // 4) + 16 * (4 * g + i[..., None] // 4) + 4 * (t % 4) + i[..., None] % 4
    s = np.arange(n)[None, :]
    return np.concatenate([i * (d // 2) + np.arange(d // 2)[None, :], v.reshape(16, -1), 16 * d + i * n + s,
                           17 * d + 4 * ((i // 4) * n + s) + i % 4], 1)


def _accept(pages, table, base, path, counts):
    """The definition: all of a sequence's keys read, then written."""
    at = _key_bytes(pages.shape[-1] // 72)
    d = pages.shape[-1] // 72
    pages = pages.copy()
    for b, c in enumerate(counts):
        place = lambda p: (table[b, p // 64], p % 64 // 16 * 18 * d + at[p % 16])  # noqa: E731
        keys = []
        for k in range(c):
            page, byte = place(base[b] + path[b, k])
            keys.append(pages[:, page, :, byte].copy())
        for k in range(c):
            page, byte = place(base[b] + k)
            pages[:, page, :, byte] = keys[k]
    return pages


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("layers,H,B,Nq,most", [(1, 1, 1, 1, 1), (1, 8, 5, 64, 9), (3, 2, 4, 130, 130), (2, 5, 30, 17, 17),
                                                (28, 3, 3, 40, 12)])
def test_cache_accept(d, layers, H, B, Nq, most):
    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(d + B)
    base = rng.integers(0, 200, B)
    nodes = rng.integers(1, Nq + 1, B)
    lens = base + nodes
    held = (lens + 63) // 64
    ids = rng.permutation(int(held.sum()) + 2)
    table, at = np.full((B, int(held.max()) + 1), -4), 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    counts = np.minimum(rng.integers(0, most + 1, B), nodes)
    counts[0] = min(most, nodes[0])
    path = np.full((B, most), -1)
    for b in range(B):
        path[b, :counts[b]] = np.sort(rng.choice(nodes[b], counts[b], replace=False))
    pages = rng.integers(0, 256, (layers, len(ids), H, 72 * d), dtype=np.uint8)
    want = _accept(pages, table, base, path, counts)
    p = _torch(pages)
    new = apa.cache_accept(p if layers > 1 else p[0], _i32(table), _i32(lens), _i32(nodes), _i32(path), _i32(counts))
    apa.check_error()
    assert np.array_equal(new.cpu().numpy(), base + counts)
    assert np.array_equal(p.cpu().numpy(), want)


def test_cache_accept_leaves_what_is_wrong():
    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(0)
    pages = rng.integers(0, 256, (5, 2, 72 * 64), dtype=np.uint8)
    table = np.array([[3, 1], [0, 4]])
    good = dict(lens=[100, 70], nodes=[20, 10], path=[[0, 5, 19], [0, 2, 9]], counts=[3, 2])
    for b, kw, base in ((0, dict(lens=[129, 70]), 128), (0, dict(lens=[-1, 70]), 0), (0, dict(nodes=[101, 10]), 100),
                        (0, dict(nodes=[-1, 10]), 100), (0, dict(counts=[4, 2]), 80), (0, dict(counts=[-1, 2]), 80),
                        (0, dict(path=[[0, 5, 5], [0, 2, 9]]), 80), (0, dict(path=[[0, 5, 20], [0, 2, 9]]), 80),
                        (0, dict(path=[[-1, 5, 9], [0, 2, 9]]), 80), (1, dict(nodes=[20, 1]), 69)):
        a = dict(good, **kw)
        p = _torch(pages)
        new = apa.cache_accept(p, _i32(table), *(_i32(a[k]) for k in ("lens", "nodes", "path", "counts")))
        with pytest.raises(apa.ApaError):
            apa.check_error()
        counts = [3, 2]
        counts[b] = 0
        want = _accept(pages[None], table, [80, 60], np.array(good["path"]), counts)[0]
        assert np.array_equal(p.cpu().numpy(), want)
        assert new.tolist() == [base if b == 0 else 83, 62 if b == 0 else base]
    # a page outside the pool: nothing moves from or to it
    good["counts"] = [3, 3]
    p = _torch(pages)
    new = apa.cache_accept(p, _i32([[3, 1], [0, 5]]), *(_i32(good[k]) for k in ("lens", "nodes", "path", "counts")))
    with pytest.raises(apa.ApaError):
        apa.check_error()
    assert new.tolist() == [83, 63]
    p2 = _torch(pages)
    apa.cache_accept(p2, _i32(table), *(_i32(good[k]) for k in ("lens", "nodes", "path", "counts")))
    apa.check_error()
    a, c = p.cpu().numpy(), p2.cpu().numpy()
    assert np.array_equal(a[[1, 3]], c[[1, 3]]) and np.array_equal(a[[2, 4]], pages[[2, 4]])
