"""Cases, plain forms and 64-bit values of the operators that check drafted trees and read an encoder:

* draft_tree        which drafted tokens each one sees, as bits, and their depths, from their parents
* attention_tree    attention of a tree of drafted tokens over the 4-bit paged K/V cache
* cache_accept      the keys of the accepted path moved behind the context
* attention_cross   attention to an encoder's states, of a length of its own for each sequence

A drafted token (node) of sequence b has its key in the cache at base + node, base = lens[b] - nodes[b]; its parent is
a node before it, or -1: the context.  A node sees the context, its ancestors and itself.  Positions are depths: node i
stands at base + depth(i), and a window leaves the keys whose position is above position - window, or below sinks.

The cache is a pool uint8 [num_pages, Hkv, 72 d]: a page holds 64 keys of all KV heads, as four blocks of 16 keys of
18 d bytes each:

  K codes   8 d bytes   key i, byte x: the E2M1 codes of channels 2x (low nibble), 2x + 1
  V codes   8 d bytes   key i, channels 16 t + g (low nibble) and 16 t + 8 + g, g < 8, at byte
                        512 (t / 4) + 16 (4 g + i / 4) + 4 (t % 4) + i % 4
  K scales    d bytes   UE4M3, key i, channels 16 t .. 16 t + 15 at byte i d / 16 + t
  V scales    d bytes   UE4M3, key i, channels 16 t .. 16 t + 15 at byte 4 ((i / 4) d / 16 + t) + i % 4

A value is E2M1 * UE4M3 * the FP32 scale of its KV head.
"""
import math

import numpy as np
import torch

own = False

TILE = 64  # keys in a page
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of E2M1


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the trees of one step of a batch, as every layer's attention then reads them
        {"name": "plan step", "op": "plan", "B": 64, "Nq": 64},
        # large trees of a large batch
        {"name": "plan wide", "op": "plan", "B": 256, "Nq": 250},
        # one conversation, a small tree: latency
        {"name": "tree single", "op": "tree", "B": 1, "Hq": 24, "Hkv": 8, "Nq": 26, "d": 128, "longest": 1000,
         "window": 0, "sinks": 0, "dtype": "bfloat16"},
        # a batch of conversations of many lengths, trees of many sizes
        {"name": "tree batch", "op": "tree", "B": 32, "Hq": 24, "Hkv": 8, "Nq": 32, "d": 128, "longest": 8192,
         "window": 0, "sinks": 0, "dtype": "bfloat16"},
        # long contexts, large trees
        {"name": "tree long", "op": "tree", "B": 4, "Hq": 32, "Hkv": 8, "Nq": 64, "d": 128, "longest": 131072,
         "window": 0, "sinks": 0, "dtype": "bfloat16"},
        # under a sliding window with sinks
        {"name": "tree window", "op": "tree", "B": 24, "Hq": 16, "Hkv": 4, "Nq": 48, "d": 64, "longest": 32768,
         "window": 4096, "sinks": 4, "dtype": "float16"},
        # what a step of a batch accepts, in one layer's pool
        {"name": "accept step", "op": "accept", "B": 64, "Hkv": 8, "Nq": 64, "d": 128, "longest": 2000, "most": 8, "layers": 1},
        # the same in the pools of all layers of a model at once
        {"name": "accept layers", "op": "accept", "B": 32, "Hkv": 8, "Nq": 64, "d": 128, "longest": 300, "most": 8, "layers": 28},
        # a decoding step: one row of each sequence over its encoder's states
        {"name": "cross step", "op": "cross", "B": 64, "Hq": 24, "Hkv": 8, "Nq": 1, "Nkv": 4096, "d": 128, "dtype": "bfloat16"},
        # the drafted rows of a small batch, short inputs
        {"name": "cross rows", "op": "cross", "B": 12, "Hq": 16, "Hkv": 4, "Nq": 48, "Nkv": 1500, "d": 64, "dtype": "float16"},
        # odd sizes, wide heads
        {"name": "cross odd", "op": "cross", "B": 8, "Hq": 6, "Hkv": 2, "Nq": 333, "Nkv": 1021, "d": 256, "dtype": "bfloat16"},
        # prompts of the decoder over long inputs
        {"name": "cross prompt", "op": "cross", "B": 4, "Hq": 24, "Hkv": 8, "Nq": 2048, "Nkv": 8192, "d": 128, "dtype": "bfloat16"},
    ]


def _log(rng, lo, hi):
    """A whole number, uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "tree", "tree", "tree", "accept", "cross", "cross", "cross"])
    heads = rng.choice([(24, 8), (32, 8), (16, 4), (8, 8), (6, 2), (5, 1), (16, 1)])
    d, dtype = rng.choice([64, 128, 256]), rng.choice(["bfloat16", "float16"])
    if op == "plan":
        return {"op": op, "B": _log(rng, 1, 256), "Nq": _log(rng, 1, 250)}
    if op == "accept":
        layers = rng.choice([1, 1, 5, 28])
        nq = _log(rng, 2, 128)
        return {"op": op, "B": _log(rng, 1, 64 if layers == 1 else 16), "Hkv": heads[1], "Nq": nq, "d": d,
                "longest": _log(rng, 140, 300 if layers > 1 else 2000), "most": rng.randint(1, min(nq, 12)), "layers": layers}
    if op == "tree":
        longest, nq = _log(rng, 1, 65536), _log(rng, 1, 128)
        room = min((1 << 29) // (longest * heads[1] * d), (1 << 37) // (longest * heads[0] * nq * max(d, 128)))
        window = rng.choice([0, 0, _log(rng, 1, 8192)])
        return {"op": op, "B": _log(rng, 1, max(1, min(64, room))), "Hq": heads[0], "Hkv": heads[1], "Nq": nq, "d": d,
                "longest": longest, "window": window, "sinks": rng.choice([0, 1, 4, 70]) if window else 0, "dtype": dtype}
    nq, nkv = rng.choice([1, rng.randint(2, 16), _log(rng, 1, 2048)]), _log(rng, 1, 8192)
    room = min((1 << 28) // (nkv * heads[1] * d), (1 << 37) // (nkv * nq * heads[0] * max(d, 128)))
    return {"op": op, "B": _log(rng, 1, max(1, min(64, room))), "Hq": heads[0], "Hkv": heads[1], "Nq": nq, "Nkv": nkv,
            "d": d, "dtype": dtype}


def _sizes(case):
    """Of the case alone: context keys and nodes of each sequence, or the keys of its encoder."""
    r = np.random.RandomState(case["B"] * 7919 + case["Nq"])
    B = case["B"]
    if case["op"] == "cross":
        n = r.randint(max(1, case["Nkv"] // 4), case["Nkv"] + 1, B)
        n[r.randint(B)] = case["Nkv"]
        if B > 8:
            n[1] = 0  # a slot of the batch that no request uses
        return n.astype(np.int64)
    nodes = r.randint((case["Nq"] + 1) // 2, case["Nq"] + 1, B)
    nodes[r.randint(B)] = case["Nq"]
    if B > 8:
        nodes[2] = 1  # a request that goes on without drafts
    if case["op"] == "plan":
        return None, nodes.astype(np.int64)
    top = case["longest"]
    n = np.minimum(np.exp(r.uniform(math.log(max(1, top // 16)), math.log(top + 1), B)).astype(np.int64), top)
    n[r.randint(B)] = top
    if B > 8:
        n[1] = nodes[1] = 0
    return n, nodes.astype(np.int64)


def _pages(n):
    return (n + TILE - 1) // TILE


# ------------------------------------------------------------------ inputs
def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _parents(r, B, nq):
    """Trees, level by level: a node hangs on one of the earlier ones, the first on the context."""
    i = np.arange(1, nq)
    p = np.full((B, nq), -1)
    if nq > 1:
        p[:, 1:] = r.randint((i - 1) // 4, (i - 1) // 2 + 1, (B, nq - 1))
    return p


def _kv(g, heads, n, d):
    """Keys and values [heads, n, d]: keys around a direction of their head, with a few large channels; values normal."""
    u = torch.randn(heads, 1, d, device="cuda", generator=g)
    k = torch.randn(heads, n, d, device="cuda", generator=g).mul_(0.5).add_(u)
    k[:, :, : d // 32] *= 4.0
    return k, torch.randn(heads, n, d, device="cuda", generator=g), u


def _encode(x, s):
    """x [..., d] under the head scales s -> E2M1 codes uint8 [..., d] and scale codes uint8 [..., d / 16]."""
    x = x.unflatten(-1, (-1, 16))
    b8 = (x.abs().amax(-1) / (6.0 * s)).clamp(max=448.0).to(torch.float8_e4m3fn)
    b = b8.float()
    y = x * torch.where(b > 0, 1.0 / (b * s), 0.0)[..., None]
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    code = torch.bucketize(y.abs(), edges).to(torch.uint8) + 8 * (y < 0).to(torch.uint8)
    return code.flatten(-2), b8.view(torch.uint8)


def _places(d):
    """The byte, in its 16-key block, of each byte of the order K codes [16, d / 2], V codes [16, d / 16, 8], K scales
    [16, d / 16], V scales [16, d / 16]."""
    i, n = np.arange(16)[:, None], d // 16
    t, g = np.arange(n)[None, :, None], np.arange(8)[None, None, :]
    v = 8 * d + 512 * (t // 4) + 16 * (4 * g + i[..., None] // 4) + 4 * (t % 4) + i[..., None] % 4
    s = np.arange(n)[None, :]
    return i * (d // 2) + np.arange(d // 2)[None, :], v.reshape(16, d // 2), 16 * d + i * n + s, 17 * d + 4 * ((i // 4) * n + s) + i % 4


def _pool(g, H, npages, d):
    """A pool of quantized keys and values; (pages, k scales, v scales, the keys' directions)."""
    k, v, u = _kv(g, H, npages * TILE, d)
    scales, parts = [], []
    for x, pair in ((k, (-1, 2)), (v, (-1, 2, 8))):
        s = (x.abs().amax((1, 2)) / 2688.0).clamp_min(2.0 ** -100)
        c, b = _encode(x, s[:, None, None])
        c = c.unflatten(-1, pair)
        low, high = (c[..., 0], c[..., 1]) if len(pair) == 2 else (c[..., 0, :], c[..., 1, :])
        flat = lambda y: y.reshape(H, npages, 4, -1).transpose(0, 1)  # noqa: E731
        scales.append(s)
        parts.append((flat((low | (high << 4)).flatten(2)), flat(b)))
        del x, c
    blocks = torch.cat([parts[0][0], parts[1][0], parts[0][1], parts[1][1]], -1)
    back = np.argsort(np.concatenate([p.ravel() for p in _places(d)]))
    return blocks.index_select(-1, torch.from_numpy(back).cuda()).reshape(npages, H, 72 * d), scales[0], scales[1], u


def _table(r, keys, spare):
    """A block table for sequences of `keys`, their pages in any order, and the number of pages of the pool."""
    held = _pages(keys)
    total, most = int(held.sum()), int(held.max()) + 1
    order = r.permutation(total + spare)
    table = np.full((len(keys), most), -1)
    table[np.arange(most)[None, :] < held[:, None]] = order[:total]
    return table, total + spare


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    r = np.random.RandomState(seed & 0x7FFFFFFF)
    op, B, nq = case["op"], case["B"], case["Nq"]
    if op == "plan":
        return {"case": case, "parents": _cuda(_parents(r, B, nq)), "nodes": _cuda(_sizes(case)[1])}
    H, d = case["Hkv"], case["d"]
    if op == "cross":  # out of projections, tokens first
        dtype = getattr(torch, case["dtype"])
        k, v, u = _kv(g, H, B * case["Nkv"], d)
        kv = torch.empty(B, case["Nkv"], 2, H, d, dtype=dtype, device="cuda")
        kv[:, :, 0] = k.view(H, B, -1, d).permute(1, 2, 0, 3)
        kv[:, :, 1] = v.view(H, B, -1, d).permute(1, 2, 0, 3)
        q = torch.randn(B, nq, H, case["Hq"] // H, d, device="cuda", generator=g).mul_(0.5).add_(u.view(H, 1, d))
        return {"case": case, "q": q.mul_(1.5).reshape(B, nq, case["Hq"], d).to(dtype).transpose(1, 2),
                "k": kv[:, :, 0].transpose(1, 2), "v": kv[:, :, 1].transpose(1, 2), "lens": _cuda(_sizes(case))}
    base, nodes = _sizes(case)
    table, npages = _table(r, base + nodes, 2)
    state = {"case": case, "table": _cuda(table), "lens": _cuda(base + nodes), "nodes": _cuda(nodes)}
    if op == "accept":
        # the root, and behind it nodes of the levels below; what is read is not written over, so that a pass can come again
        counts = np.minimum(r.randint(1, case["most"] + 1, B), nodes)
        path = np.zeros((B, case["most"]), np.int64)
        for b in range(B):
            behind = np.arange(max(1, counts[b]), nodes[b])
            counts[b] = min(counts[b], 1 + len(behind)) if nodes[b] else 0
            path[b, 1: counts[b]] = np.sort(r.choice(behind, max(0, counts[b] - 1), replace=False)) if counts[b] > 1 else 0
        pool = [_pool(g, H, npages, d)[0] for _ in range(case["layers"])]
        return dict(state, pages=torch.stack(pool) if case["layers"] > 1 else pool[0], path=_cuda(path), counts=_cuda(counts))
    state["pages"], state["ks"], state["vs"], u = _pool(g, H, npages, d)
    plan = _plain_plan(_cuda(_parents(r, B, nq)), state["nodes"])
    q = torch.randn(B, nq, H, case["Hq"] // H, d, device="cuda", generator=g).mul_(0.5).add_(u.view(H, 1, d))
    return dict(state, q=q.mul_(1.5).reshape(B, nq, case["Hq"], d).to(getattr(torch, case["dtype"])).transpose(1, 2),
                mask=plan["mask"], depths=plan["depths"])


# ------------------------------------------------------------------ the plain forms
def _plain_plan(parents, nodes):
    B, n = parents.shape
    i = torch.arange(n, device="cuda")
    used = i[None, :] < nodes[:, None]
    reach = ((parents[:, :, None] == i) | (i[:, None] == i)).float()  # [B, row, node]
    for _ in range(max(1, n - 1).bit_length()):
        reach = (reach @ reach > 0).float()
    bits = (reach > 0) & used[:, :, None] & used[:, None, :]
    depths = torch.where(used, bits.sum(-1) - 1, 0)
    words = torch.nn.functional.pad(bits, (0, -n % 32)).unflatten(-1, (-1, 32)).long()
    return {"mask": (words << torch.arange(32, device="cuda")).sum(-1).to(torch.int32), "depths": depths.to(torch.int32)}


def _decode(blocks, d, ks, vs):
    """Keys and values [..., 16, d] in FP32 from 16-key blocks [..., 18 d]; ks, vs: head scales, to broadcast."""
    order = torch.from_numpy(np.concatenate([p.ravel() for p in _places(d)])).cuda()
    kc, vc, sk, sv = blocks.index_select(-1, order).split([8 * d, 8 * d, d, d], -1)
    lut = torch.tensor(GRID + tuple(-x for x in GRID), device="cuda")
    value = lambda c: lut.index_select(0, c.reshape(-1).int()).view(c.shape)  # noqa: E731
    k = torch.stack([value(kc & 15), value(kc >> 4)], -1).unflatten(-2, (16, -1)).flatten(-2)
    vc = vc.unflatten(-1, (16, -1, 8))
    v = torch.stack([value(vc & 15), value(vc >> 4)], -2).flatten(-3)
    scale = lambda c, s: c.contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (16, -1))[..., None] * s[..., None, None]  # noqa: E731
    return tuple((x.unflatten(-1, (-1, 16)) * scale(c, s)).flatten(-2) for x, c, s in ((k, sk, ks), (v, sv, vs)))


def _attend(q, k, v, see):
    """q [B, Hq, Nq, d], k and v [B, H, keys, d] in FP32, see [B, Nq or 1, keys] -> (out, lse); rows that see nothing
    give zeros and -inf."""
    B, Hq, Nq, d = q.shape
    H = k.shape[1]
    score = q.float().reshape(B, H, -1, d) @ k.transpose(2, 3) * (1.0 / math.sqrt(d))
    score = score.view(B, Hq, Nq, -1).masked_fill_(~see[:, None], -math.inf)
    m = score.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = score.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(B, H, -1, p.shape[-1]) @ v).view(B, Hq, Nq, d) / torch.where(total > 0, total, 1.0)
    return {"out": out.to(q.dtype), "lse": (m + torch.log(total))[..., 0]}


def _plain_tree(s):
    case, q = s["case"], s["q"]
    B, _, Nq, d = q.shape
    H = case["Hkv"]
    k, v = _decode(s["pages"][s["table"].clamp_min(0).long()].unflatten(-1, (4, 18 * d)), d, s["ks"].view(-1, 1, 1),
                   s["vs"].view(-1, 1, 1))
    k, v = (x.permute(0, 2, 1, 3, 4, 5).reshape(B, H, -1, d) for x in (k, v))
    j, base = torch.arange(k.shape[2], device="cuda"), (s["lens"] - s["nodes"]).view(B, 1)
    node = j - base
    drafted = (node >= 0) & (node < s["nodes"].view(B, 1))
    at = node.clamp(0, Nq - 1)
    bit = (s["mask"].gather(2, (at // 32)[:, None].expand(-1, Nq, -1)) >> (at % 32)[:, None]) & 1
    see = (node < 0)[:, None] | (drafted[:, None] & (bit != 0))
    see = see & (torch.arange(Nq, device="cuda")[None, :, None] < s["nodes"].view(B, 1, 1))
    if case["window"]:
        pos = torch.where(node < 0, j, base + s["depths"].gather(1, at))[:, None]
        see &= (pos > base[:, :, None] + s["depths"][:, :, None] - case["window"]) | (pos < case["sinks"])
    return _attend(q, k, v, see)


def _plain_accept(s):
    pages, table = s["pages"], s["table"].long()
    layers = pages if pages.dim() == 4 else pages[None]
    H, d = layers.shape[2], layers.shape[3] // 72
    base = (s["lens"] - s["nodes"]).long()
    k = torch.arange(s["path"].shape[1], device="cuda")
    b, k = (k[None, :] < s["counts"][:, None]).nonzero(as_tuple=True)
    src, dst = base[b] + s["path"][b, k], base[b] + k
    at = torch.from_numpy(np.concatenate(_places(d), 1)).cuda()  # [key of its block, bytes of a key]

    def index(pos):  # bytes of the keys, all heads: [moved, H, bytes]
        page = table[b, pos // TILE]
        head = (page[:, None] * H + torch.arange(H, device="cuda")) * (72 * d)
        return (head + (pos % TILE // 16 * (18 * d))[:, None])[..., None] + at[pos % 16][:, None]

    flat = layers.reshape(layers.shape[0], -1)
    flat[:, index(dst).reshape(-1)] = flat[:, index(src).reshape(-1)]
    return {"lens": (base + s["counts"]).to(torch.int32), "pages": pages}


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import mixed_precision_attention_gb300 as apa
        if op == "plan":
            return apa.draft_tree(state["parents"], state["nodes"])
        if op == "accept":
            lens = apa.cache_accept(state["pages"], state["table"], state["lens"], state["nodes"], state["path"], state["counts"])
            return {"lens": lens, "pages": state["pages"]}
        if op == "tree":
            out, lse = apa.attention_tree(state["q"], state["pages"], state["table"], state["lens"], state["nodes"], state["mask"],
                                          state["ks"], state["vs"], depths=state["depths"], window=case["window"],
                                          sinks=case["sinks"])
        else:
            out, lse = apa.attention_cross(state["q"], state["k"], state["v"], state["lens"])
        return {"out": out, "lse": lse}
    if op == "plan":
        return _plain_plan(state["parents"], state["nodes"])
    if op == "accept":
        return _plain_accept(state)
    if op == "tree":
        return _plain_tree(state)
    see = torch.arange(case["Nkv"], device="cuda") < state["lens"].view(-1, 1, 1)
    return _attend(state["q"], state["k"].float(), state["v"].float(), see)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, B, nq = case["op"], case["B"], case["Nq"]
    if op == "plan":
        return {"bytes": 4.0 * B * (nq + 1 + nq * ((nq + 31) // 32) + nq), "flops": 0.0}
    d, H = case["d"], case["Hkv"]
    if op == "accept":  # the keys behind the root, read and written
        moved = B * (case["most"] - 1) / 2.0
        return {"bytes": moved * H * 2 * d * 9 / 16 * 2 * case["layers"] + 4.0 * B * (case["most"] + 6), "flops": 0.0}
    if op == "cross":
        keys = float(_sizes(case).sum())
        return {"bytes": keys * H * 4 * d + B * case["Hq"] * nq * (4.0 * d + 4) + 4.0 * B,
                "flops": 4.0 * d * case["Hq"] * nq * keys}
    base, nodes = (x.astype(np.float64) for x in _sizes(case))
    seen = base + nodes  # of a sequence; a row sees its context and, at least, itself
    each = base + 1
    if case["window"]:
        each = np.minimum(base + 1, case["window"]) + np.minimum(np.maximum(base + 1 - case["window"], 0), case["sinks"])
        seen = np.minimum(base, case["window"] - 1) + np.minimum(np.maximum(base + 1 - case["window"], 0), case["sinks"]) + nodes
    rows = float(nodes.sum()) * case["Hq"]
    return {"bytes": float(np.where(nodes > 0, seen, 0).sum()) * H * 2 * d * 9 / 16 + rows * 2 * d + B * case["Hq"] * nq * (2.0 * d + 4)
            + 4.0 * (B * nq * ((nq + 31) // 32) + 2 * B + float(_pages(base + nodes).sum())),
            "flops": 4.0 * d * case["Hq"] * float((each * nodes).sum())}


# ------------------------------------------------------------------ in 64 bits, apart from the above
def _values(block, d):
    """Keys and values [..., 16, d] in 64 bits, without head scales, of 16-key blocks [..., 18 d]: each value's byte
    and nibble looked up, and the formats' definitions."""
    i, ch = torch.arange(16, device="cuda")[:, None], torch.arange(d, device="cuda")[None, :]
    byte = lambda at: block[..., at.reshape(-1)].unflatten(-1, (16, d)).long()  # noqa: E731

    def e2m1(c):
        e, m = (c >> 1) & 3, c & 1
        return torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2((e - 1).double())) * (1 - 2 * (c >> 3))

    def e4m3(c):
        e, m = c >> 3, c & 7
        return torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * torch.exp2((e - 7).double()))

    t = ch // 16
    k = e2m1((byte(i * (d // 2) + ch // 2) >> (4 * (ch % 2))) & 15) * e4m3(byte(16 * d + i * (d // 16) + t))
    v = byte(8 * d + 512 * (t // 4) + 16 * (4 * (ch % 8) + i // 4) + 4 * (t % 4) + i % 4) >> (4 * (ch // 8 % 2))
    return k, e2m1(v & 15) * e4m3(byte(17 * d + 4 * ((i // 4) * (d // 16) + t) + i % 4))


def exact(case, seed):
    op, B, nq = case["op"], case["B"], case["Nq"]
    if op in ("plan", "accept"):
        return None  # whole numbers throughout
    if work(case)["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    Hq, H, d = case["Hq"], case["Hkv"], case["d"]
    G = Hq // H
    out = torch.zeros(B, Hq, nq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, nq), -math.inf, dtype=torch.float64, device="cuda")
    if op == "cross":
        for b, n in enumerate(_sizes(case).tolist()):
            for h in range(Hq):
                if n:
                    x = s["q"][b, h].double() @ s["k"][b, h // G, :n].double().T / math.sqrt(d)
                    lse[b, h] = torch.logsumexp(x, 1)
                    out[b, h] = torch.softmax(x, 1) @ s["v"][b, h // G, :n].double()
        return {"out": out, "lse": lse}
    # the trees again, as prepare() draws them behind the table
    r = np.random.RandomState(seed & 0x7FFFFFFF)
    base, nodes = _sizes(case)
    table, _ = _table(r, base + nodes, 2)
    parents = _parents(r, B, nq)
    for b in range(B):
        n0, nn = int(base[b]), int(nodes[b])
        if not nn:
            continue
        sees = np.ones((nn, n0 + nn), bool)
        sees[:, n0:] = False
        pos = np.arange(n0 + nn)
        for i in range(nn):
            at = i
            while at >= 0:
                sees[i, n0 + at] = True
                at = parents[b, at]
            pos[n0 + i] = n0 + sees[i, n0:].sum() - 1
        if case["window"]:
            sees &= (pos[None, :] > pos[n0:, None] - case["window"]) | (pos[None, :] < case["sinks"])
        hidden = torch.from_numpy(~sees).cuda()
        pages = s["pages"][torch.from_numpy(table[b, : -(-(n0 + nn) // TILE)].astype(np.int64)).cuda()]
        for h in range(H):
            k, v = (x.reshape(-1, d)[: n0 + nn] for x in _values(pages[:, h].unflatten(-1, (4, 18 * d)), d))
            k, v = k * s["ks"][h].double(), v * s["vs"][h].double()
            for g in range(h * G, h * G + G):
                x = (s["q"][b, g, :nn].double() @ k.T / math.sqrt(d)).masked_fill_(hidden, -math.inf)
                lse[b, g, :nn] = torch.logsumexp(x, 1)
                out[b, g, :nn] = torch.softmax(x, 1) @ v
    return {"out": out, "lse": lse}
