"""Cases, plain forms and 64-bit values of the serving operators around the 4-bit paged K/V cache:

* cache_tables      block tables and slot maps from request lengths, on the GPU
* cache_write       tokens' K and V quantized to NVFP4 into the pages of the cache
* cache_read        the values that cached tokens stand for
* attention_cache   attention of a few query rows per sequence over that cache, with an
                    optional sliding window and first tokens that stay visible (sinks)
* attention_window  causal prefill attention with a sliding window and sinks

The cache is a pool uint8 [num_pages, Hkv, 72 d]: a page holds 64 keys of all KV heads, as
four blocks of 16 keys of 18 d bytes each:

  K codes   8 d bytes   key i, byte x: the E2M1 codes of channels 2x (low nibble), 2x + 1
  V codes   8 d bytes   key i, channels 16 t + g (low nibble) and 16 t + 8 + g, g < 8, at byte
                        512 (t / 4) + 16 (4 g + i / 4) + 4 (t % 4) + i % 4
  K scales    d bytes   UE4M3, key i, channels 16 t .. 16 t + 15 at byte i d / 16 + t
  V scales    d bytes   UE4M3, key i, channels 16 t .. 16 t + 15 at byte 4 ((i / 4) d / 16 + t) + i % 4

A value is E2M1 * UE4M3 * the FP32 scale of its KV head.  Quantizing a group of 16 values x
under the head scale s, in FP32: scale code b = UE4M3(max|x| / (6 s)), codes 0 if b is 0, else
E2M1(x * (1 / (b s))), each rounded to nearest even and saturating.
"""
import math

import numpy as np
import torch

own = False

TILE = 64  # keys in a page
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one step of a decoding batch: every request grows by a token, a few end, a few begin
        {"name": "tables step", "op": "tables", "B": 192, "longest": 9000, "kind": "step", "max_tokens": 256},
        # a batch of new prompts enters an empty cache
        {"name": "tables prompts", "op": "tables", "B": 41, "longest": 9000, "kind": "prompts", "max_tokens": 262144},
        # the new token of each sequence of a decoding batch
        {"name": "write step", "op": "write", "T": 128, "Hkv": 8, "d": 128, "kind": "step", "dtype": "bfloat16"},
        # a prompt, out of a fused projection's output (so with strides), odd start and length
        {"name": "write prompt", "op": "write", "T": 16411, "Hkv": 8, "d": 128, "kind": "prompt", "dtype": "bfloat16"},
        # a cached prefix taken out again, for a prompt that shares it
        {"name": "read prefix", "op": "read", "T": 40000, "Hkv": 8, "d": 128, "kind": "prompt", "dtype": "bfloat16"},
        # the first tokens of a single conversation: latency
        {"name": "decode single", "op": "decode", "B": 1, "Hq": 24, "Hkv": 8, "Nq": 1, "d": 128, "longest": 1000,
         "window": 0, "sinks": 0, "dtype": "bfloat16"},
        # a batch of conversations of many lengths
        {"name": "decode batch", "op": "decode", "B": 64, "Hq": 24, "Hkv": 8, "Nq": 1, "d": 128, "longest": 8192,
         "window": 0, "sinks": 0, "dtype": "bfloat16"},
        # long contexts
        {"name": "decode long", "op": "decode", "B": 8, "Hq": 32, "Hkv": 8, "Nq": 1, "d": 128, "longest": 131072,
         "window": 0, "sinks": 0, "dtype": "bfloat16"},
        # four drafted tokens per sequence, checked at once, under a sliding window with sinks
        {"name": "decode drafted window", "op": "decode", "B": 48, "Hq": 16, "Hkv": 4, "Nq": 4, "d": 64,
         "longest": 32768, "window": 4096, "sinks": 4, "dtype": "float16"},
        # a short prompt
        {"name": "window short", "op": "window", "B": 1, "Hq": 8, "Hkv": 2, "Nq": 509, "Nkv": 509, "d": 64,
         "window": 128, "sinks": 4},
        # a prompt under a narrow window
        {"name": "window prompt", "op": "window", "B": 1, "Hq": 24, "Hkv": 8, "Nq": 8192, "Nkv": 8192, "d": 128,
         "window": 1024, "sinks": 4},
        # a chunk at the end of a long prompt, under a wide window
        {"name": "window chunk", "op": "window", "B": 1, "Hq": 24, "Hkv": 8, "Nq": 16384, "Nkv": 122880, "d": 128,
         "window": 4096, "sinks": 16},
    ]


def _log(rng, lo, hi):
    """A whole number, uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "write", "read", "decode", "decode", "window", "window"])
    heads = rng.choice([(24, 8), (32, 8), (16, 4), (8, 8), (6, 2), (5, 1), (16, 1)])
    if op == "tables":
        kind = rng.choice(["step", "prompts"])
        B = _log(rng, 1, 512 if kind == "step" else 41)
        longest = _log(rng, 70, 9000)
        return {"op": op, "B": B, "longest": longest, "kind": kind,
                "max_tokens": B + rng.randrange(64) if kind == "step" else B * longest + rng.randrange(1000)}
    if op in ("write", "read"):
        kind = rng.choice(["step", "prompt"])
        return {"op": op, "T": _log(rng, 1, 512 if kind == "step" else 16384), "Hkv": heads[1],
                "d": rng.choice([64, 128, 256]), "kind": kind, "dtype": rng.choice(["bfloat16", "float16"])}
    if op == "decode":
        d = rng.choice([64, 128, 256])
        longest = _log(rng, 1, 65536)
        B = _log(rng, 1, max(1, min(256, (1 << 30) // (longest * heads[1] * d))))
        window = rng.choice([0, 0, _log(rng, 1, 8192)])
        return {"op": op, "B": B, "Hq": heads[0], "Hkv": heads[1], "Nq": rng.choice([1, 1, 2, 3, 5, 8]), "d": d,
                "longest": longest, "window": window, "sinks": rng.choice([0, 1, 4, 70]) if window else 0,
                "dtype": rng.choice(["bfloat16", "float16"])}
    d = rng.choice([64, 128, 256])
    B = rng.choice([1, 1, 2])
    nq = _log(rng, 1, min(8192, 8192 * 128 // (B * d)))
    return {"op": op, "B": B, "Hq": heads[0], "Hkv": heads[1], "Nq": nq,
            "Nkv": nq + rng.choice([0, _log(rng, 1, 16384)]), "d": d, "window": _log(rng, 1, 4096),
            "sinks": rng.choice([0, 1, 4, 100])}


def _lens(case):
    """(old, new) lengths of a tables case, or the lengths of a decode case: of the case alone."""
    r = np.random.RandomState(case["B"] * 7919 + case["longest"])
    B, top = case["B"], case["longest"]
    if case["op"] == "decode":
        n = np.exp(r.uniform(math.log(max(1, top // 16)), math.log(top + 1), B)).astype(np.int64)
        n[r.randint(B)] = top
        if B > 8:
            n[1] = 0  # a slot of the batch that no request uses
        return np.minimum(n, top).astype(np.int32)
    n = r.randint(1, top, B)
    if case["kind"] == "prompts":
        return np.zeros(B, np.int32), n.astype(np.int32)
    new = n + 1
    what = r.randint(0, 16, B)
    new[what == 0] = 0                       # ends: its pages go back
    n[what == 1], new[what == 1] = 0, 1      # begins
    return n.astype(np.int32), new.astype(np.int32)


def _pages(n):
    return (n + TILE - 1) // TILE


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _kv(g, heads, n, d, dtype):
    """Keys and values [heads, n, d]: keys around a direction of their head, with a few large channels, the first
    key larger; values normal."""
    u = torch.randn(heads, 1, d, device="cuda", generator=g)
    k = torch.randn(heads, n, d, device="cuda", generator=g).mul_(0.5).add_(u)
    k[:, :, : d // 32] *= 4.0
    if n:
        k[:, 0] *= 2.0
    v = torch.randn(heads, n, d, device="cuda", generator=g)
    return k.to(dtype), v.to(dtype), u


def _scales(x):
    """The FP32 scale of each head of x [heads, n, d]: its largest value falls on 6 * 448."""
    return (x.float().abs().amax((1, 2)) / 2688.0).clamp_min(2.0 ** -100)


def prepare(case, seed):
    g = _gen(seed)
    r = np.random.RandomState(seed & 0x7FFFFFFF)
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
    op = case["op"]
    if op == "tables":
        old, new = _lens(case)
        B = case["B"]
        most = int(_pages(np.maximum(old, new)).max()) + 2
        held = _pages(old)
        cap = int(held.sum()) + int(np.maximum(_pages(new) - held, 0).sum()) + 64
        order = r.permutation(cap)
        table = np.full((B, most), -1)
        table[np.arange(most)[None, :] < held[:, None]] = order[: held.sum()]
        free = np.full(cap, -1)
        free[: cap - held.sum()] = order[held.sum():]
        return {"case": case, "old": cuda(old), "new": cuda(new), "table": cuda(table), "free": cuda(free),
                "count": cuda([cap - held.sum()])}
    if op in ("write", "read"):
        T, H, d, dtype = case["T"], case["Hkv"], case["d"], getattr(torch, case["dtype"])
        if case["kind"] == "step":  # one token per sequence, each in a page of its own
            npages = T + 3
            slots = r.permutation(npages)[:T] * TILE + r.randint(0, TILE, T)
        else:  # consecutive positions from an odd start, in pages of any order, a padded end
            first = int(r.randint(0, TILE))
            npages = _pages(first + T) + 2
            at = first + np.arange(T)
            slots = r.permutation(npages)[at // TILE] * TILE + at % TILE
            slots[T - T // 64:] = -1
        k, v, _ = _kv(g, H, T, d, dtype)
        qkv = torch.empty(T, 3 * H, d, dtype=dtype, device="cuda")  # the projection's output, tokens first
        qkv[:, H: 2 * H] = k.transpose(0, 1)
        qkv[:, 2 * H:] = v.transpose(0, 1)
        state = {"case": case, "k": qkv[:, H: 2 * H].transpose(0, 1), "v": qkv[:, 2 * H:].transpose(0, 1),
                 "slots": cuda(slots), "pages": torch.zeros(npages, H, 72 * d, dtype=torch.uint8, device="cuda"),
                 "ks": _scales(k), "vs": _scales(v)}
        if op == "read":
            _plain_write(state["k"], state["v"], state["slots"], state["pages"], state["ks"], state["vs"])
            del state["k"], state["v"]
        return state
    if op == "decode":
        B, H, d, dtype = case["B"], case["Hkv"], case["d"], getattr(torch, case["dtype"])
        lens = _lens(case)
        held = _pages(lens.astype(np.int64))
        total = int(held.sum())
        most = int(held.max()) + 1
        npages = total + 2
        order = r.permutation(npages)
        table = np.full((B, most), -1)
        table[np.arange(most)[None, :] < held[:, None]] = order[:total]
        k, v, u = _kv(g, H, npages * TILE, d, dtype)
        ks, vs = _scales(k), _scales(v)
        paged = lambda x: x.view(H, npages, TILE, d).transpose(0, 1)  # noqa: E731
        pages = _pack(_encode(paged(k), ks[None, :, None, None]), _encode(paged(v), vs[None, :, None, None]))
        del k, v
        q = torch.randn(B, case["Nq"], H, case["Hq"] // H, d, device="cuda", generator=g).mul_(0.5)
        q = (q + u.view(1, 1, H, 1, d)).mul_(1.5).reshape(B, case["Nq"], case["Hq"], d).to(dtype)
        return {"case": case, "q": q.transpose(1, 2), "pages": pages, "table": cuda(table), "lens": cuda(lens),
                "ks": ks, "vs": vs}
    B, Hq, H, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    k, v, u = _kv(g, B * H, case["Nkv"], d, torch.bfloat16)
    q = torch.randn(B * H, Hq // H, case["Nq"], d, device="cuda", generator=g).mul_(0.5).add_(u[:, :, None])
    return {"case": case, "q": q.to(torch.bfloat16).view(B, Hq, case["Nq"], d), "k": k.view(B, H, -1, d),
            "v": v.view(B, H, -1, d)}


# ------------------------------------------------------------------ the plain forms
def _encode(x, s):
    """x [..., d], head scales s -> (codes uint8 [..., d], scale codes uint8 [..., d / 16])."""
    x = x.float().unflatten(-1, (-1, 16))
    a = x.abs().amax(-1)
    b8 = (a / (6.0 * s)).clamp(max=448.0).to(torch.float8_e4m3fn)
    b = b8.float()
    inv = torch.where(b > 0, 1.0 / (b * s), 0.0)
    y = x * inv[..., None]
    m = y.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code += torch.signbit(y).to(torch.uint8) * ((b > 0)[..., None] * 8).to(torch.uint8)
    return code.flatten(-2), b8.view(torch.uint8)


def _places(d):
    """The byte, in its 16-key block of 18 d bytes, of each byte of the order K codes [16, d / 2], V codes
    [16, d / 16, 8], K scales [16, d / 16], V scales [16, d / 16]."""
    i, n = np.arange(16)[:, None], d // 16
    t, g = np.arange(n)[None, :, None], np.arange(8)[None, None, :]
    kc = i * (d // 2) + np.arange(d // 2)[None, :]
    vc = 8 * d + 512 * (t // 4) + 16 * (4 * g + i[..., None] // 4) + 4 * (t % 4) + i[..., None] % 4
    ks = 16 * d + i * n + np.arange(n)[None, :]
    vs = 17 * d + 4 * ((i // 4) * n + np.arange(n)[None, :]) + i % 4
    return kc, vc.reshape(16, d // 2), ks, vs


def _nibbles(k, v):
    """Code bytes of keys and values [..., d / 2] from codes [..., d]."""
    k = k.unflatten(-1, (-1, 2))
    v = v.unflatten(-1, (-1, 2, 8))
    return k[..., 0] | (k[..., 1] << 4), (v[..., 0, :] | (v[..., 1, :] << 4)).flatten(-2)


def _pack(kq, vq):
    """Whole pages [num_pages, Hkv, 72 d] from encoded keys and values [num_pages, Hkv, 64, ...]."""
    P, H, _, d = kq[0].shape
    kc, vc = _nibbles(kq[0], vq[0])
    flat = torch.cat([x.reshape(P, H, 4, -1) for x in (kc, vc, kq[1], vq[1])], -1)
    back = np.argsort(np.concatenate([p.ravel() for p in _places(d)]))
    return flat.index_select(-1, torch.from_numpy(back).cuda()).view(P, H, 72 * d)


def _decode(blocks, d, ks, vs):
    """Keys and values [..., 16, d] in FP32 from 16-key blocks [..., 18 d]; ks, vs: head scales, to broadcast."""
    order = torch.from_numpy(np.concatenate([p.ravel() for p in _places(d)])).cuda()
    x = blocks.index_select(-1, order)
    kc, vc, sk, sv = x.split([8 * d, 8 * d, d, d], -1)
    lut = torch.tensor(E2M1, device="cuda")
    value = lambda c: lut.index_select(0, c.reshape(-1).int()).view(c.shape)  # noqa: E731
    k = torch.stack([value(kc & 15), value(kc >> 4)], -1).unflatten(-2, (16, -1)).flatten(-2)
    vc = vc.unflatten(-1, (16, -1, 8))
    v = torch.stack([value(vc & 15), value(vc >> 4)], -2).flatten(-3)
    scale = lambda c: c.contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (16, -1))  # noqa: E731
    times = lambda v, c, s: ((v.unflatten(-1, (-1, 16)) * scale(c)[..., None]) * s[..., None]).flatten(-2)  # noqa: E731
    return times(k, sk, ks), times(v, sv, vs)


def _plain_write(k, v, slots, pages, ks, vs):
    H, T, d = k.shape
    use = (slots >= 0).nonzero()[:, 0]
    slot = slots[use].long()
    (kc, ksc), (vc, vsc) = (_encode(x[:, use], s[:, None, None]) for x, s in ((k, ks), (v, vs)))
    kb, vb = _nibbles(kc, vc)
    base = ((slot // TILE) * H + torch.arange(H, device="cuda")[:, None]) * (72 * d) + (slot % TILE // 16) * (18 * d)
    at = torch.from_numpy(np.concatenate(_places(d), 1)).cuda()[slot % 16]  # [tokens, bytes of a token]
    pages.view(-1)[(base[..., None] + at).reshape(-1)] = torch.cat([kb, vb, ksc, vsc], -1).reshape(-1)


def _plain_read(pages, slots, ks, vs, dtype):
    P, H, n = pages.shape
    d = n // 72
    slot = slots.clamp_min(0).long()
    blocks = pages.view(P, H, 4, 18 * d)[slot // TILE, :, slot % TILE // 16]  # [T, H, 18 d]
    at = torch.from_numpy(np.concatenate(_places(d), 1)).cuda()[slot % 16]
    x = blocks.gather(-1, at[:, None].expand(-1, H, -1)).transpose(0, 1)
    kc, vc, sk, sv = x.split([d // 2, d // 2, d // 16, d // 16], -1)
    lut = torch.tensor(E2M1, device="cuda")
    value = lambda c: lut.index_select(0, c.reshape(-1).int()).view(c.shape)  # noqa: E731
    k = torch.stack([value(kc & 15), value(kc >> 4)], -1).flatten(-2)
    vc = vc.unflatten(-1, (-1, 8))
    v = torch.stack([value(vc & 15), value(vc >> 4)], -2).flatten(-3)
    scale = lambda c: c.contiguous().view(torch.float8_e4m3fn).float()[..., None]  # noqa: E731
    used = (slots >= 0)[None, :, None, None]
    times = lambda v, c, s: torch.where(used, (v.unflatten(-1, (-1, 16)) * scale(c)) * s[:, None, None, None],  # noqa: E731
                                        0.0).flatten(-2).to(dtype)
    return times(k, sk, ks), times(v, sv, vs)


def _plain_tables(s):
    old, new, table, free = s["old"].long(), s["new"].long(), s["table"], s["free"]
    B, most = table.shape
    top = s["case"]["max_tokens"]
    count = s["count"][0].long()
    had, has = (old + TILE - 1) // TILE, (new + TILE - 1) // TILE
    p = torch.arange(most, device="cuda")[None, :]
    give, take = (p >= has[:, None]) & (p < had[:, None]), (p >= had[:, None]) & (p < has[:, None])
    flat = lambda m: m.reshape(-1)  # noqa: E731
    # the pages given back go on top of the free ones, in order; then the new ones come off the top, in order
    stack = torch.cat([free.long(), free.new_zeros(B * most).long()])
    at = torch.where(flat(give), count + flat(give).cumsum(0) - 1, free.numel() + B * most - 1)
    stack.scatter_(0, at, torch.where(flat(give), flat(table).long(), 0))
    full = count + give.sum()
    rank = flat(take).cumsum(0) - 1
    new_table = torch.where(flat(take), stack[(full - 1 - rank).clamp_min(0)], flat(table).long()).view(B, most)
    left = full - take.sum()
    i = torch.arange(free.numel(), device="cuda")
    new_free = torch.where((i >= count) & (i < left), stack[: free.numel()], free.long())
    grown = (new - old).clamp_min(0)
    starts = torch.cat([grown.new_zeros(1), grown.cumsum(0)])
    t = torch.arange(top, device="cuda")
    b = torch.searchsorted(starts, t, right=True).clamp(max=B) - 1
    pos = old[b] + t - starts[b]
    used = t < starts[-1]
    page = new_table.reshape(-1)[(b * most + pos // TILE).clamp(0, B * most - 1)]
    whole = lambda x: x.to(torch.int32)  # noqa: E731
    return {"slots": whole(torch.where(used, page * TILE + pos % TILE, -1)), "positions": whole(torch.where(used, pos, 0)),
            "starts": whole(starts), "free_count": whole(left.view(1)), "status": whole(starts[:1] * 0),
            "table": whole(new_table), "free": whole(new_free)}


def _softmax_out(score, v):
    """Rows of scores [..., rows, keys] (-inf where masked) and values [..., keys, d] -> (out, lse); a row without a
    key gives zeros and -inf."""
    m = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total > 0, total, 1.0)
    return out, (torch.where(m == -math.inf, 0.0, m) + torch.log(total))[..., 0]


def _plain_decode(s):
    case, q = s["case"], s["q"]
    B, Hq, Nq, d = q.shape
    H = case["Hkv"]
    pages = s["pages"][s["table"].clamp_min(0).long()]  # [B, most, H, 72 d]
    k, v = _decode(pages.unflatten(-1, (4, 18 * d)), d, s["ks"].view(-1, 1, 1, 1), s["vs"].view(-1, 1, 1, 1))
    k, v = (x.permute(0, 2, 1, 3, 4, 5).reshape(B, H, -1, d) for x in (k, v))
    j = torch.arange(k.shape[2], device="cuda")
    pos = s["lens"].view(B, 1, 1) - Nq + torch.arange(Nq, device="cuda").view(1, Nq, 1)
    see = j <= pos
    if case["window"]:
        see &= (j > pos - case["window"]) | (j < case["sinks"])
    see = see[:, None, None].expand(B, H, Hq // H, Nq, -1).reshape(B, H, -1, j.numel())
    score = q.float().reshape(B, H, -1, d) @ k.transpose(2, 3) * (1.0 / math.sqrt(d))
    out, lse = _softmax_out(torch.where(see, score, -math.inf), v)
    return {"out": out.view(B, Hq, Nq, d).to(q.dtype), "lse": lse.view(B, Hq, Nq)}


def _plain_window(s):
    """Rows in blocks of 128; each block against the keys that its rows' windows reach, and the sinks."""
    case, q, k, v = s["case"], s["q"].float(), s["k"].float(), s["v"].float()
    B, Hq, Nq, d = q.shape
    H, N, W = k.shape[1], k.shape[2], min(case["window"], k.shape[2])
    S, rows, G = min(case["sinks"], N), 128, Hq // H
    nb = -(-Nq // rows)
    q = torch.nn.functional.pad(q, (0, 0, 0, nb * rows - Nq)).view(B, H, G, nb, rows, d).transpose(2, 3)
    pos = (N - Nq + torch.arange(nb * rows, device="cuda")).view(nb, rows, 1)
    j = pos[:, :1] - W + 1 + torch.arange(W + rows - 1, device="cuda")  # [nb, 1, W + rows - 1]
    see = (j >= 0) & (j <= pos) & (j > pos - W) & (j < N)
    first = torch.arange(S, device="cuda")
    see = torch.cat([see, (first <= pos - W)], -1)[:, None]  # sinks that the window does not reach
    at = torch.cat([j[:, 0].clamp(0, N - 1), first.expand(nb, S)], -1)
    keys, values = k[:, :, at], v[:, :, at]  # [B, H, nb, keys, d]
    score = q.reshape(B, H, nb, G * rows, d) @ keys.transpose(-1, -2) * (1.0 / math.sqrt(d))
    score = torch.where(see, score.unflatten(3, (G, rows)), -math.inf).flatten(3, 4)
    out, lse = _softmax_out(score, values)
    out = out.view(B, H, nb, G, rows, d).transpose(2, 3).reshape(B, Hq, nb * rows, d)[:, :, :Nq]
    lse = lse.view(B, H, nb, G, rows).transpose(2, 3).reshape(B, Hq, nb * rows)[:, :, :Nq]
    return {"out": out.to(torch.bfloat16), "lse": lse}


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import mixed_precision_attention_gb300 as apa
        if op == "tables":
            r = apa.cache_tables(state["old"], state["new"], state["table"], state["free"], state["count"],
                                 case["max_tokens"])
            return dict(r, table=state["table"], free=state["free"])
        if op == "write":
            apa.cache_write(state["k"], state["v"], state["slots"], state["pages"], state["ks"], state["vs"])
        if op in ("write", "read"):
            k, v = apa.cache_read(state["pages"], state["slots"], state["ks"], state["vs"],
                                  dtype=getattr(torch, case["dtype"]))
            return {"k": k, "v": v}
        if op == "decode":
            out, lse = apa.attention_cache(state["q"], state["pages"], state["table"], state["lens"], state["ks"],
                                           state["vs"], window=case["window"], sinks=case["sinks"])
        else:
            out, lse = apa.attention_window(state["q"], state["k"], state["v"], case["window"], sinks=case["sinks"])
        return {"out": out, "lse": lse}
    if op == "tables":
        return _plain_tables(state)
    if op == "write":
        _plain_write(state["k"], state["v"], state["slots"], state["pages"], state["ks"], state["vs"])
    if op in ("write", "read"):
        k, v = _plain_read(state["pages"], state["slots"], state["ks"], state["vs"], getattr(torch, case["dtype"]))
        return {"k": k, "v": v}
    return _plain_decode(state) if op == "decode" else _plain_window(state)


# ------------------------------------------------------------------ what a pass cannot do without
def _pairs(first, last, window, sinks):
    """Visible (row, key) pairs of the rows at positions first .. last, one head."""
    p = np.arange(max(0, first), last + 1, dtype=np.float64)
    if not window:
        return float((p + 1).sum())
    w = np.minimum(p + 1, window)
    return float((w + np.minimum(np.maximum(p + 1 - window, 0), sinks)).sum())


def work(case):
    op = case["op"]
    if op == "tables":
        old, new = _lens(case)
        moved = np.abs(_pages(old.astype(np.int64)) - _pages(new.astype(np.int64))).sum()
        # lengths in; slots, positions and starts out; every page that changes hands read and written
        return {"bytes": 4.0 * (2 * case["B"] + 2 * case["max_tokens"] + case["B"] + 1 + 2 * moved + 3), "flops": 0.0}
    if op in ("write", "read"):
        T, H, d = case["T"], case["Hkv"], case["d"]
        used = T if case["kind"] == "step" else T - T // 64
        cached, values = 2 * used * H * d * 9 / 16, 2 * T * H * d * 2
        if op == "read":
            return {"bytes": float(cached + values + 4 * T), "flops": 2.0 * used * H * d}
        # values in and cached bytes out; then the cached bytes in and values out
        return {"bytes": float(2 * cached + 2 * used * H * d * 2 + values + 8 * T), "flops": 10.0 * used * H * d}
    if op == "decode":
        d, Nq, W, S = case["d"], case["Nq"], case["window"], case["sinks"]
        lens = _lens(case).astype(np.int64)
        reach = np.minimum(lens, W + Nq - 1) if W else lens
        keys = int((reach + np.minimum(np.maximum(lens - reach, 0), S)).sum())
        pairs = sum(_pairs(n - Nq, n - 1, W, S) for n in lens.tolist())
        rows = case["B"] * case["Hq"] * Nq
        return {"bytes": float(keys * case["Hkv"] * 2 * d * 9 / 16 + rows * (4 * d + 4) + 4 * (2 * case["B"]) + 4 * _pages(lens).sum()),
                "flops": 4.0 * d * case["Hq"] * pairs}
    B, Nq, N, d, W = case["B"], case["Nq"], case["Nkv"], case["d"], case["window"]
    keys = min(N, Nq + W - 1) + min(max(0, N - (Nq + W - 1)), case["sinks"])
    return {"bytes": float(B * (2 * case["Hkv"] * keys * d * 2 + case["Hq"] * Nq * (4 * d + 4))),
            "flops": 4.0 * d * case["Hq"] * B * _pairs(N - Nq, N - 1, W, case["sinks"])}


# ------------------------------------------------------------------ in 64 bits, apart from the above
def _value_tables():
    """The values of the 16 E2M1 and the 128 non-negative E4M3 codes, from the formats' definitions."""
    e2m1 = [(-1.0) ** (c >> 3) * ((c & 1) * 0.5 if (c >> 1) & 3 == 0 else 2.0 ** (((c >> 1) & 3) - 1) * (1 + 0.5 * (c & 1)))
            for c in range(16)]
    e4m3 = [(c & 7) * 2.0 ** -9 if c >> 3 == 0 else 2.0 ** ((c >> 3) - 7) * (1 + (c & 7) / 8.0) for c in range(127)] + [math.nan]
    return np.array(e2m1), np.array(e4m3)


def _unpack64(block, d):
    """Keys and values [..., 16, d] of 16-key blocks [..., 18 d], without the head scales: each value's byte and nibble
    looked up."""
    e2m1, e4m3 = (torch.from_numpy(t).cuda() for t in _value_tables())
    i, ch = torch.arange(16, device="cuda")[:, None], torch.arange(d, device="cuda")[None, :]
    t, g, high = ch // 16, ch % 8, ch // 8 % 2
    byte = lambda at: block[..., at.reshape(-1)].unflatten(-1, (16, d)).long()  # noqa: E731
    kb, vb = byte(i * (d // 2) + ch // 2), byte(8 * d + 512 * (t // 4) + 16 * (4 * g + i // 4) + 4 * (t % 4) + i % 4)
    k = e2m1[(kb >> (4 * (ch % 2))) & 15] * e4m3[byte(16 * d + i * (d // 16) + t)]
    v = e2m1[(vb >> (4 * high)) & 15] * e4m3[byte(17 * d + 4 * ((i // 4) * (d // 16) + t) + i % 4)]
    return k, v


def _quantized64(x, s):
    """What quantizing x [..., d] under the head scales s stands for; the FP32 steps of the definition rounded from 64 bits."""
    f32 = lambda a: a.astype(np.float32).astype(np.float64)  # noqa: E731
    e2m1, e4m3 = _value_tables()
    grid, codes = e2m1[:8], e4m3[:127]

    def nearest(y, values):  # ties to the even code
        lo = np.clip(np.searchsorted(values, y, side="right") - 1, 0, len(values) - 2)
        down, up = y - values[lo], values[lo + 1] - y
        return np.where((up < down) | ((up == down) & (lo % 2 == 1)), lo + 1, lo)

    g = x.reshape(x.shape[:-1] + (-1, 16))
    b = codes[nearest(np.minimum(f32(np.abs(g).max(-1) / f32(6.0 * s)), 448.0), codes)]
    with np.errstate(divide="ignore", invalid="ignore"):
        y = f32(g * f32(1.0 / f32(b * s))[..., None])
    y = np.where(b[..., None] > 0, y, 0.0)
    q = grid[nearest(np.minimum(np.abs(y), 6.0), grid)] * np.sign(y)
    return (q * (b * s)[..., None]).reshape(x.shape)


def exact(case, seed):
    op = case["op"]
    if op == "tables":
        return None  # whole numbers throughout
    if op in ("write", "read"):
        s = prepare(dict(case, op="write"), seed)
        used = (s["slots"].cpu().numpy() >= 0)[None, :, None]
        at = lambda x, c: np.where(used, _quantized64(x.double().cpu().numpy(), c.double().cpu().numpy()[:, None, None]), 0.0)  # noqa: E731
        return {"k": at(s["k"], s["ks"]), "v": at(s["v"], s["vs"])}
    s = prepare(case, seed)
    if op == "decode":
        q, table = s["q"].double(), s["table"].cpu().numpy()
        B, Hq, Nq, d = q.shape
        H = case["Hkv"]
        G = Hq // H
        out = torch.zeros(B, Hq, Nq, d, dtype=torch.float64, device="cuda")
        lse = torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(_lens(case).tolist()):
            if not n:
                continue
            pages = s["pages"][torch.from_numpy(table[b, : -(-n // TILE)].astype(np.int64)).cuda()]
            k, v = _unpack64(pages.view(-1, H, 4, 18 * d), d)
            k, v = (x.permute(1, 0, 2, 3, 4).reshape(H, -1, d)[:, :n] for x in (k, v))
            for h in range(H):
                for i in range(Nq):
                    p = n - Nq + i
                    if p < 0:
                        continue
                    lo = max(0, p + 1 - case["window"]) if case["window"] else 0
                    seen = torch.cat([torch.arange(min(case["sinks"], lo), device="cuda"), torch.arange(lo, p + 1, device="cuda")])
                    x = (k[h, seen] * s["ks"][h].double()) @ q[b, h * G: (h + 1) * G, i].T / math.sqrt(d)  # [keys, G]
                    lse[b, h * G: (h + 1) * G, i] = torch.logsumexp(x, 0)
                    out[b, h * G: (h + 1) * G, i] = torch.softmax(x, 0).T @ (v[h, seen] * s["vs"][h].double())
        return {"out": out, "lse": lse}
    B, Hq, Nq, d = s["q"].shape
    G, N = Hq // case["Hkv"], case["Nkv"]
    if float(B * Hq * Nq) * min(N, case["window"] + 600) * d > 2e12:
        return None
    out = torch.empty(B, Hq, Nq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(B, Hq, Nq, dtype=torch.float64, device="cuda")
    for b in range(B):
        for h in range(Hq):
            k, v = s["k"][b, h // G].double(), s["v"][b, h // G].double()
            for r in range(0, Nq, 512):
                p = N - Nq + torch.arange(r, min(Nq, r + 512), device="cuda")
                lo = max(0, int(p[0]) + 1 - case["window"])
                seen = torch.cat([torch.arange(min(case["sinks"], lo), device="cuda"), torch.arange(lo, int(p[-1]) + 1, device="cuda")])
                x = s["q"][b, h, r: r + 512].double() @ k[seen].T / math.sqrt(d)
                hidden = (seen[None] > p[:, None]) | ((seen[None] <= p[:, None] - case["window"]) & (seen[None] >= case["sinks"]))
                x = x.masked_fill(hidden, -math.inf)
                lse[b, h, r: r + 512] = torch.logsumexp(x, 1)
                out[b, h, r: r + 512] = torch.softmax(x, 1) @ v[seen]
    return {"out": out, "lse": lse}
