"""The 4-bit paged K/V cache: tables, writing, reading and attention over it, against
plain 64-bit implementations written here from the formulas in include/apa.h.

Tolerances count roundings of half a step, torch.finfo(t).eps / 2 of the value: bf16 has 8
significant bits, so its values in [1, 2) are 2^-7 apart and a rounding is off by up to
2^-8; fp16 has 11 bits, 2^-11.  An attention output is one rounding to its type of a sum
of softmax-weighted values whose weights were rounded to FP16 (2^-11 each); the weights
and their sum come from FP32 scores, off by at most a few 2^-24 of |s| (2^-14 covers
scores up to a few hundred).  So
|out - ref| <= 2^-8 (or 2^-11) |ref| + (2^-11 + 2^-14) * sum_j w_j |v_j|, and
|lse - ref| <= 1e-5 * max(1, |ref|).
(One key of value v gives out = round(v): the error reaches 2^-8 |v| in bf16, and no
tolerance below that can hold.)
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6])
E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else 2.0 ** ((c >> 3) - 7) * (1 + (c & 7) / 8) for c in range(127)])


def _quantize(x, s):
    """(codes, scale codes) of x [..., d] under head scale s, by the definition: its FP32 steps in numpy float32."""
    x = np.asarray(x, np.float32)
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // 16, 16))
    s = np.asarray(s, np.float32)
    r = np.minimum(np.abs(g).max(-1) / (np.float32(6) * s), np.float32(448)).astype(np.float64)

    def nearest(y, values):  # ties to even codes
        lo = np.clip(np.searchsorted(values, y, side="right") - 1, 0, len(values) - 2)
        a, b = y - values[lo], values[lo + 1] - y
        return np.where((b < a) | ((a == b) & (lo % 2 == 1)), lo + 1, lo)

    sb = nearest(r, E4M3)
    with np.errstate(divide="ignore", invalid="ignore"):
        y = g * (np.float32(1) / (E4M3[sb].astype(np.float32) * s))[..., None]
    y = np.where((sb > 0)[..., None], y, 0)
    m = nearest(np.minimum(np.abs(y).astype(np.float64), 6.0), E2M1[:8])
    code = m + 8 * (np.signbit(y) & (sb > 0)[..., None])
    return code.reshape(x.shape).astype(np.uint8), sb.astype(np.uint8)


def _value(code, sb):
    return E2M1[code] * np.repeat(E4M3[np.minimum(sb, 126)], 16, -1)


def _set(pages, slot, h, kq, vq):
    """Puts one key's and value's codes into a pool, byte by byte as include/apa.h lays it out."""
    d = len(kq[0])
    i, base = slot % 64 % 16, slot % 64 // 16 * 18 * d
    at = pages[slot // 64, h, base:base + 18 * d]
    for x in range(d // 2):
        at[i * (d // 2) + x] = kq[0][2 * x] | kq[0][2 * x + 1] << 4
    for t in range(d // 16):
        for g in range(8):
            at[8 * d + 512 * (t // 4) + 16 * (4 * g + i // 4) + 4 * (t % 4) + i % 4] = \
                vq[0][16 * t + g] | vq[0][16 * t + 8 + g] << 4
        at[16 * d + i * (d // 16) + t] = kq[1][t]
        at[17 * d + 4 * ((i // 4) * (d // 16) + t) + i % 4] = vq[1][t]


def _torch(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def _types():
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ tables
def _tables(old, new, table, free, count, max_tokens):
    """The definition, one page and one token at a time."""
    table, stack = table.copy(), list(free[:count])
    pages = lambda n: (n + 63) // 64  # noqa: E731
    for b in range(len(old)):
        stack += [table[b, e] for e in range(pages(new[b]), pages(old[b]))]
    for b in range(len(old)):
        for e in range(pages(old[b]), pages(new[b])):
            table[b, e] = stack.pop()
    slots, pos, starts = np.full(max_tokens, -1), np.zeros(max_tokens, int), [0]
    for b in range(len(old)):
        for p in range(old[b], new[b]):
            i = starts[b] + p - old[b]
            slots[i], pos[i] = table[b, p // 64] * 64 + p % 64, p
        starts.append(starts[b] + max(0, new[b] - old[b]))
    return slots, pos, np.array(starts), table, stack


def _batch(rng, B, longest, spare):
    old = rng.integers(0, longest + 1, B)
    new = np.clip(old + rng.integers(-longest // 2, longest // 2 + 1, B), 0, longest)
    new = np.where(rng.integers(0, 4, B) == 0, 0, new)
    held = (old + 63) // 64
    P = int(held.sum() + np.maximum((new + 63) // 64 - held, 0).sum()) + spare
    ids = rng.permutation(P)
    most = max(1, (longest + 63) // 64)
    table = np.full((B, most), -5)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = np.full(P, -9)
    free[:P - at] = ids[at:]
    return old, new, table, free, P - at


@pytest.mark.parametrize("B,longest,spare", [(1, 1, 0), (1, 64, 0), (3, 65, 1), (40, 1000, 0), (1024, 200, 7),
                                             (1025, 130, 3), (2048, 70, 1), (2456, 70, 0),
                                             (8192, 70, 0), (5, 30000, 2)])
def test_tables(B, longest, spare):
    import torch

    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(B + longest)
    old, new, table, free, count = _batch(rng, B, longest, spare)
    most = int(np.maximum(new - old, 0).sum()) + 5
    ref = _tables(old, new, table, free, count, most)
    i32 = lambda a: _torch(np.asarray(a, np.int32))  # noqa: E731
    t, f, c = i32(table), i32(free), i32([count])
    for again in range(2):  # the second call gives the same: nothing it reads was changed by the first
        r = apa.cache_tables(i32(old), i32(new), t, f, c, most)
        assert int(r["status"]) == 0
        for name, want in zip(("slots", "positions", "starts"), ref):
            assert np.array_equal(r[name].cpu().numpy(), want), (name, again)
        assert np.array_equal(t.cpu().numpy(), ref[3])
        assert int(r["free_count"]) == len(ref[4]) and int(c) == count
        got = f.cpu().numpy()
        assert np.array_equal(got[:len(ref[4])], ref[4])
        assert np.array_equal(got[len(ref[4]):][max(0, count - len(ref[4])):], free[max(count, len(ref[4])):])
    # in place: the count is input and output
    assert apa.cache_tables(i32(old), i32(new), t, f, c, most, free_count_out=c)["free_count"] is c
    assert int(c) == len(ref[4])
    torch.cuda.synchronize()


def test_tables_refusals_change_nothing():
    import mixed_precision_attention_gb300 as apa
    i32 = lambda a: _torch(np.asarray(a, np.int32))  # noqa: E731
    table, free = np.arange(8).reshape(2, 4), np.array([20, 21, 22, -1, -1])
    for old, new, count, most, status in [
        ([0, -1], [1, 1], 3, 9, 1), ([0, 0], [1, 257], 3, 300, 1), ([0, 300], [1, 1], 3, 9, 1),
        ([0, 0], [5, 5], 3, 9, 2), ([0, 0], [2 ** 31 - 1, 5], 3, 9, 1),
        ([0, 0], [128, 128], 3, 500, 3), ([64, 0], [64, 256], 3, 500, 3),
        ([200, 0], [0, 1], 3, 9, 4), ([0, 0], [1, 1], -1, 9, 4), ([0, 0], [1, 1], 6, 9, 4),
    ]:
        t, f, c = i32(table), i32(free), i32([count])
        r = apa.cache_tables(i32(old), i32(new), t, f, c, most)
        assert int(r["status"]) == status and status in apa.TABLES_STATUS
        assert (r["slots"].cpu().numpy() == -1).all() and not r["positions"].any() and not r["starts"].any()
        assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(f.cpu().numpy(), free)
        assert int(r["free_count"]) == count
    # and with nothing to place, no tokens asked for
    r = apa.cache_tables(i32([3, 0]), i32([3, 0]), i32(table), i32(free), i32([3]), 0)
    assert int(r["status"]) == 0 and r["slots"].numel() == 0 and int(r["free_count"]) == 3


# ------------------------------------------------------------------ write, read
def _tokens(rng, H, T, d, dtype):
    """k, v [H, T, d] with the values where quantizing can go wrong: ties, zeros of both signs, tiny and huge groups."""
    x = rng.standard_normal((2, H, T, d)) * np.exp(rng.standard_normal((2, H, T, d // 16)) * 2).repeat(16, -1)
    if T > 3:
        x[:, :, 0] = np.tile([6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -5, -3.5, -2.5, -1.75, -1.25, -0.75, -0.25, -0.0], d // 16)
        x[:, :, 1] = 0.0
        x[:, :, 2] = -0.0
        x[:, :, 3, :16] = 1e-6
    return [_torch(a, dtype) for a in x]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,H,order", [(1, 1, "any"), (37, 3, "any"), (200, 2, "run"), (16, 1, "run"), (67, 8, "mixed")])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_write_then_read(d, T, H, order, dtype):
    import torch

    import mixed_precision_attention_gb300 as apa
    dt = _types()[dtype]
    rng = np.random.default_rng(T * d)
    P = max(4, (T + 63) // 64 + 2)
    if order == "any":
        slots = rng.permutation(P * 64)[:T]
    else:
        first = 5 if order == "run" else 16
        at = first + np.arange(T)
        slots = rng.permutation(P)[at // 64] * 64 + at % 64
        if order == "mixed":  # runs that end inside blocks, padding among them, and one block backwards
            slots[20:27] = -1
            slots[32:48] = slots[32:48][::-1].copy()
    k, v = _tokens(rng, H, T, d, dt)
    if T == 67:  # a projection's output: tokens first, with another tensor between
        big = torch.zeros(T, 3 * H, d, dtype=dt, device="cuda")
        big[:, H:2 * H], big[:, 2 * H:] = k.transpose(0, 1), v.transpose(0, 1)
        k, v = big[:, H:2 * H].transpose(0, 1), big[:, 2 * H:].transpose(0, 1)
    ks, vs = rng.uniform(0.3, 2, (2, H)).astype(np.float32) / 448
    ks[0] = 1 / 448  # the ties of token 0 stay ties: scale code 448, E2M1 units
    before = rng.integers(0, 256, (P, H, 72 * d), dtype=np.uint8)
    want = before.copy()
    kq, vq = (_quantize(x.double().cpu().numpy(), s[:, None, None]) for x, s in ((k, ks), (v, vs)))
    for t in np.flatnonzero(slots >= 0):
        for h in range(H):
            _set(want, slots[t], h, (kq[0][h, t], kq[1][h, t]), (vq[0][h, t], vq[1][h, t]))
    pages = _torch(before)
    s32 = _torch(np.asarray(slots, np.int32))
    apa.cache_write(k, v, s32, pages, _torch(ks), _torch(vs))
    apa.check_error()
    assert np.array_equal(pages.cpu().numpy(), want)  # every other byte as it was
    rk, rv = apa.cache_read(pages, s32, _torch(ks), _torch(vs), dtype=dt)
    for got, q, s in ((rk, kq, ks), (rv, vq, vs)):
        ref = np.where((slots >= 0)[None, :, None], _value(*q).astype(np.float32) * s[:, None, None], np.float32(0))
        assert torch.equal(got, _torch(ref, dt))  # one rounding of the same FP32 value


def test_write_and_read_bad_slots():
    import torch

    import mixed_precision_attention_gb300 as apa
    k = torch.ones(1, 3, 64, dtype=torch.bfloat16, device="cuda")
    s = torch.ones(1, device="cuda")
    pages = apa.cache_pages(2, 1, 64)
    slots = _torch(np.array([128, -1, 2 ** 31 - 1], np.int32))
    apa.cache_write(k, k, slots, pages, s, s)
    with pytest.raises(apa.ApaError):
        apa.check_error()
    assert not pages.any()
    rk, rv = apa.cache_read(pages, slots, s, s)
    with pytest.raises(apa.ApaError):
        apa.check_error()
    assert not rk.any() and not rv.any()
    apa.cache_write(k[:, :0], k[:, :0], slots[:0], pages, s, s)  # no tokens
    assert apa.cache_read(pages, slots[:0], s, s)[0].shape == (1, 0, 64)
    apa.check_error()


# ------------------------------------------------------------------ attention
def _cache(rng, B, H, d, lens, most, junk=0x7F):
    """Pool, table, and the values [B, H, n, d] of each sequence (without the head scales).  What is behind a
    sequence's end, and every unused page, holds NaN scales."""
    import torch

    import mixed_precision_attention_gb300 as apa
    held = [(n + 63) // 64 for n in lens]
    P = sum(held) + 2
    ids = rng.permutation(P)
    table = np.full((B, most), -3, np.int32)
    pages = np.full((P, H, 72 * d), junk, np.uint8)
    pages = _torch(pages)
    ks, vs = rng.uniform(0.5, 2, (2, H)).astype(np.float32) / 500
    kv, at = [], 0
    for b, n in enumerate(lens):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
        x = rng.standard_normal((2, H, n, d)).astype(np.float32)
        x[0] += 1.5 * rng.standard_normal((H, 1, d))
        slots = table[b, np.arange(n) // 64] * 64 + np.arange(n) % 64
        k, v = (_torch(a, torch.bfloat16) for a in x)
        apa.cache_write(k, v, _torch(slots.astype(np.int32)), pages, _torch(ks), _torch(vs))
        kv.append([_value(*_quantize(a.double().cpu().numpy(), s[:, None, None])) * s[:, None, None].astype(np.float64)
                   for a, s in ((k, ks), (v, vs))])
    return pages, _torch(table), ks, vs, kv


def _attend(q, kv, lens, window, sinks):
    """64-bit attention, and sum_j w_j |v_j| of each output."""
    B, Hq, Nq, d = q.shape
    out, lse, mag = np.zeros(q.shape), np.full((B, Hq, Nq), -np.inf), np.zeros(q.shape)
    for b, n in enumerate(lens):
        k, v = kv[b]
        G = Hq // k.shape[0]
        for i in range(Nq):
            p = n - Nq + i
            j = np.arange(max(0, p + 1))
            j = j[(j > p - window) | (j < sinks)] if window else j
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


def _near(out, lse, ref, dtype):
    step = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    o, r = out.double().cpu().numpy(), ref
    assert np.all(np.abs(o - r[0]) <= np.abs(r[0]) * step + r[2] * (2.0 ** -11 + 2.0 ** -14) + 2.0 ** -25), np.abs(o - r[0]).max()
    got = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(got), np.isneginf(r[1]))
    fin = np.isfinite(r[1])
    assert np.all(np.abs(got[fin] - r[1][fin]) <= 1e-5 * np.maximum(1, np.abs(r[1][fin])))


SHAPES = [  # B, Hq, Hkv, Nq, d, lens, window, sinks
    (1, 1, 1, 1, 64, [1], 0, 0),
    (1, 3, 1, 1, 128, [16], 0, 0),
    (2, 6, 2, 1, 128, [0, 17], 0, 0),
    (4, 8, 2, 1, 64, [63, 64, 65, 1000], 0, 0),
    (3, 8, 1, 1, 256, [31, 33, 700], 0, 0),
    (2, 5, 1, 3, 128, [2, 129], 0, 0),          # rows before the first key see nothing
    (2, 8, 2, 4, 128, [4, 300], 0, 0),          # 16 rows
    (1, 24, 2, 3, 64, [777], 0, 0),             # 36 rows: more than one row block
    (1, 16, 1, 2, 256, [333], 0, 0),            # 32 rows at d = 256
    (1, 40, 1, 1, 128, [4100], 0, 0),
    (2, 4, 2, 1, 64, [1000, 90], 1, 0),         # only itself
    (2, 4, 2, 1, 64, [1000, 90], 32, 0),
    (2, 4, 1, 5, 128, [1500, 7], 100, 4),
    (3, 4, 1, 2, 128, [1500, 200, 50], 129, 70),
    (1, 6, 2, 3, 256, [900], 200, 33),
    (1, 2, 1, 1, 128, [640], 5000, 3),
    (1, 2, 1, 4, 64, [3000], 7, 2999),          # the sinks reach into the window
    (300, 2, 1, 1, 64, None, 0, 0),
]


@pytest.mark.parametrize("case", range(len(SHAPES)))
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_attention_cache(case, dtype):
    import mixed_precision_attention_gb300 as apa
    B, Hq, H, Nq, d, lens, window, sinks = SHAPES[case]
    rng = np.random.default_rng(case)
    lens = rng.integers(0, 150, B) if lens is None else lens
    pages, table, ks, vs, kv = _cache(rng, B, H, d, lens, max(lens) // 64 + 2)
    q = _torch(rng.standard_normal((B, Hq, Nq, d)) * 2, _types()[dtype])
    ref = _attend(q.double().cpu().numpy(), kv, lens, window, sinks)
    n32 = _torch(np.asarray(lens, np.int32))
    out, lse = apa.attention_cache(q, pages, table, n32, _torch(ks), _torch(vs), window=window, sinks=sinks)
    apa.check_error()
    _near(out, lse, ref, dtype)
    # a strided q (rows before heads), no lse, and bitwise the same again
    qt = q.transpose(1, 2).contiguous().transpose(1, 2)
    again, none = apa.attention_cache(qt, pages, table, n32, _torch(ks), _torch(vs), window=window, sinks=sinks,
                                      return_lse=False)
    assert none is None and (again == out).all()


def test_attention_cache_long_and_uneven():
    # one long sequence among short ones: its keys are split over the GPU and joined
    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(5)
    B, Hq, H, Nq, d = 6, 6, 2, 1, 128
    lens = [20011, 1, 130, 0, 4096, 77]
    pages, table, ks, vs, kv = _cache(rng, B, H, d, lens, 400)
    q = _torch(rng.standard_normal((B, Hq, Nq, d)) * 3, _types()["bf16"])
    out, lse = apa.attention_cache(q, pages, table, _torch(np.asarray(lens, np.int32)), _torch(ks), _torch(vs))
    apa.check_error()
    _near(out, lse, _attend(q.double().cpu().numpy(), kv, lens, 0, 0), "bf16")


def test_attention_cache_extreme_scores():
    # scores that grow along the sequence by far more than FP16 spans, and ones of -1e4 and below
    import torch

    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(8)
    n, d = 700, 64
    k = np.zeros((1, n, d), np.float32)
    k[0, :, 0] = np.linspace(-6, 6, n) * 400
    k[0, :, 16:] = rng.standard_normal((n, d - 16))
    v = rng.standard_normal((1, n, d)).astype(np.float32)
    one = np.ones(1, np.float32)
    pages = apa.cache_pages(11, 1, d)
    slots = _torch(np.arange(n, dtype=np.int32))
    kt, vt = _torch(k, torch.bfloat16), _torch(v, torch.bfloat16)
    apa.cache_write(kt, vt, slots, pages, _torch(one), _torch(one / 448))
    kv = [[_value(*_quantize(kt.double().cpu().numpy(), one[:, None, None])),
           _value(*_quantize(vt.double().cpu().numpy(), one[:, None, None] / 448)) * np.float64(one[0] / np.float32(448))]]
    q = np.zeros((1, 4, 1, d))
    q[0, :, 0, 0] = [1, -1, 30, 0]
    q[0, 3] = rng.standard_normal(d)
    qt = _torch(q, torch.bfloat16)
    table = _torch(np.arange(11, dtype=np.int32)[None])
    out, lse = apa.attention_cache(qt, pages, table, _torch(np.array([n], np.int32)), _torch(one), _torch(one / np.float32(448)))
    ref = _attend(qt.double().cpu().numpy(), kv, [n], 0, 0)
    _near(out, lse, ref, "bf16")


def test_attention_cache_bad_lengths_and_pages():
    import torch

    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(1)
    lens = [100, 64]
    pages, table, ks, vs, kv = _cache(rng, 2, 1, 64, lens, 2, junk=0)
    q = torch.randn(2, 2, 1, 64, device="cuda").bfloat16()
    args = (_torch(ks), _torch(vs))
    good, _ = apa.attention_cache(q, pages, table, _torch(np.array(lens, np.int32)), *args)
    apa.check_error()
    # a length beyond the table is clamped to it, a negative one is empty; both are reported
    out, lse = apa.attention_cache(q, pages, table[:, :1].contiguous(), _torch(np.array([1 << 30, -4], np.int32)), *args)
    with pytest.raises(apa.ApaError):
        apa.check_error()
    assert not out[1].any() and torch.isneginf(lse[1]).all() and torch.isfinite(out).all()
    # a bad page reads page 0 and is reported; the other sequence is not touched by it
    t = table.clone()
    t[0, 1] = pages.shape[0]
    out, _ = apa.attention_cache(q, pages, t, _torch(np.array(lens, np.int32)), *args)
    with pytest.raises(apa.ApaError):
        apa.check_error()
    assert torch.equal(out[1], good[1]) and torch.isfinite(out).all()
    apa.check_error()


# ------------------------------------------------------------------ together
def test_serving_loop_in_a_graph():
    """Tables, write and attention of one decoding step, captured once and replayed as lengths grow, on a stream of
    its own, against the formulas at each step."""
    import torch

    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(3)
    B, Hq, H, d, steps = 3, 6, 2, 128, 5
    lens = np.array([62, 127, 0])
    free = _torch(np.arange(16, dtype=np.int32)[::-1].copy())
    count = _torch(np.array([16], np.int32))
    table = _torch(np.full((B, 4), -1, np.int32))
    pages = apa.cache_pages(16, H, d)
    ks, vs = (np.full(H, 4 / 2688, np.float32) for _ in range(2))
    old, new = _torch(np.zeros(B, np.int32)), _torch(lens.astype(np.int32))
    t = apa.cache_tables(old, new, table, free, count, int(lens.sum()), free_count_out=count)
    hist = [[rng.standard_normal((H, n, d)).astype(np.float32) for n in lens] for _ in range(2)]
    k, v = (_torch(np.concatenate(x, 1), torch.bfloat16) for x in hist)
    apa.cache_write(k, v, t["slots"], pages, _torch(ks), _torch(vs))
    hist = [[_torch(a, torch.bfloat16).double().cpu().numpy() for a in x] for x in hist]

    kn, vn = (torch.zeros(H, B, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(B, Hq, 1, d, dtype=torch.bfloat16, device="cuda")
    kst, vst = _torch(ks), _torch(vs)

    def step():
        old.copy_(new)
        new.add_(1)
        s = apa.cache_tables(old, new, table, free, count, B, free_count_out=count)
        apa.cache_write(kn, vn, s["slots"], pages, kst, vst)
        return apa.attention_cache(q, pages, table, new, kst, vst)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out, lse = step()
    for i in range(steps):
        x = rng.standard_normal((2, H, B, d))
        kn.copy_(_torch(x[0], torch.bfloat16))
        vn.copy_(_torch(x[1], torch.bfloat16))
        q.copy_(_torch(rng.standard_normal(q.shape) * 2, torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        apa.check_error()
        lens = lens + 1
        for n, a in enumerate((kn, vn)):
            a = a.double().cpu().numpy()
            hist[n] = [np.concatenate([hist[n][b], a[:, b:b + 1]], 1) for b in range(B)]
        assert np.array_equal(new.cpu().numpy(), lens)
        kv = [[_value(*_quantize(hist[n][b], s[:, None, None])) * s[:, None, None].astype(np.float64)
               for n, s in ((0, ks), (1, vs))] for b in range(B)]
        _near(out, lse, _attend(q.double().cpu().numpy(), kv, lens, 0, 0), "bf16")
    held = int(sum((n + 63) // 64 for n in lens))
    assert int(count) == 16 - held


def test_a_cached_prefix_feeds_prefill():
    """cache_read's layout is attention()'s: a chunk of queries over a prefix taken out of the cache."""
    import torch

    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(4)
    H, d, n, Nq = 2, 64, 200, 40
    pages, table, ks, vs, kv = _cache(rng, 1, H, d, [n], 4)
    slots = table[0, torch.arange(n, device="cuda") // 64] * 64 + torch.arange(n, device="cuda", dtype=torch.int32) % 64
    k, v = apa.cache_read(pages, slots.to(torch.int32), _torch(ks), _torch(vs))
    q = _torch(rng.standard_normal((1, 4, Nq, d)), torch.bfloat16)
    out, _, _ = apa.attention(q, k[None], v[None], eps=0.0)
    ref, _, _ = _attend(q.double().cpu().numpy(), [[x.double().cpu().numpy() for x in (k, v)]], [n], 0, 0)
    assert np.abs(out.cpu().numpy() - ref).max() <= 4e-3  # attention()'s own bound at eps = 0


@pytest.mark.parametrize("B,Hq,H,Nq,d", [(8192, 1, 1, 1, 64), (3000, 4, 1, 4, 256), (8192, 8, 1, 4, 128)])
def test_attention_cache_many_sequences(B, Hq, H, Nq, d):
    # as many sequences as the calls allow, most of them empty; the rest share their pages
    import torch

    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(B + d)
    n0 = 40
    pages, table, ks, vs, kv = _cache(rng, 1, H, d, [n0], 1)
    lens = np.where(rng.integers(0, 8, B) == 0, rng.integers(1, n0 + 1, B), 0)
    lens[-1] = n0
    q = _torch(rng.standard_normal((B, Hq, Nq, d)), torch.bfloat16)
    out, lse = apa.attention_cache(q, pages, table.expand(B, 1).contiguous(), _torch(lens.astype(np.int32)), _torch(ks),
                                   _torch(vs))
    apa.check_error()
    some = np.concatenate([np.flatnonzero(lens)[:20], np.flatnonzero(lens == 0)[:5], [B - 1]])
    ref = _attend(q[some].double().cpu().numpy(), [[x[:, :lens[b]] for x in kv[0]] for b in some], lens[some], 0, 0)
    _near(out[some], lse[some], ref, "bf16")
    empty = _torch(lens == 0)
    assert not out[empty].any() and torch.isneginf(lse[empty]).all()


def test_bindings_refuse_what_does_not_fit():
    import torch

    import mixed_precision_attention_gb300 as apa
    dev = "cuda"
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)  # noqa: E731
    f32 = torch.ones(2, device=dev)
    k = torch.zeros(2, 3, 64, dtype=torch.bfloat16, device=dev)
    pages, q = apa.cache_pages(3, 2, 64), torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device=dev)
    refused = [
        lambda: apa.cache_tables(i32(2), i32(3), i32(2, 4), i32(5), i32(1), 4),
        lambda: apa.cache_tables(i32(2), i32(2), i32(3, 4), i32(5), i32(1), 4),
        lambda: apa.cache_tables(i32(2), i32(2), i32(2, 4), i32(5), i32(2), 4),
        lambda: apa.cache_tables(i32(2), i32(2), i32(4, 2).t(), i32(5), i32(1), 4),
        lambda: apa.cache_tables(i32(2), i32(2), i32(2, 4), i32(5), i32(1), -1),
        lambda: apa.cache_write(k, k[:, :2], i32(3), pages, f32, f32),
        lambda: apa.cache_write(k, k.half(), i32(3), pages, f32, f32),
        lambda: apa.cache_write(k, k, i32(2), pages, f32, f32),
        lambda: apa.cache_write(k, k, i32(3), apa.cache_pages(3, 1, 64), f32[:1], f32[:1]),
        lambda: apa.cache_write(k, k, i32(3), apa.cache_pages(3, 2, 128), f32, f32),
        lambda: apa.cache_write(k, k, i32(3), pages, f32[:1], f32),
        lambda: apa.cache_write(k.transpose(1, 2), k.transpose(1, 2), i32(64), pages, f32, f32),
        lambda: apa.cache_read(pages[:, :, :100].contiguous(), i32(3), f32, f32),
        lambda: apa.attention_cache(q, pages, i32(3, 4), i32(2), f32, f32),
        lambda: apa.attention_cache(q, pages, i32(2, 4), i32(3), f32, f32),
        lambda: apa.attention_cache(q, apa.cache_pages(3, 2, 128), i32(2, 4), i32(2), f32, f32),
        lambda: apa.attention_window(q, k[None], k[None], 4),
    ]
    for i, call in enumerate(refused):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    with pytest.raises(TypeError):
        apa.attention_cache(q.float(), pages, i32(2, 4), i32(2), f32, f32)
    with pytest.raises(TypeError):
        apa.attention_cache(q, pages, i32(2, 4).long(), i32(2), f32, f32)
    with pytest.raises(TypeError):
        apa.cache_read(pages, i32(3), f32, f32, dtype=torch.float32)
    for window, sinks in ((-1, 0), (4, -1)):
        with pytest.raises(apa.ApaError):
            apa.attention_cache(q, pages, i32(2, 4), i32(2), f32, f32, window=window, sinks=sinks)
    with pytest.raises(apa.ApaError):  # rows that do not start on 16 bytes
        wide = torch.zeros(2, 4, 1, 68, dtype=torch.bfloat16, device=dev)
        apa.attention_cache(wide[..., :64], pages, i32(2, 4), i32(2), f32, f32)
    need = apa.attention_cache_workspace_bytes(2, 4, 2, 1, 64)
    with pytest.raises(apa.ApaError):
        apa.attention_cache(q, pages, i32(2, 4), i32(2), f32, f32, workspace=torch.zeros(need - 1, dtype=torch.uint8, device=dev))
    ws = torch.zeros(need, dtype=torch.uint8, device=dev)
    out, lse = apa.attention_cache(q, pages, i32(2, 4), i32(2), f32, f32, workspace=ws)
    assert not out.any() and torch.isneginf(lse).all()


def test_two_streams_at_once():
    """Two sequences' writes and attention on two streams, interleaved: each has its own workspace and pages."""
    import torch

    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(12)
    args, want = [], []
    for d in (64, 128):
        pages, table, ks, vs, _ = _cache(rng, 3, 2, d, [700, 64, 1], 12)
        q = _torch(rng.standard_normal((3, 6, 2, d)), torch.bfloat16)
        args.append((q, pages, table, _torch(np.array([700, 64, 1], np.int32)), _torch(ks), _torch(vs)))
        want.append(apa.attention_cache(*args[-1]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(apa.attention_cache(*args[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])
    apa.check_error()


def test_numbers_past_32_bits_keep_their_meaning():
    """A window or sinks past 2^32 reach over every key (and are not their low 32 bits); a negative one is refused."""
    import torch

    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(13)
    pages, table, ks, vs, _ = _cache(rng, 1, 2, 64, [300], 6)
    q = _torch(rng.standard_normal((1, 4, 2, 64)), torch.bfloat16)
    args = (q, pages, table, _torch(np.array([300], np.int32)), _torch(ks), _torch(vs))
    want = apa.attention_cache(*args)
    kv = [_torch(rng.standard_normal((1, 2, 300, 64)), torch.bfloat16) for _ in range(2)]
    full = apa.attention_window(q, *kv, 300)
    for window, sinks in ((2**32 + 1, 0), (2**31, 0), (1, 2**32), (1, 2**31 + 5)):
        assert all(torch.equal(a, b) for a, b in zip(apa.attention_cache(*args, window=window, sinks=sinks), want))
        assert all(torch.equal(a, b) for a, b in zip(apa.attention_window(q, *kv, window, sinks), full))
    for window, sinks in ((-2**32 + 5, 0), (4, -2**32)):
        with pytest.raises(apa.ApaError):
            apa.attention_cache(*args, window=window, sinks=sinks)
        with pytest.raises(apa.ApaError):
            apa.attention_window(q, *kv, window, sinks)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    with pytest.raises(ValueError):
        apa.cache_tables(i32(1), i32(1), i32(1, 1), i32(1), i32(1), 2**32 + 1)
