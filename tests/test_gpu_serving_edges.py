"""The serving operators at the borders of what their documentation allows: rows and scales whose products leave
FP32's range, values that are no numbers, axes of one element, long lists, two streams.  References and
tolerances are those of tests/test_gpu_cache.py."""
import math

import numpy as np
import pytest

from tests.test_gpu_cache import _attend, _cache, _near, _quantize, _set, _tables, _torch, _types, _value

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ the score's factor at the ends of its range
@pytest.mark.parametrize("d,Hq,Nq,lens,window,sinks", [
    (64, 4, 1, [33, 1, 64], 0, 0), (128, 4, 1, [45, 300], 0, 0), (256, 4, 1, [7, 95], 0, 0),
    (128, 4, 4, [2, 131], 0, 0),             # rows before the first key, row blocks of 16
    (64, 8, 5, [200, 3], 50, 3), (128, 4, 1, [1500], 40, 2)])
@pytest.mark.parametrize("k_scale", [2.0 ** -100, 1e-12, 1e-10, 2.0 ** 20])
def test_rows_of_zeros_under_any_key_scale(d, Hq, Nq, lens, window, sinks, k_scale):
    """Every key zero, so each row's weights are equal whatever its values: out is the mean of V over the keys it sees and
    lse the logarithm of their number.  Rows of zeros, of tiny and of huge values."""
    import torch

    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(len(lens) + d)
    B, H = len(lens), Hq // 4
    pages, table, ks, vs, kv = _cache(rng, B, H, d, lens, max(lens) // 64 + 2)
    for b, n in enumerate(lens):  # the same values, under keys of zeros
        slots = table[b, torch.arange(n, device="cuda") // 64] * 64 + torch.arange(n, device="cuda", dtype=torch.int32) % 64
        _, v = apa.cache_read(pages, slots.to(torch.int32), _torch(ks), _torch(vs), dtype=torch.bfloat16)
        apa.cache_write(torch.zeros_like(v), v, slots.to(torch.int32), pages, _torch(ks), _torch(vs))
        kv[b][0][:] = 0
        q8 = _quantize(v.double().cpu().numpy(), vs[:, None, None])
        kv[b][1] = _value(*q8) * vs[:, None, None].astype(np.float64)
    ks = np.full(H, k_scale, np.float32)
    q = rng.standard_normal((B, Hq, Nq, d))
    q[:, 0::4] = 0
    q[:, 1::4] *= 2.0 ** -120
    q[:, 2::4, :, 1:] = 0
    q[:, 2::4, :, 0] = 2.0 ** 126
    qt = _torch(q, torch.bfloat16)
    out, lse = apa.attention_cache(qt, pages, table, _torch(np.asarray(lens, np.int32)), _torch(ks), _torch(vs), window=window,
                                   sinks=sinks)
    apa.check_error()
    _near(out, lse, _attend(qt.double().cpu().numpy(), kv, lens, window, sinks), "bf16")


# ------------------------------------------------------------------ values that are no numbers
def _with_nonfinite(rng, H, T, d, dtype):
    """k, v [H, T, d] of which some groups of 16 hold a NaN (one, or all 16), some infinities, some both."""
    import torch
    x = rng.standard_normal((2, H, T, d))
    x[0, 0, 1, 3] = x[1, 0, 2, 17] = np.nan
    x[0, H - 1, 3, 16:32] = x[1, H - 1, 3, 48:64] = np.nan
    x[0, 0, 5, 40], x[1, 0, 5, 41] = np.inf, -np.inf
    x[0, 0, T - 1, :2], x[1, 0, T - 1, :2] = (np.nan, np.inf), (-np.inf, np.nan)
    return [_torch(a, dtype) for a in x]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("order", ["run", "any"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_a_nan_stays_one_and_infinities_saturate(d, order, dtype):
    """A NaN makes its group of 16 NaN (scale code 0x7F, codes 0) and no other; an infinity is the largest value."""
    import torch

    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(d)
    H, T, P, dt = 2, 23, 4, _types()[dtype]
    slots = 64 + 4 + np.arange(T) if order == "run" else rng.permutation(P * 64)[:T]
    k, v = _with_nonfinite(rng, H, T, d, dt)
    ks, vs = rng.uniform(0.3, 2, (2, H)).astype(np.float32) / 448
    want = rng.integers(0, 256, (P, H, 72 * d), dtype=np.uint8)
    pages = _torch(want.copy())
    values = []
    quantized = []
    for x, s in ((k, ks), (v, vs)):
        a = x.double().cpu().numpy()
        nan = np.isnan(a).reshape(H, T, d // 16, 16).any(-1)
        code, sb = _quantize(np.where(nan.repeat(16, -1), 0, a), s[:, None, None])
        assert (sb[np.isinf(a).reshape(H, T, d // 16, 16).any(-1) & ~nan] == 126).all()
        sb[nan] = 0x7F
        quantized.append((code, sb))
        # (_value takes the code 0x7F for the largest scale)
        values.append(np.where(nan.repeat(16, -1), np.nan, _value(code, sb).astype(np.float32) * s[:, None, None]))
    for t in range(T):
        for h in range(H):
            _set(want, slots[t], h, *[(c[h, t], sb[h, t]) for c, sb in quantized])
    s32 = _torch(slots.astype(np.int32))
    apa.cache_write(k, v, s32, pages, _torch(ks), _torch(vs))
    apa.check_error()
    assert np.array_equal(pages.cpu().numpy(), want)
    for got, ref in zip(apa.cache_read(pages, s32, _torch(ks), _torch(vs), dtype=dt), values):
        ref = _torch(ref.astype(np.float32)).to(dt)
        assert torch.equal(got.isnan(), ref.isnan()) and torch.equal(got.nan_to_num(0), ref.nan_to_num(0))


@pytest.mark.parametrize("d,Hq,Nq,n,window,sinks,bad", [
    (64, 2, 1, 130, 20, 0, [96, 109]),       # in the half page in which the window starts
    (128, 6, 1, 200, 70, 5, [5, 31, 129]),   # behind the sinks; before the window
    (256, 2, 1, 190, 29, 2, [2, 160]),
    (128, 4, 3, 310, 40, 33, [33, 63, 267]),
    (64, 40, 1, 100, 3, 1, [1, 96]),         # more than one row block
    (64, 1, 1, 40, 1, 0, [32, 38])])
def test_a_nan_that_no_row_sees(d, Hq, Nq, n, window, sinks, bad):
    """Keys between the sinks and the window, NaN in every channel of K and V, in units that the rows do read."""
    import torch

    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(n)
    pages, table, ks, vs, kv = _cache(rng, 1, 1, d, [n], n // 64 + 2)
    first = n - Nq
    assert all(sinks <= j <= first - window for j in bad)
    slots = (table[0, torch.tensor(bad, device="cuda") // 64] * 64 + torch.tensor(bad, device="cuda", dtype=torch.int32) % 64)
    x = torch.full((1, len(bad), d), math.nan, dtype=torch.bfloat16, device="cuda")
    apa.cache_write(x, x, slots.to(torch.int32), pages, _torch(ks), _torch(vs))
    q = _torch(rng.standard_normal((1, Hq, Nq, d)) * 2, torch.bfloat16)
    out, lse = apa.attention_cache(q, pages, table, _torch(np.array([n], np.int32)), _torch(ks), _torch(vs), window=window,
                                   sinks=sinks)
    apa.check_error()
    _near(out, lse, _attend(q.double().cpu().numpy(), kv, [n], window, sinks), "bf16")
    # with the window open it is seen, by every row
    out, lse = apa.attention_cache(q, pages, table, _torch(np.array([n], np.int32)), _torch(ks), _torch(vs))
    assert out.isnan().all() and lse.isnan().all()


@pytest.mark.parametrize("d,Hq", [(64, 32), (128, 32), (256, 16)])
@pytest.mark.parametrize("n,window,sinks", [(130, 20, 0), (229, 100, 7), (97, 1, 3)])
def test_a_nan_that_later_rows_do_not_see(d, Hq, n, window, sinks):
    """As many heads as a row block has rows, so that each position is a block of its own: the key with which the first
    row's window starts is hidden from the other two, and a NaN there stays out of their outputs."""
    import torch

    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(n + d)
    Nq, bad = 3, n - 3 - window + 1
    pages, table, ks, vs, kv = _cache(rng, 1, 1, d, [n], n // 64 + 2)
    x = torch.full((1, 1, d), math.nan, dtype=torch.bfloat16, device="cuda")
    apa.cache_write(x, x, table[0, bad // 64].view(1) * 64 + bad % 64, pages, _torch(ks), _torch(vs))
    q = _torch(rng.standard_normal((1, Hq, Nq, d)) * 2, torch.bfloat16)
    out, lse = apa.attention_cache(q, pages, table, _torch(np.array([n], np.int32)), _torch(ks), _torch(vs), window=window,
                                   sinks=sinks)
    apa.check_error()
    ref = _attend(q.double().cpu().numpy(), kv, [n], window, sinks)
    _near(out[:, :, 1:], lse[:, :, 1:], [r[:, :, 1:] for r in ref], "bf16")
    assert out[:, :, 0].isnan().all() and lse[:, :, 0].isnan().all()


# ------------------------------------------------------------------ axes of one element
def test_strides_of_axes_of_length_one_do_not_matter():
    """They are never used, so any value of theirs is taken: here 1, 3 and 5 elements."""
    import torch

    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(2)
    d = 64
    pages, table, ks, vs, _ = _cache(rng, 1, 1, d, [70], 3)
    s = (_torch(ks), _torch(vs))
    n = _torch(np.array([70], np.int32))
    q = _torch(rng.standard_normal((1, 1, 1, d)), torch.bfloat16)
    want = apa.attention_cache(q, pages, table, n, *s)
    got = apa.attention_cache(q.as_strided(q.shape, (1, 3, 5, 1)), pages, table, n, *s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # one row of many heads, as a view that puts the row's axis last makes it
    q = _torch(rng.standard_normal((1, 3, 1, d)), torch.bfloat16)
    want = apa.attention_cache(q, pages, table, n, *s)
    got = apa.attention_cache(q.reshape(1, 3, d, 1).transpose(2, 3), pages, table, n, *s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))

    k, v = (_torch(rng.standard_normal((1, 1, d)), torch.bfloat16) for _ in range(2))
    slot = _torch(np.array([77], np.int32))
    a, b = pages.clone(), pages.clone()
    apa.cache_write(k, v, slot, a, *s)
    apa.cache_write(k.as_strided(k.shape, (1, 5, 1)), v.as_strided(v.shape, (3, 1, 1)), slot, b, *s)
    assert torch.equal(a, b) and not torch.equal(a, pages)
    apa.check_error()
    # those of longer axes do
    two = torch.zeros(200, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(apa.ApaError):
        apa.attention_cache(two.as_strided((1, 2, 1, d), (1, 68, 3, 1)), pages, table, n, *s)
    with pytest.raises(apa.ApaError):
        apa.cache_write(two.as_strided((1, 2, d), (1, 68, 1)), two.as_strided((1, 2, d), (1, 68, 1)),
                        _torch(np.array([3, 4], np.int32)), pages, *s)


# ------------------------------------------------------------------ long lists
@pytest.mark.parametrize("most", [8192, 8193, 20001])
def test_tables_that_are_refused_fill_every_slot(most):
    """Statuses of calls on both sides of 8192 tokens: every slot -1, every position 0, nothing changed."""
    import mixed_precision_attention_gb300 as apa
    i32 = lambda a: _torch(np.asarray(a, np.int32))  # noqa: E731
    pages = most // 64 + 3
    table, free = np.full((2, pages), -7), np.arange(pages + 1)
    table[0, :3] = [900, 901, 902]
    for old, new, count, status in [
        ([0, -1], [1, 1], 3, 1), ([0, 0], [1, 64 * pages + 1], 3, 1), ([0, 0], [most, 1], pages, 2),
        ([0, 0], [most, 0], 2, 3), ([129, 0], [0, most - 1], 0, 3), ([192, 0], [0, 1], pages, 4), ([0, 0], [1, 1], pages + 2, 4),
    ]:
        t, f, c = i32(table), i32(free), i32([count])
        r = apa.cache_tables(i32(old), i32(new), t, f, c, most)
        assert int(r["status"]) == status
        assert (r["slots"] == -1).all() and not r["positions"].any() and not r["starts"].any()
        assert r["slots"].numel() == most and int(r["free_count"]) == count
        assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(f.cpu().numpy(), free)


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("most", [8193, 9002, 9003])
def test_tables_of_many_tokens_into_any_buffers(most, shift):
    """The C entry point's slots and positions need not start on 16 bytes, nor their count be a multiple of 4."""
    import torch

    import mixed_precision_attention_gb300 as apa
    from mixed_precision_attention_gb300 import _lib
    i32 = lambda a: _torch(np.asarray(a, np.int32))  # noqa: E731
    rng = np.random.default_rng(most)
    old, new = np.array([0, 70, 5, 64, 3]), np.array([3001, 71, 5, 0, 6000 - 6])
    held = (old + 63) // 64
    ids = rng.permutation(400)
    table, at = np.full((5, 100), -1), 0
    for b in range(5):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = np.full(400, -1)
    free[:400 - at] = ids[at:]
    if int(np.maximum(new - old, 0).sum()) > most:
        new[4] = most - 3002 + 3
    ref = _tables(old, new, table, free, 400 - at, most)
    t, f, c, o, n = i32(table), i32(free), i32([400 - at]), i32(old), i32(new)
    slots, pos = (torch.full((most + 8,), 77, dtype=torch.int32, device="cuda") for _ in range(2))
    starts, status = torch.empty(6, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    st = _lib.load().apa_cache_tables(o.data_ptr(), n.data_ptr(), 5, t.data_ptr(), 100, f.data_ptr(), 400, c.data_ptr(), most,
                                      slots[shift:].data_ptr(), pos[shift:].data_ptr(), starts.data_ptr(), c.data_ptr(),
                                      status.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == 0 and int(status) == 0
    for got, want in ((slots, ref[0]), (pos, ref[1])):
        got = got.cpu().numpy()
        assert np.array_equal(got[shift:shift + most], want) and (got[:shift] == 77).all() and (got[shift + most:] == 77).all()
    assert np.array_equal(starts.cpu().numpy(), ref[2]) and np.array_equal(t.cpu().numpy(), ref[3])
    assert int(c) == len(ref[4]) and np.array_equal(f.cpu().numpy()[:len(ref[4])], ref[4])
    apa.check_error()


def test_one_long_sequence_among_many_rows():
    """More than 1216 rows, so one warp joins a row, and a sequence that more than 32 CTAs hold parts of."""
    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(9)
    B, d, n = 1301, 64, 42001
    pages, table, ks, vs, kv = _cache(rng, 1, 1, d, [n], n // 64 + 1)
    lens = rng.integers(0, 33, B)  # a unit each, of the first page
    lens[700] = n
    assert n / 32 / ((n / 32 + B) / 152) > 64
    q = _torch(rng.standard_normal((B, 1, 1, d)) * 2, _types()["bf16"])
    out, lse = apa.attention_cache(q, pages, table.expand(B, -1).contiguous(), _torch(lens.astype(np.int32)), _torch(ks), _torch(vs))
    apa.check_error()
    some = np.array([0, 1, 699, 700, 701, 1300])
    ref = _attend(q[some].double().cpu().numpy(), [[x[:, :lens[b]] for x in kv[0]] for b in some], lens[some], 0, 0)
    _near(out[some], lse[some], ref, "bf16")


# ------------------------------------------------------------------ two streams
def test_every_operator_on_two_streams_at_once():
    """Tables, writes, reads and both attentions on two streams, interleaved, each with a pool, tables and lists of its own,
    against the same calls one after the other."""
    import torch

    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(21)
    i32 = lambda a: _torch(np.asarray(a, np.int32))  # noqa: E731

    def state(d, T, H):
        x = [_torch(rng.standard_normal((H, T, d)), torch.bfloat16) for _ in range(2)]
        return {"d": d, "T": T, "H": H, "kv": x, "s": [torch.full((H,), 4 / 2688, device="cuda") for _ in range(2)],
                "q": _torch(rng.standard_normal((2, 2 * H, 3, d)), torch.bfloat16),
                "qw": _torch(rng.standard_normal((1, 2 * H, 150, d)), torch.bfloat16)}

    def loop(st):
        d, T, H = st["d"], st["T"], st["H"]
        pages = apa.cache_pages(2 * (T // 64 + 2), H, d)
        table = torch.full((2, T // 64 + 2), -1, dtype=torch.int32, device="cuda")
        free, count = torch.arange(pages.shape[0], dtype=torch.int32, device="cuda"), torch.full((1,), pages.shape[0], dtype=torch.int32, device="cuda")
        got = []
        old = torch.zeros(2, dtype=torch.int32, device="cuda")
        for new in st["lens"]:
            t = apa.cache_tables(old, new, table, free, count, T, free_count_out=count)
            apa.cache_write(*st["kv"], t["slots"], pages, *st["s"])
            k, v = apa.cache_read(pages, t["slots"], *st["s"])
            got += [t["slots"], k, v, *apa.attention_cache(st["q"], pages, table, new, *st["s"], window=90, sinks=3)]
            got += apa.attention_window(st["qw"], k[None], v[None], 70, sinks=2)
            old = new
        return got + [pages, table, free[:1], count]

    states = [state(64, 700, 2), state(128, 300, 3)]
    for st in states:
        T = st["T"]
        st["lens"] = [i32([T // 3, T // 2]), i32([T // 3 + 1, T // 2 + 1]), i32([T // 3 + 2, 0]), i32([T, 5])]
    want = [loop(st) for st in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(3):
        for i, side in enumerate(streams):
            with torch.cuda.stream(side):
                got[i].append(loop(states[i]))
    torch.cuda.synchronize()
    apa.check_error()
    for i in range(2):
        for run in got[i]:
            assert len(run) == len(want[i]) and all(torch.equal(a, b) for a, b in zip(run, want[i]))


@pytest.mark.parametrize("d,Hq,n,window,sinks,at", [(64, 1, 300, 20, 0, 130), (128, 3, 400, 200, 4, 64), (256, 2, 200, 1, 1, 100)])
@pytest.mark.parametrize("what", [math.nan, math.inf, 3e38])
def test_window_hides_scores_that_are_no_numbers(d, Hq, n, window, sinks, at, what):
    """One key whose products with Q are NaN or overflow: the rows that do not see it are as they would be without it."""
    import torch

    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(n)
    q, k, v = (_torch(rng.standard_normal((1, h, n, d)), torch.bfloat16) for h in (Hq, 1, 1))
    if what == 3e38:
        q[..., 0] = 8
    want, want_lse = apa.attention_window(q, k, v, window, sinks=sinks)
    k[0, 0, at] = what
    out, lse = apa.attention_window(q, k, v, window, sinks=sinks)
    apa.check_error()
    hidden = [p for p in range(n) if p < at or p >= at + window]
    assert torch.equal(out[:, :, hidden], want[:, :, hidden]) and torch.equal(lse[:, :, hidden], want_lse[:, :, hidden])


# ------------------------------------------------------------------ large
@pytest.mark.parametrize("d,Hq,Nq,lens,window,sinks", [
    (128, 8, 150, [400, 90], 0, 0), (64, 6, 333, [333], 50, 70), (256, 4, 100, [1000, 0, 31], 200, 3)])
def test_many_query_rows(d, Hq, Nq, lens, window, sinks):
    """The end of a prompt: hundreds of rows per head, so many row blocks of one item's keys."""
    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(Nq)
    pages, table, ks, vs, kv = _cache(rng, len(lens), 2, d, lens, max(lens) // 64 + 2)
    q = _torch(rng.standard_normal((len(lens), Hq, Nq, d)), _types()["bf16"])
    out, lse = apa.attention_cache(q, pages, table, _torch(np.asarray(lens, np.int32)), _torch(ks), _torch(vs), window=window,
                                   sinks=sinks)
    apa.check_error()
    _near(out, lse, _attend(q.double().cpu().numpy(), kv, lens, window, sinks), "bf16")


def test_a_pool_and_values_past_32_bits():
    """Pages behind the first 4 GB of a pool, and tokens behind the first 4 GB of what is written and read, are what they
    are in a small one."""
    import torch

    import mixed_precision_attention_gb300 as apa
    H, d, n = 8, 256, 1200
    rng = np.random.default_rng(6)
    big = torch.empty(40000, H, 72 * d, dtype=torch.uint8, device="cuda")
    small = apa.cache_pages(20, H, d)
    big[39900:] = 0
    assert big.numel() > 2 ** 32
    T = 1100000  # of which the last n have slots
    k, v = (torch.zeros(T, H, d, dtype=torch.bfloat16, device="cuda").transpose(0, 1) for _ in range(2))
    assert k.numel() * 2 > 2 ** 32
    for x in (k, v):
        x[:, T - n:] = _torch(rng.standard_normal((H, n, d)), torch.bfloat16)
    s = (_torch(np.full(H, 5 / 2688, np.float32)),) * 2
    at = torch.arange(n, dtype=torch.int32, device="cuda")
    slots = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    slots[T - n:] = (39999 - at // 64) * 64 + at % 64
    apa.cache_write(k, v, slots, big, *s)
    apa.cache_write(k[:, T - n:], v[:, T - n:], at, small, *s)
    assert torch.equal(big[39981:].flip(0), small[:19])
    got = apa.cache_read(big, slots, *s)
    want = apa.cache_read(small, at, *s)
    for a, b in zip(got, want):
        assert torch.equal(a[:, T - n:], b) and not a[:, :T - n].any()
    q = _torch(rng.standard_normal((1, 2 * H, 1, d)), torch.bfloat16)
    lens = _torch(np.array([n], np.int32))
    table = torch.arange(20, dtype=torch.int32, device="cuda")[None]
    want = apa.attention_cache(q, small, table, lens, *s)
    got = apa.attention_cache(q, big, 39999 - table, lens, *s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    apa.check_error()


def test_window_over_keys_past_32_bits():
    """The last rows of a context whose keys and values are more than 4 GB each."""
    import torch

    import mixed_precision_attention_gb300 as apa
    g = torch.Generator(device="cuda").manual_seed(3)
    H, d, N, Nq, tail = 8, 128, 2200000, 70, 3000
    k, v = (torch.zeros(1, H, N, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert k.numel() * 2 > 2 ** 32
    for x in (k, v):
        x[:, :, N - tail:] = torch.randn(1, H, tail, d, device="cuda", generator=g).bfloat16()
    q = torch.randn(1, 2 * H, Nq, d, device="cuda", generator=g).bfloat16()
    got = apa.attention_window(q, k, v, 500)
    assert (N - tail - 8) % 64 == 0  # so that the short context has the same tiles
    want = apa.attention_window(q, k[:, :, N - tail - 8:].contiguous(), v[:, :, N - tail - 8:].contiguous(), 500)
    apa.check_error()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
