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
