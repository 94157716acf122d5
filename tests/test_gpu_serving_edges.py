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
