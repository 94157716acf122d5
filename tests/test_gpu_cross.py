"""attention_cross against the formula in 64 bits."""
import math

import pytest
import torch

import mixed_precision_attention_gb300 as apa

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def inputs(B, Hq, H, Nq, N, d, dtype, seed=0, spread=1.0):
    """q [B, Hq, Nq, d] and k, v [B, H, N, d] as a projection leaves them (tokens first), so with strides."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    u = torch.randn(H, 1, d, device="cuda", generator=g)
    kv = torch.randn(B, N, 2, H, d, device="cuda", generator=g)
    kv[:, :, 0] = kv[:, :, 0] * 0.5 + u[:, 0]
    kv = kv.to(dtype)
    q = torch.randn(B, Nq, H, Hq // H, d, device="cuda", generator=g) * 0.5 + u
    q = (q * spread).reshape(B, Nq, Hq, d).to(dtype)
    return q.transpose(1, 2), kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)


def formula(q, k, v, lens):
    """(out, lse, sum of w |v|) in 64 bits."""
    B, Hq, Nq, d = q.shape
    out = torch.zeros(B, Hq, Nq, d, dtype=torch.float64, device=q.device)
    size = torch.zeros_like(out)
    lse = torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64, device=q.device)
    G = Hq // k.shape[1]
    for b, n in enumerate(lens):
        if n:
            kk, vv = (x[b, :, :n].double().repeat_interleave(G, 0) for x in (k, v))
            x = q[b].double() @ kk.transpose(1, 2) / math.sqrt(d)
            lse[b] = torch.logsumexp(x, -1)
            w = torch.softmax(x, -1)
            out[b], size[b] = w @ vv, w @ vv.abs()
    return out, lse, size


def check(q, k, v, lens, got):
    """Weights are rounded to the type once (half a step of it, relative), the output once more; FP32 products and sums
    of n terms are off by less than n 2^-24 of the sum of the magnitudes, exponentials by 2^-21 and by the FP32
    rounding of scores up to 2^7 in log2 units (2^-17)."""
    out, lse = got
    ref, ref_lse, size = formula(q, k, v, lens)
    half = torch.finfo(q.dtype).eps / 2
    n = max(max(lens), 1)
    tol = size * (half + 2 ** -16 + n * 2.0 ** -24) + ref.abs() * half + (2.0 ** -25 if q.dtype is F16 else 0)
    err = (out.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol.clamp_min(1e-300)).max())
    seen = torch.isfinite(ref_lse)
    assert torch.equal(torch.isfinite(lse), seen) and bool((lse[~seen] == -math.inf).all())
    assert float((lse.double() - ref_lse)[seen].abs().max() if seen.any() else 0) <= 2 ** -14
    assert bool((out[~seen] == 0).all())


def run(q, k, v, lens, **kw):
    t = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = apa.attention_cross(q, k, v, t, **kw)
    apa.check_error()
    return got


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Nq,lens", [
    (1, [1]), (1, [64, 63, 65]), (1, [500, 0, 128, 129, 1]), (5, [77, 300]), (128, [200]), (129, [1, 127, 513]),
    (300, [1000, 64]), (70, [0, 0, 3])])
def test_lengths_and_rows(dtype, d, Nq, lens):
    q, k, v = inputs(len(lens), 6, 2, Nq, max(max(lens), 1) + 7, d, dtype, seed=Nq + d)
    check(q, k, v, lens, run(q, k, v, lens))


@pytest.mark.parametrize("Hq,H", [(1, 1), (5, 1), (16, 1), (8, 8), (24, 8)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_heads(Hq, H, d):
    q, k, v = inputs(2, Hq, H, 37, 200, d, BF16, seed=Hq)
    check(q, k, v, [200, 90], run(q, k, v, [200, 90]))
    check(q, k, v, [200, 200], run(q, k, v, None))
