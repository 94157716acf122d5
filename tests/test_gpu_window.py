"""attention_window: causal attention with a sliding window and sinks, against a plain
64-bit implementation.

Tolerance: the output is one rounding to bf16 (half a step, eps / 2 = 2^-8: bf16 has 8
significant bits) of a sum whose softmax weights were rounded to bf16 (2^-8 each), so
|out - ref| <= 2^-8 |ref| + 2^-8 * sum_j w_j |v_j|, with 2^-14 of that sum more for the
FP32 scores and sums; |lse - ref| <= 1e-5 * max(1, |ref|).
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _ref(q, k, v, window, sinks):
    B, Hq, Nq, d = q.shape
    G, N = Hq // k.shape[1], k.shape[2]
    p = (N - Nq + np.arange(Nq))[:, None]
    j = np.arange(N)[None]
    see = (j <= p) & ((j > p - window) | (j < sinks))
    out, lse, mag = np.zeros(q.shape), np.zeros(q.shape[:3]), np.zeros(q.shape)
    for b in range(B):
        for h in range(Hq):
            s = np.where(see, q[b, h] @ k[b, h // G].T / math.sqrt(d), -np.inf)
            m = s.max(1, keepdims=True)
            w = np.exp(s - m)
            lse[b, h] = m[:, 0] + np.log(w.sum(1))
            w /= w.sum(1, keepdims=True)
            out[b, h], mag[b, h] = w @ v[b, h // G], w @ np.abs(v[b, h // G])
    return out, lse, mag


SHAPES = [  # B, Hq, Hkv, Nq, Nkv, d, window, sinks
    (1, 1, 1, 1, 1, 64, 1, 0),
    (1, 2, 1, 1, 300, 128, 100, 4),
    (2, 4, 2, 130, 130, 64, 1, 0),
    (1, 4, 2, 130, 130, 64, 1, 1),
    (1, 6, 2, 333, 333, 128, 64, 0),
    (1, 3, 1, 200, 1000, 128, 65, 4),
    (1, 5, 1, 77, 900, 64, 300, 64),
    (1, 5, 1, 77, 900, 64, 300, 65),
    (2, 8, 2, 100, 1100, 256, 127, 3),
    (1, 2, 2, 700, 700, 256, 200, 100),
    (1, 4, 1, 500, 500, 128, 500, 0),
    (1, 4, 1, 500, 640, 128, 2 ** 31 - 1, 2 ** 31 - 1),
    (1, 2, 1, 64, 2000, 128, 10, 1990),     # the sinks reach into the window
    (1, 24, 8, 129, 257, 64, 33, 17),
    (1, 1, 1, 1000, 1003, 64, 3, 200),
]


@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_window(case):
    import torch

    import mixed_precision_attention_gb300 as apa
    B, Hq, H, Nq, N, d, window, sinks = SHAPES[case]
    rng = np.random.default_rng(case)
    x = [rng.standard_normal((B, Hq, Nq, d)) * 2, rng.standard_normal((B, H, N, d)) + rng.standard_normal((B, H, 1, d)),
         rng.standard_normal((B, H, N, d))]
    q, k, v = (torch.from_numpy(a).cuda().to(torch.bfloat16) for a in x)
    out, lse = apa.attention_window(q, k, v, window, sinks=sinks)
    apa.check_error()
    ro, rl, mag = _ref(*(a.double().cpu().numpy() for a in (q, k, v)), window, sinks)
    assert out.dtype is torch.bfloat16
    err = np.abs(out.double().cpu().numpy() - ro)
    assert np.all(err <= 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2.0 ** -14) * mag), err.max()
    assert np.all(np.abs(lse.double().cpu().numpy() - rl) <= 1e-5 * np.maximum(1, np.abs(rl)))
    again, none = apa.attention_window(q, k, v, window, sinks=sinks, return_lse=False)
    assert none is None and torch.equal(again, out)


def test_a_window_of_everything_is_attention():
    import torch

    import mixed_precision_attention_gb300 as apa
    torch.manual_seed(0)
    q = torch.randn(1, 6, 200, 128, device="cuda").bfloat16()
    k, v = (torch.randn(1, 2, 1000, 128, device="cuda").bfloat16() for _ in range(2))
    exact, exact_lse, _ = apa.attention(q, k, v, eps=0.0)
    out, lse = apa.attention_window(q, k, v, 1000)
    # both bounds of this file and attention()'s 4e-3 at eps = 0, on values below 4
    assert (out.float() - exact).abs().max() <= 4e-3 + 2 * 4 * 2.0 ** -8
    assert (lse - exact_lse).abs().max() <= 2e-4


def test_window_on_a_stream_and_in_a_graph():
    import torch

    import mixed_precision_attention_gb300 as apa
    torch.manual_seed(1)
    q = torch.randn(1, 4, 300, 64, device="cuda").bfloat16()
    k, v = (torch.randn(1, 2, 300, 64, device="cuda").bfloat16() for _ in range(2))
    want, _ = apa.attention_window(q, k, v, 50, sinks=2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        out, _ = apa.attention_window(q, k, v, 50, sinks=2)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("d,B,Hq,H,Nq,N,window,sinks", [
    (64, 1, 24, 8, 5001, 5001, 70, 3), (128, 2, 24, 8, 2500, 6000, 333, 130), (256, 1, 16, 4, 3333, 3333, 64, 0),
    (128, 1, 8, 8, 40000, 40000, 1, 1)])
def test_more_row_blocks_than_ctas(d, B, Hq, H, Nq, N, window, sinks):
    # each CTA takes several row blocks in turn; against 64-bit attention over each row's own keys
    import torch

    import mixed_precision_attention_gb300 as apa
    g = torch.Generator(device="cuda").manual_seed(d + Nq)
    q = (2 * torch.randn(B, Hq, Nq, d, device="cuda", generator=g)).bfloat16()
    k, v = (torch.randn(B, H, N, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    out, lse = apa.attention_window(q, k, v, window, sinks=sinks)
    apa.check_error()
    at = torch.arange(N - Nq, N, device="cuda")
    for b in range(B):
        for h in range(0, Hq, 5):
            for r in range(0, Nq, 2048):
                p = at[r:r + 2048, None]
                j = torch.cat([torch.arange(sinks, device="cuda").expand(len(p), -1),
                               p - window + 1 + torch.arange(window, device="cuda")], 1)
                see = torch.cat([j[:, :sinks] <= p - window, j[:, sinks:] >= 0], 1)
                j = j.clamp(0, N - 1)
                kj, vj = k[b, h * H // Hq].double()[j], v[b, h * H // Hq].double()[j]
                s = torch.einsum("rd,rjd->rj", q[b, h, r:r + 2048].double(), kj) / math.sqrt(d)
                s = s.masked_fill(~see, -math.inf)
                w = torch.softmax(s, 1)
                ref, mag = torch.einsum("rj,rjd->rd", w, vj), torch.einsum("rj,rjd->rd", w, vj.abs())
                err = (out[b, h, r:r + 2048].double() - ref).abs()
                assert (err <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -14) * mag).all()
                rl = torch.logsumexp(s, 1)
                assert ((lse[b, h, r:r + 2048].double() - rl).abs() <= 1e-5 * rl.abs().clamp_min(1)).all()
