"""Exact causal prefill attention with a sliding window and sinks: the binding of
``apa_attention_window`` (``include/apa.h``)."""
from __future__ import annotations

from .cache import _Tensor, _empty, _enqueue, _f32, _int, _need, torch

_bf16 = torch.bfloat16


def attention_window(q, k, v, window: int, sinks: int = 0, return_lse: bool = True):
    """Exact causal attention with a sliding window and sinks (apa_attention_window).

    q: [B, Hq, Nq, d] bf16; k, v: [B, Hkv, Nkv, d] bf16 (CUDA, contiguous, Nkv >= Nq).  Query row i, at
    position p = i + Nkv - Nq, sees the keys j <= p with j > p - window (window >= 1 keys, its own among
    them) or j < sinks.  Returns (out bf16 [B, Hq, Nq, d], lse fp32 [B, Hq, Nq] or None).  Scores, softmax
    and sums are FP32; the weights are rounded to bf16 (2^-8 relative) for the product with V, which must be
    finite."""
    if not isinstance(q, _Tensor) or not q.is_cuda:
        raise ValueError("q must be on a CUDA device")
    index = q.get_device()
    _need("q", q, _bf16, 4, index)
    _need("k", k, _bf16, 4, index)
    _need("v", v, _bf16, 4, index)
    B, Hq, Nq, d = q.shape
    b, Hkv, Nkv, dk = k.shape
    if v.shape != k.shape or b != B or dk != d:
        raise ValueError("k and v must be [B, Hkv, Nkv, d] with q's B and d")
    dev = q.device
    out = _empty((B, Hq, Nq, d), dtype=_bf16, device=dev)
    lse = _empty((B, Hq, Nq), dtype=_f32, device=dev) if return_lse else None
    _enqueue(index, "apa_attention_window", q.data_ptr(), k.data_ptr(), v.data_ptr(), B, Hq, Hkv, Nq, Nkv, d, _int(window),
             _int(sinks), out.data_ptr(), None if lse is None else lse.data_ptr())
    return out, lse
