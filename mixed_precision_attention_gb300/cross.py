"""Attention to an encoder's states: the binding of ``apa_attention_cross`` (``include/apa.h``)."""
from __future__ import annotations

from . import _lib
from .cache import _DTYPES, _empty, _enqueue, _f32, _i32, _int, _need, _need_rows, _u8


def attention_cross_workspace_bytes(B: int, Hq: int, Hkv: int, Nq: int, d: int) -> int:
    """Bytes of workspace that attention_cross() needs for these sizes; 0 if it does not take them."""
    return _lib.load().apa_attention_cross_workspace_bytes(_int(B), _int(Hq), _int(Hkv), _int(Nq), _int(d))


def attention_cross(q, k, v, lens=None, return_lse: bool = True, workspace=None):
    """Attention of every query row to its sequence's encoder states (apa_attention_cross).

    q: [B, Hq, Nq, d], k, v: [B, Hkv, Nkv, d], bf16 or fp16, all alike; channels contiguous, the rest at any
    stride that is a multiple of 8 elements (projections' [B, N, H, d] outputs go in as ``x.transpose(1, 2)``;
    k and v may be expanded over the batch or the heads).  lens: int32 [B], the keys of each sequence, or None:
    all Nkv.  Returns (out [B, Hq, Nq, d] of q's dtype, contiguous; lse fp32 [B, Hq, Nq] or None); rows of a
    sequence without keys give zeros and -inf; those whose largest score is beyond 2^29 in bf16, 2^24 in fp16
    (times log2 e) NaN.
    workspace: optional uint8 CUDA tensor of at least attention_cross_workspace_bytes(...) bytes, 256-byte
    aligned; calls that can overlap on the GPU need one each."""
    index = _need_rows("q", q, 4)
    if _need_rows("k", k, 4) != index or _need_rows("v", v, 4) != index or v.shape != k.shape \
            or k.dtype is not q.dtype or v.dtype is not q.dtype:
        raise ValueError("q, k and v must be of one dtype and on one device, k and v of one shape")
    B, Hq, Nq, d = q.shape
    b, Hkv, Nkv, dk = k.shape
    if b != B or dk != d:
        raise ValueError("k and v must be [B, Hkv, Nkv, d] with q's B and d")
    if (B | Hq | Nq | Hkv | Nkv | d) >> 31:  # (an expanded axis may be as long; a C int would lose its upper bits)
        raise ValueError("sizes must be below 2^31")
    if lens is not None:
        _need("lens", lens, _i32, 1, index)
        if lens.shape[0] != B:
            raise ValueError("lens must be [B]")
    dev = q.device
    if workspace is None:
        workspace = _empty(_lib.load().apa_attention_cross_workspace_bytes(B, Hq, Hkv, Nq, d), dtype=_u8, device=dev)
    else:
        _need("workspace", workspace, _u8, 1, index)
    out = _empty((B, Hq, Nq, d), dtype=q.dtype, device=dev)
    lse = _empty((B, Hq, Nq), dtype=_f32, device=dev) if return_lse else None
    qb, qh, qr, _ = q.stride()
    kb, kh, kt, _ = k.stride()
    vb, vh, vt, _ = v.stride()
    _enqueue(index, "apa_attention_cross", q.data_ptr(), _DTYPES[q.dtype], qb, qh, qr, k.data_ptr(), kb, kh, kt,
             v.data_ptr(), vb, vh, vt, None if lens is None else lens.data_ptr(), B, Hq, Hkv, Nq, Nkv, d, out.data_ptr(),
             None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.numel())
    return out, lse
