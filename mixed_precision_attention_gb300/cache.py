"""The 4-bit paged K/V cache: tables, writing, reading, and attention over it.

Bindings of the ``apa_cache_*`` and ``apa_attention_cache`` entry points of
``include/apa.h`` (page layout and numerics there).  The pool is a uint8 CUDA
tensor ``[num_pages, Hkv, 72 * d]`` (``cache_pages``); a key's slot in it is
``page * 64 + key within the page``.  A serving loop:

    pages = apa.cache_pages(num_pages, Hkv, d, device)
    t = apa.cache_tables(old_lens, new_lens, block_table, free_pages, free_count, max_tokens)
    apa.cache_write(k, v, t["slots"], pages, k_scale, v_scale)       # every layer, its own pool
    out, lse = apa.attention_cache(q, pages, block_table, new_lens, k_scale, v_scale)

Every call only enqueues work on the current stream of its tensors' device, and
can be captured into a CUDA graph.
"""
from __future__ import annotations

import torch

from . import _lib

PAGE = 64  # keys per page
_DTYPES = {torch.bfloat16: 0, torch.float16: 1}  # APA_DTYPE_*
TABLES_STATUS = {0: "ok", 1: "a length is out of range", 2: "more tokens than max_tokens", 3: "too few free pages",
                 4: "the free list's count is out of range, or its capacity too small"}


def _enqueue(dev, name, *args):
    """Calls an entry point with the current stream of `dev`, which is made current for it (the raw stream: a decoding
    step makes several of these calls, and a Stream object costs more than a launch)."""
    fn = getattr(_lib.load(), name)
    index = dev.index
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if st:
        _lib.check(st, name)


def _need(name, t, dtype, dim, dev=None, contiguous=True):
    if not isinstance(t, torch.Tensor) or t.dim() != dim or (t.dtype is not dtype if dtype else t.dtype not in _DTYPES):
        raise TypeError(f"{name} must be a {dim}-D tensor of {dtype or 'torch.bfloat16 or torch.float16'}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} must be on {dev}, not {t.device}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need_rows(name, t, dim, dev=None):
    """16-bit, channels contiguous and 16-byte aligned, the other axes at any stride."""
    _need(name, t, None, dim, dev, contiguous=False)
    if t.stride(-1) != 1 and t.numel():
        raise ValueError(f"{name}'s last dimension must be contiguous")


def _pool(pages, Hkv=None, d=None):
    _need("pages", pages, torch.uint8, 3)
    if pages.shape[2] % 72 or (Hkv is not None and tuple(pages.shape[1:]) != (Hkv, 72 * d)):
        raise ValueError("pages must be [num_pages, Hkv, 72 * d]")
    return pages.device


def _scales(Hkv, dev, k_scale, v_scale):
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        _need(name, t, torch.float32, 1, dev)
        if t.shape[0] != Hkv:
            raise ValueError(f"{name} must be [Hkv]")


def cache_pages(num_pages: int, Hkv: int, d: int, device="cuda"):
    """An empty pool: uint8 zeros [num_pages, Hkv, 72 * d]."""
    if d not in (64, 128, 256):
        raise ValueError("d must be 64, 128 or 256")
    return torch.zeros((num_pages, Hkv, 72 * d), dtype=torch.uint8, device=device)


def cache_tables(old_lens, new_lens, block_table, free_pages, free_count, max_tokens: int, free_count_out=None):
    """Grows, shrinks and places requests and maps their new tokens to slots (apa_cache_tables).

    old_lens, new_lens: int32 [B] key counts before and after; block_table: int32 [B, max_pages] and
    free_pages: int32 [capacity], a stack of free page numbers with free_count (int32 [1]) of them in use,
    both updated in place.  Returns a dict of int32 CUDA tensors: slots and positions [max_tokens] of the new
    tokens, packed by request (slot -1, position 0 behind the last), starts [B + 1], free_count [1] (in
    free_count_out if given, which may be free_count itself), and status [1] (TABLES_STATUS): where it is not
    0 nothing was changed and every slot is -1."""
    _need("old_lens", old_lens, torch.int32, 1)
    dev = old_lens.device
    _need("new_lens", new_lens, torch.int32, 1, dev)
    _need("block_table", block_table, torch.int32, 2, dev)
    _need("free_pages", free_pages, torch.int32, 1, dev)
    _need("free_count", free_count, torch.int32, 1, dev)
    B = old_lens.shape[0]
    if new_lens.shape[0] != B or block_table.shape[0] != B or free_count.shape[0] != 1:
        raise ValueError("old_lens and new_lens must be [B], block_table [B, max_pages], free_count [1]")
    max_tokens = int(max_tokens)
    if max_tokens < 0:
        raise ValueError("max_tokens must not be negative")
    if free_count_out is not None:
        _need("free_count_out", free_count_out, torch.int32, 1, dev)
        if free_count_out.shape[0] != 1:
            raise ValueError("free_count_out must be [1]")
    slots = torch.empty(max_tokens, dtype=torch.int32, device=dev)
    positions = torch.empty(max_tokens, dtype=torch.int32, device=dev)
    starts = torch.empty(B + 1, dtype=torch.int32, device=dev)
    status = torch.empty(1, dtype=torch.int32, device=dev)
    count = torch.empty(1, dtype=torch.int32, device=dev) if free_count_out is None else free_count_out
    _enqueue(dev, "apa_cache_tables", old_lens.data_ptr(), new_lens.data_ptr(), B, block_table.data_ptr(),
             block_table.shape[1], free_pages.data_ptr(), free_pages.shape[0], free_count.data_ptr(), max_tokens,
             slots.data_ptr(), positions.data_ptr(), starts.data_ptr(), count.data_ptr(), status.data_ptr())
    return {"slots": slots, "positions": positions, "starts": starts, "free_count": count, "status": status}


def cache_write(k, v, slots, pages, k_scale, v_scale):
    """Quantizes tokens into the cache (apa_cache_write).

    k, v: [Hkv, T, d] bf16 or fp16; channels contiguous, heads and tokens at any stride that is a multiple of
    8 elements (a projection's [T, Hkv, d] output goes in as ``k.transpose(0, 1)``).  slots: int32 [T], one
    for each token, no two alike; a token of a negative slot is skipped.  pages: the pool, written in place.
    k_scale, v_scale: fp32 [Hkv], positive (largest magnitude expected / 2688; larger values saturate)."""
    _need_rows("k", k, 3)
    dev = k.device
    _need_rows("v", v, 3, dev)
    Hkv, T, d = k.shape
    if v.shape != k.shape or v.dtype is not k.dtype:
        raise ValueError("k and v must be alike")
    _need("slots", slots, torch.int32, 1, dev)
    if slots.shape[0] != T:
        raise ValueError("slots must be [T]")
    if _pool(pages, Hkv, d) != dev:
        raise ValueError("pages must be on k's device")
    _scales(Hkv, dev, k_scale, v_scale)
    kh, kt, _ = k.stride()
    vh, vt, _ = v.stride()
    _enqueue(dev, "apa_cache_write", k.data_ptr(), v.data_ptr(), _DTYPES[k.dtype], Hkv, T, d, kh, kt, vh, vt,
             slots.data_ptr(), pages.data_ptr(), pages.shape[0], k_scale.data_ptr(), v_scale.data_ptr())


def cache_read(pages, slots, k_scale, v_scale, dtype=torch.bfloat16):
    """The values that cached tokens stand for (apa_cache_read): k, v [Hkv, T, d] of `dtype` (bf16 or fp16),
    contiguous, so that ``k[None]`` is what attention() takes.  Tokens of negative slots are zero."""
    dev = _pool(pages)
    _need("slots", slots, torch.int32, 1, dev)
    num_pages, Hkv, n = pages.shape
    _scales(Hkv, dev, k_scale, v_scale)
    if dtype not in _DTYPES:
        raise TypeError("dtype must be torch.bfloat16 or torch.float16")
    T, d = slots.shape[0], n // 72
    k = torch.empty((Hkv, T, d), dtype=dtype, device=dev)
    v = torch.empty((Hkv, T, d), dtype=dtype, device=dev)
    _enqueue(dev, "apa_cache_read", pages.data_ptr(), num_pages, _DTYPES[dtype], Hkv, T, d, slots.data_ptr(),
             k_scale.data_ptr(), v_scale.data_ptr(), k.data_ptr(), v.data_ptr())
    return k, v


def attention_cache_workspace_bytes(B: int, Hq: int, Hkv: int, Nq: int, d: int) -> int:
    """Bytes of workspace that attention_cache() needs for these sizes."""
    return int(_lib.load().apa_attention_cache_workspace_bytes(B, Hq, Hkv, Nq, d))


def attention_cache(q, pages, block_table, lens, k_scale, v_scale, window: int = 0, sinks: int = 0,
                    return_lse: bool = True, workspace=None):
    """Attention of the last Nq query rows of each sequence over the 4-bit cache (apa_attention_cache).

    q: [B, Hq, Nq, d] bf16 or fp16; channels contiguous, the rest at any stride that is a multiple of 8
    elements.  pages: the pool [num_pages, Hkv, 72 * d]; block_table: int32 [B, max_pages]; lens: int32 [B],
    each sequence's keys with the rows' own.  Row i, at position p = lens - Nq + i, sees the keys j <= p, with
    window >= 1 only those with j > p - window or j < sinks.  Returns (out [B, Hq, Nq, d] of q's dtype,
    contiguous; lse fp32 [B, Hq, Nq] or None); a row that sees no key gives zeros and -inf.
    workspace: optional uint8 CUDA tensor of at least attention_cache_workspace_bytes(...) bytes; calls that
    can overlap on the GPU need one each."""
    _need_rows("q", q, 4)
    dev = q.device
    B, Hq, Nq, d = q.shape
    if _pool(pages) != dev or pages.shape[2] != 72 * d:
        raise ValueError("pages must be [num_pages, Hkv, 72 * d] with q's d, on q's device")
    num_pages, Hkv, _ = pages.shape
    _need("block_table", block_table, torch.int32, 2, dev)
    _need("lens", lens, torch.int32, 1, dev)
    if block_table.shape[0] != B or lens.shape[0] != B:
        raise ValueError("block_table must be [B, max_pages] and lens [B]")
    _scales(Hkv, dev, k_scale, v_scale)
    if workspace is None:
        workspace = torch.empty(attention_cache_workspace_bytes(B, Hq, Hkv, Nq, d), dtype=torch.uint8, device=dev)
    else:
        _need("workspace", workspace, torch.uint8, 1, dev)
    out = torch.empty((B, Hq, Nq, d), dtype=q.dtype, device=dev)
    lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=dev) if return_lse else None
    qb, qh, qr, _ = q.stride()
    _enqueue(dev, "apa_attention_cache", q.data_ptr(), _DTYPES[q.dtype], qb, qh, qr, pages.data_ptr(), num_pages,
             block_table.data_ptr(), block_table.shape[1], lens.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), B, Hq,
             Hkv, Nq, d, int(window), int(sinks), out.data_ptr(), None if lse is None else lse.data_ptr(),
             workspace.data_ptr(), workspace.numel())
    return out, lse
