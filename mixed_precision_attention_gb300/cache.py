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


_Tensor = torch.Tensor
_empty = torch.empty
_i32, _f32, _u8 = torch.int32, torch.float32, torch.uint8
_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _int(x):
    """x as a C int that the entry points read as it is meant: ctypes would drop the upper bits of a larger one.  Window
    and sinks beyond every position mean any such number; negative ones, and counts past 2^31, are refused there."""
    x = int(x)
    return x if -1 <= x <= 0x7FFFFFFF else 0x7FFFFFFF if x > 0 else -1


def _enqueue(index, name, *args):
    """Calls an entry point with the current stream of device `index`, which is made current for it (the raw stream: a
    decoding step makes several of these calls, and a Stream object costs more than a launch)."""
    fn = getattr(_lib.load(), name)
    if _device() == index:
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _raw_stream(index))
    if st:
        _lib.check(st, name)


def _need(name, t, dtype, dim, index):
    """t must be a contiguous `dim`-D tensor of `dtype` on CUDA device `index`."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.dim() == dim and t.get_device() == index and t.is_contiguous():
        return
    if not isinstance(t, _Tensor) or t.dim() != dim or t.dtype is not dtype:
        raise TypeError(f"{name} must be a {dim}-D tensor of {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must be on cuda:{index}, not {t.device}")


def _need_rows(name, t, dim):
    """t must be a `dim`-D bf16 or fp16 CUDA tensor with contiguous channels, the other axes at any stride.  Returns
    its device's index."""
    if not isinstance(t, _Tensor) or t.dim() != dim or t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be a {dim}-D tensor of torch.bfloat16 or torch.float16")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.stride(-1) != 1 and t.numel():
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return t.get_device()


def _need_pool(pages, k_scale, v_scale, index):
    """Checks a pool and its scales; returns (num_pages, Hkv, d)."""
    _need("pages", pages, _u8, 3, index)
    num_pages, Hkv, n = pages.shape
    if n % 72:
        raise ValueError("pages must be [num_pages, Hkv, 72 * d]")
    _need("k_scale", k_scale, _f32, 1, index)
    _need("v_scale", v_scale, _f32, 1, index)
    if k_scale.shape[0] != Hkv or v_scale.shape[0] != Hkv:
        raise ValueError("k_scale and v_scale must be [Hkv]")
    return num_pages, Hkv, n // 72


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
    if not isinstance(old_lens, _Tensor) or not old_lens.is_cuda:
        raise ValueError("old_lens must be on a CUDA device")
    index = old_lens.get_device()
    _need("old_lens", old_lens, _i32, 1, index)
    _need("new_lens", new_lens, _i32, 1, index)
    _need("block_table", block_table, _i32, 2, index)
    _need("free_pages", free_pages, _i32, 1, index)
    _need("free_count", free_count, _i32, 1, index)
    B = old_lens.shape[0]
    if new_lens.shape[0] != B or block_table.shape[0] != B or free_count.shape[0] != 1:
        raise ValueError("old_lens and new_lens must be [B], block_table [B, max_pages], free_count [1]")
    max_tokens = int(max_tokens)
    if not 0 <= max_tokens <= 1 << 30:
        raise ValueError("max_tokens must be in [0, 2^30]")
    if free_count_out is not None:
        _need("free_count_out", free_count_out, _i32, 1, index)
        if free_count_out.shape[0] != 1:
            raise ValueError("free_count_out must be [1]")
    dev = old_lens.device
    slots = _empty(max_tokens, dtype=_i32, device=dev)
    positions = _empty(max_tokens, dtype=_i32, device=dev)
    starts = _empty(B + 1, dtype=_i32, device=dev)
    status = _empty(1, dtype=_i32, device=dev)
    count = _empty(1, dtype=_i32, device=dev) if free_count_out is None else free_count_out
    _enqueue(index, "apa_cache_tables", old_lens.data_ptr(), new_lens.data_ptr(), B, block_table.data_ptr(),
             _int(block_table.shape[1]), free_pages.data_ptr(), _int(free_pages.shape[0]), free_count.data_ptr(), max_tokens,
             slots.data_ptr(), positions.data_ptr(), starts.data_ptr(), count.data_ptr(), status.data_ptr())
    return {"slots": slots, "positions": positions, "starts": starts, "free_count": count, "status": status}


def cache_write(k, v, slots, pages, k_scale, v_scale):
    """Quantizes tokens into the cache (apa_cache_write).

    k, v: [Hkv, T, d] bf16 or fp16; channels contiguous, heads and tokens at any stride that is a multiple of
    8 elements (a projection's [T, Hkv, d] output goes in as ``k.transpose(0, 1)``).  slots: int32 [T], one
    for each token, no two alike; a token of a negative slot is skipped.  pages: the pool, written in place.
    k_scale, v_scale: fp32 [Hkv], 2^-100 .. 2^100 (largest magnitude expected / 2688; larger values, and
    infinities, saturate).  A NaN makes its group of 16 channels NaN."""
    index = _need_rows("k", k, 3)
    Hkv, T, d = k.shape
    if _need_rows("v", v, 3) != index or v.shape != k.shape or v.dtype is not k.dtype:
        raise ValueError("k and v must be alike")
    _need("slots", slots, _i32, 1, index)
    if slots.shape[0] != T or T > 0x7FFFFFFF:
        raise ValueError("slots must be [T], T < 2^31")
    num_pages, heads, dim = _need_pool(pages, k_scale, v_scale, index)
    if heads != Hkv or dim != d:
        raise ValueError("pages must be [num_pages, Hkv, 72 * d] with k's Hkv and d")
    kh, kt, _ = k.stride()
    vh, vt, _ = v.stride()
    _enqueue(index, "apa_cache_write", k.data_ptr(), v.data_ptr(), _DTYPES[k.dtype], Hkv, T, d, kh, kt, vh, vt,
             slots.data_ptr(), pages.data_ptr(), num_pages, k_scale.data_ptr(), v_scale.data_ptr())


def cache_read(pages, slots, k_scale, v_scale, dtype=torch.bfloat16):
    """The values that cached tokens stand for (apa_cache_read): k, v [Hkv, T, d] of `dtype` (bf16 or fp16),
    contiguous, so that ``k[None]`` is what attention() takes.  Tokens of negative slots are zero."""
    if not isinstance(pages, _Tensor) or not pages.is_cuda:
        raise ValueError("pages must be on a CUDA device")
    index = pages.get_device()
    num_pages, Hkv, d = _need_pool(pages, k_scale, v_scale, index)
    _need("slots", slots, _i32, 1, index)
    if dtype not in _DTYPES:
        raise TypeError("dtype must be torch.bfloat16 or torch.float16")
    T, dev = slots.shape[0], pages.device
    if T > 0x7FFFFFFF:
        raise ValueError("slots must be [T], T < 2^31")
    k = _empty((Hkv, T, d), dtype=dtype, device=dev)
    v = _empty((Hkv, T, d), dtype=dtype, device=dev)
    _enqueue(index, "apa_cache_read", pages.data_ptr(), num_pages, _DTYPES[dtype], Hkv, T, d, slots.data_ptr(),
             k_scale.data_ptr(), v_scale.data_ptr(), k.data_ptr(), v.data_ptr())
    return k, v


def attention_cache_workspace_bytes(B: int, Hq: int, Hkv: int, Nq: int, d: int) -> int:
    """Bytes of workspace that attention_cache() needs for these sizes; 0 if it does not take them."""
    return _lib.load().apa_attention_cache_workspace_bytes(_int(B), _int(Hq), _int(Hkv), _int(Nq), _int(d))


def attention_cache(q, pages, block_table, lens, k_scale, v_scale, window: int = 0, sinks: int = 0,
                    return_lse: bool = True, workspace=None):
    """Attention of the last Nq query rows of each sequence over the 4-bit cache (apa_attention_cache).

    q: [B, Hq, Nq, d] bf16 or fp16; channels contiguous, the rest at any stride that is a multiple of 8
    elements.  pages: the pool [num_pages, Hkv, 72 * d]; block_table: int32 [B, max_pages]; lens: int32 [B],
    each sequence's keys with the rows' own.  Row i, at position p = lens - Nq + i, sees the keys j <= p, with
    window >= 1 only those with j > p - window or j < sinks.  Returns (out [B, Hq, Nq, d] of q's dtype,
    contiguous; lse fp32 [B, Hq, Nq] or None); a row that sees no key gives zeros and -inf.
    workspace: optional uint8 CUDA tensor of at least attention_cache_workspace_bytes(...) bytes, 256-byte
    aligned; calls that can overlap on the GPU need one each."""
    index = _need_rows("q", q, 4)
    B, Hq, Nq, d = q.shape
    num_pages, Hkv, dim = _need_pool(pages, k_scale, v_scale, index)
    if dim != d:
        raise ValueError("pages must be [num_pages, Hkv, 72 * d] with q's d")
    _need("block_table", block_table, _i32, 2, index)
    _need("lens", lens, _i32, 1, index)
    if block_table.shape[0] != B or lens.shape[0] != B:
        raise ValueError("block_table must be [B, max_pages] and lens [B]")
    dev = q.device
    if workspace is None:
        workspace = _empty(_lib.load().apa_attention_cache_workspace_bytes(B, Hq, Hkv, Nq, d), dtype=_u8, device=dev)
    else:
        _need("workspace", workspace, _u8, 1, index)
    out = _empty((B, Hq, Nq, d), dtype=q.dtype, device=dev)
    lse = _empty((B, Hq, Nq), dtype=_f32, device=dev) if return_lse else None
    qb, qh, qr, _ = q.stride()
    _enqueue(index, "apa_attention_cache", q.data_ptr(), _DTYPES[q.dtype], qb, qh, qr, pages.data_ptr(), num_pages,
             block_table.data_ptr(), _int(block_table.shape[1]), lens.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), B, Hq,
             Hkv, Nq, d, _int(window), _int(sinks), out.data_ptr(), None if lse is None else lse.data_ptr(),
             workspace.data_ptr(), workspace.numel())
    return out, lse
