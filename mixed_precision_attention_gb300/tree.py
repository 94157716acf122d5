"""Checking a tree of drafted tokens over the 4-bit paged K/V cache.

Bindings of ``apa_draft_tree``, ``apa_attention_tree`` and ``apa_cache_accept`` (``include/apa.h``).  A step of a
request with `base` keys in the cache and `nodes` drafted tokens (`lens` = base + nodes), node n at key base + n:

    tree = apa.draft_tree(parents, nodes)                            # once per step; rotary positions: base + depths
    t = apa.cache_tables(base, lens, block_table, free_pages, free_count, max_tokens, free_count_out=free_count)
    apa.cache_write(k, v, t["slots"], pages, k_scale, v_scale)       # every layer, its own pool
    out, lse = apa.attention_tree(q, pages, block_table, lens, nodes, tree["mask"], k_scale, v_scale)
    new_lens = apa.cache_accept(all_pages, block_table, lens, nodes, path, counts)       # once the path is known
    apa.cache_tables(lens, new_lens, block_table, free_pages, free_count, 0, free_count_out=free_count)

Every call only enqueues work on the current stream of its tensors' device, and can be captured into a CUDA graph.
"""
from __future__ import annotations

from . import _lib
from .cache import _DTYPES, _Tensor, _empty, _enqueue, _f32, _i32, _int, _need, _need_pool, _need_rows, _u8

TREE_MAX_NODES = 1024


def draft_tree(parents, nodes=None):
    """Which drafted tokens each one sees, and their depths (apa_draft_tree).

    parents: int32 [B, Nq]; a node's parent is a node before it, or -1: the context.  nodes: int32 [B], the nodes of
    each sequence, or None: Nq.  Returns a dict of int32 CUDA tensors: mask [B, Nq, ceil(Nq / 32)], bit n % 32 of word
    n / 32 of a row for each ancestor n and the node itself, and depths [B, Nq]; both 0 for rows from nodes on."""
    if not isinstance(parents, _Tensor) or not parents.is_cuda:
        raise ValueError("parents must be on a CUDA device")
    index = parents.get_device()
    _need("parents", parents, _i32, 2, index)
    B, Nq = parents.shape
    if nodes is not None:
        _need("nodes", nodes, _i32, 1, index)
        if nodes.shape[0] != B:
            raise ValueError("nodes must be [B]")
    mask = _empty((B, Nq, (Nq + 31) // 32), dtype=_i32, device=parents.device)
    depths = _empty((B, Nq), dtype=_i32, device=parents.device)
    _enqueue(index, "apa_draft_tree", parents.data_ptr(), None if nodes is None else nodes.data_ptr(), _int(B), _int(Nq),
             mask.data_ptr(), depths.data_ptr())
    return {"mask": mask, "depths": depths}


def attention_tree_workspace_bytes(B: int, Hq: int, Hkv: int, Nq: int, d: int) -> int:
    """Bytes of workspace that attention_tree() needs for these sizes; 0 if it does not take them."""
    return _lib.load().apa_attention_tree_workspace_bytes(_int(B), _int(Hq), _int(Hkv), _int(Nq), _int(d))


def _need_tree(name, t, dim, index, B, Nq):
    """t must be an int32 tensor [B or 1, Nq, ...] whose sequences are contiguous; returns their distance (0: one for
    all)."""
    if not isinstance(t, _Tensor) or t.dim() != dim or t.dtype is not _i32:
        raise TypeError(f"{name} must be a {dim}-D tensor of torch.int32")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, not {t.device}")
    if B == 0 or t.shape[0] not in (1, B) or t.shape[1] != Nq or dim == 3 and t.shape[2] != (Nq + 31) // 32:
        raise ValueError(f"{name} must be [B or 1, Nq{', ceil(Nq / 32)' if dim == 3 else ''}]")
    if not t[0].is_contiguous():
        raise ValueError(f"each sequence's {name} must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else 0


def attention_tree(q, pages, block_table, lens, nodes, mask, k_scale, v_scale, depths=None, window: int = 0,
                   sinks: int = 0, return_lse: bool = True, workspace=None):
    """Attention of drafted tokens over the 4-bit cache, each to the context and the nodes of its mask
    (apa_attention_tree).

    q: [B, Hq, Nq, d] bf16 or fp16; channels contiguous, the rest at any stride that is a multiple of 8 elements.
    pages, block_table, k_scale, v_scale: as for attention_cache().  lens: int32 [B], each sequence's keys with its
    nodes' own; nodes: int32 [B], or None: Nq for all.  mask: int32 [B or 1, Nq, ceil(Nq / 32)], depths: int32 [B or 1,
    Nq] (draft_tree(); one sequence's are for all).  With window >= 1 (which needs depths) a row sees, of those keys,
    the ones whose position is above its own - window, or below sinks; a node's position is lens - nodes + depth.
    Returns (out [B, Hq, Nq, d] of q's dtype, contiguous; lse fp32 [B, Hq, Nq] or None); a row that sees no key, and
    those from nodes on, give zeros and -inf; one whose largest score is beyond 2^24 (times log2 e) NaN.
    workspace: optional uint8 CUDA tensor of at least attention_tree_workspace_bytes(...) bytes, 256-byte aligned;
    calls that can overlap on the GPU need one each."""
    index = _need_rows("q", q, 4)
    B, Hq, Nq, d = q.shape
    num_pages, Hkv, dim = _need_pool(pages, k_scale, v_scale, index)
    if (B | Hq | Nq | Hkv | num_pages) >> 31:  # (a C int would lose the upper bits)
        raise ValueError("sizes must be below 2^31")
    if dim != d:
        raise ValueError("pages must be [num_pages, Hkv, 72 * d] with q's d")
    _need("block_table", block_table, _i32, 2, index)
    _need("lens", lens, _i32, 1, index)
    if nodes is not None:
        _need("nodes", nodes, _i32, 1, index)
    if block_table.shape[0] != B or lens.shape[0] != B or nodes is not None and nodes.shape[0] != B:
        raise ValueError("block_table must be [B, max_pages], lens and nodes [B]")
    mask_stride = _need_tree("mask", mask, 3, index, B, Nq)
    depth_stride = 0 if depths is None else _need_tree("depths", depths, 2, index, B, Nq)
    window = _int(window)
    if window and depths is None:
        raise ValueError("a window needs depths")
    dev = q.device
    if workspace is None:
        workspace = _empty(_lib.load().apa_attention_tree_workspace_bytes(B, Hq, Hkv, Nq, d), dtype=_u8, device=dev)
    else:
        _need("workspace", workspace, _u8, 1, index)
    out = _empty((B, Hq, Nq, d), dtype=q.dtype, device=dev)
    lse = _empty((B, Hq, Nq), dtype=_f32, device=dev) if return_lse else None
    qb, qh, qr, _ = q.stride()
    _enqueue(index, "apa_attention_tree", q.data_ptr(), _DTYPES[q.dtype], qb, qh, qr, pages.data_ptr(), num_pages,
             block_table.data_ptr(), _int(block_table.shape[1]), lens.data_ptr(), None if nodes is None else nodes.data_ptr(),
             mask.data_ptr(), mask_stride, None if depths is None else depths.data_ptr(), depth_stride, k_scale.data_ptr(),
             v_scale.data_ptr(), B, Hq, Hkv, Nq, d, window, _int(sinks), out.data_ptr(),
             None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.numel())
    return out, lse


def cache_accept(pages, block_table, lens, nodes, path, counts):
    """Keeps each tree's accepted path: moves its keys behind the context (apa_cache_accept).

    pages: the pool [num_pages, Hkv, 72 * d], or the layers' pools in one tensor [layers, num_pages, Hkv, 72 * d];
    written in place.  lens, nodes: int32 [B], as for attention_tree().  path: int32 [B, path_len], rising node numbers;
    counts: int32 [B], how many of them are accepted.  Returns the new lengths, int32 [B]: lens - nodes + counts."""
    if not isinstance(pages, _Tensor) or not pages.is_cuda:
        raise ValueError("pages must be on a CUDA device")
    index = pages.get_device()
    if pages.dim() == 3:
        pages = pages[None]
    _need("pages", pages, _u8, 4, index)
    layers, num_pages, Hkv, n = pages.shape
    if n % 72:
        raise ValueError("pages must be [num_pages, Hkv, 72 * d] or [layers, num_pages, Hkv, 72 * d]")
    _need("block_table", block_table, _i32, 2, index)
    _need("lens", lens, _i32, 1, index)
    _need("nodes", nodes, _i32, 1, index)
    _need("path", path, _i32, 2, index)
    _need("counts", counts, _i32, 1, index)
    B = lens.shape[0]
    if block_table.shape[0] != B or nodes.shape[0] != B or path.shape[0] != B or counts.shape[0] != B:
        raise ValueError("block_table must be [B, max_pages], path [B, path_len], lens, nodes and counts [B]")
    new_lens = _empty(B, dtype=_i32, device=lens.device)
    _enqueue(index, "apa_cache_accept", pages.data_ptr(), _int(layers), _int(num_pages), _int(Hkv), _int(n // 72),
             block_table.data_ptr(), _int(block_table.shape[1]), lens.data_ptr(), nodes.data_ptr(), path.data_ptr(),
             _int(path.shape[1]), counts.data_ptr(), _int(B), new_lens.data_ptr())
    return new_lens
