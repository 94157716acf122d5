"""The entry points of drafted trees and of cross attention refuse bad arguments on the host, before anything is enqueued
(CPU only: the fake pointers below are never dereferenced)."""
import ctypes

import pytest

from mixed_precision_attention_gb300 import _lib, build

P = ctypes.c_void_p
A = [P(0x10000 * (i + 1)) for i in range(16)]  # aligned fake pointers


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def _draft(lib, parents=A[0], nodes=None, B=2, Nq=5, mask=A[1], depths=A[2]):
    return lib.apa_draft_tree(parents, nodes, B, Nq, mask, depths, None)


@pytest.mark.parametrize("kw,status", [
    (dict(parents=None), -1), (dict(mask=None), -1), (dict(depths=None), -1), (dict(B=0), -2), (dict(Nq=0), -2),
    (dict(Nq=1025), -2), (dict(mask=P(0x10004)), -8),
])
def test_draft_refusals(lib, kw, status):
    assert _draft(lib, **kw) == status


def _tree(lib, q=A[0], dtype=0, sb=512, sh=64, sr=256, pages=A[1], num_pages=5, table=A[2], max_pages=4, lens=A[3], nodes=A[4],
          mask=A[5], ms=2, depths=A[6], ds=2, sk=A[7], sv=A[8], B=2, Hq=4, Hkv=2, Nq=2, d=64, window=0, sinks=0, out=A[9],
          ws=A[10], nbytes=1 << 40):
    return lib.apa_attention_tree(q, dtype, sb, sh, sr, pages, num_pages, table, max_pages, lens, nodes, mask, ms, depths, ds, sk,
                                  sv, B, Hq, Hkv, Nq, d, window, sinks, out, None, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), -1), (dict(pages=None), -1), (dict(table=None), -1), (dict(lens=None), -1), (dict(mask=None), -1),
    (dict(sk=None), -1), (dict(sv=None), -1), (dict(out=None), -1), (dict(window=3, depths=None), -1), (dict(B=0), -2),
    (dict(B=8193), -2), (dict(Hq=3), -2), (dict(Nq=0), -2), (dict(Nq=1025), -2), (dict(num_pages=0), -2),
    (dict(num_pages=1 << 25), -2), (dict(max_pages=0), -2), (dict(max_pages=1 << 28), -2), (dict(ms=-1), -2), (dict(ds=-2), -2),
    (dict(d=80), -4), (dict(dtype=3), -11), (dict(window=-1), -12), (dict(sinks=-1), -12), (dict(q=P(0x10002)), -8),
    (dict(pages=P(0x10008)), -8), (dict(out=P(0x10008)), -8), (dict(sr=12), -8), (dict(sh=4), -8), (dict(nbytes=16), -6),
    (dict(ws=P(0x10010)), -6),
])
def test_tree_refusals(lib, kw, status):
    assert _tree(lib, **kw) == status


def _accept(lib, pages=A[0], layers=2, num_pages=5, Hkv=2, d=64, table=A[1], max_pages=4, lens=A[2], nodes=A[3], path=A[4],
            most=3, counts=A[5], B=2, new=A[6]):
    return lib.apa_cache_accept(pages, layers, num_pages, Hkv, d, table, max_pages, lens, nodes, path, most, counts, B, new, None)


@pytest.mark.parametrize("kw,status", [
    (dict(pages=None), -1), (dict(table=None), -1), (dict(lens=None), -1), (dict(nodes=None), -1), (dict(path=None), -1),
    (dict(counts=None), -1), (dict(new=None), -1), (dict(layers=0), -2), (dict(layers=65536), -2), (dict(num_pages=0), -2),
    (dict(num_pages=1 << 25), -2), (dict(Hkv=0), -2), (dict(max_pages=0), -2), (dict(most=0), -2), (dict(most=1025), -2),
    (dict(B=0), -2), (dict(new=A[2]), -2), (dict(d=96), -4), (dict(pages=P(0x10008)), -8),
])
def test_accept_refusals(lib, kw, status):
    assert _accept(lib, **kw) == status


def _cross(lib, q=A[0], dtype=0, qs=(512, 64, 256), k=A[1], ks=(2560, 64, 128), v=A[2], vs=(2560, 64, 128), lens=A[3], B=2,
           Hq=4, Hkv=2, Nq=2, Nkv=20, d=64, out=A[4], ws=A[5], nbytes=1 << 40):
    return lib.apa_attention_cross(q, dtype, *qs, k, *ks, v, *vs, lens, B, Hq, Hkv, Nq, Nkv, d, out, None, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(out=None), -1), (dict(B=0), -2), (dict(B=8193), -2),
    (dict(Hq=3), -2), (dict(Nq=0), -2), (dict(Nkv=0), -2), (dict(Nkv=(1 << 30) + 1), -2), (dict(Nq=1 << 20), -2), (dict(d=80), -4),
    (dict(dtype=2), -11), (dict(q=P(0x10008)), -8), (dict(k=P(0x10008)), -8), (dict(v=P(0x10002)), -8), (dict(out=P(0x10004)), -8),
    (dict(qs=(512, 64, 12)), -8), (dict(ks=(2560, 64, 100)), -8), (dict(vs=(2564, 64, 128)), -8), (dict(ks=(2560, -64, 128)), -8),
    (dict(ks=(2560, 64, 0)), -8), (dict(vs=(2560, 64, 0)), -8), (dict(ks=(1 << 39, 64, 128)), -8), (dict(nbytes=16), -6),
    (dict(ws=P(0x10010)), -6),
])
def test_cross_refusals(lib, kw, status):
    assert _cross(lib, **kw) == status


def test_sizes(lib):
    for size in (lib.apa_attention_tree_workspace_bytes, lib.apa_attention_cross_workspace_bytes):
        one = size(1, 24, 8, 32, 128)
        assert one > 0 and one == size(8192, 24, 8, 32, 128)  # it does not grow with the sequences
        assert size(1, 24, 8, 100, 128) > 0 and size(1, 24, 8, 1, 64) < size(1, 24, 8, 1, 256)
        assert size(1, 5, 2, 1, 128) == size(1, 24, 8, 1, 96) == size(0, 24, 8, 1, 128) == size(1, 24, 8, 0, 128) == 0
    assert lib.apa_attention_tree_workspace_bytes(1, 8, 8, 1025, 64) == 0
    assert lib.apa_attention_cross_workspace_bytes(1, 8, 8, 1025, 64) > 0


def test_bindings_refuse_host_tensors_and_other_types():
    import torch

    import mixed_precision_attention_gb300 as apa
    i32, f32 = torch.zeros(2, dtype=torch.int32), torch.ones(2)
    q = torch.zeros(2, 4, 3, 64, dtype=torch.bfloat16)
    pages = torch.zeros(3, 2, 72 * 64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        apa.draft_tree(i32[None])
    with pytest.raises(ValueError):
        apa.attention_tree(q, pages, i32[None], i32, i32, i32[None, None], f32, f32)
    with pytest.raises(ValueError):
        apa.cache_accept(pages, i32[None], i32, i32, i32[None], i32)
    with pytest.raises(ValueError):
        apa.attention_cross(q, q, q)
    for bad in (q.float(), q[0], None):
        with pytest.raises(TypeError):
            apa.attention_cross(bad, q, q)
        with pytest.raises(TypeError):
            apa.attention_tree(bad, pages, i32[None], i32, i32, i32[None, None], f32, f32)
    assert apa.TREE_MAX_NODES == 1024
