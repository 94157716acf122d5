"""The cache and window entry points refuse bad arguments on the host, before anything is
enqueued (CPU only: the fake pointers below are never dereferenced)."""
import ctypes

import pytest

from mixed_precision_attention_gb300 import _lib, build

P = ctypes.c_void_p
A = [P(0x10000 * (i + 1)) for i in range(16)]  # aligned fake pointers


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def _window(lib, q=A[0], k=A[1], v=A[2], B=1, Hq=4, Hkv=2, Nq=64, Nkv=128, d=64, window=16, sinks=0, out=A[3]):
    return lib.apa_attention_window(q, k, v, B, Hq, Hkv, Nq, Nkv, d, window, sinks, out, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(out=None), -1), (dict(B=0), -2),
    (dict(Hq=3), -2), (dict(Nq=129), -2), (dict(Nkv=0), -2), (dict(Nkv=64 * 65536), -2), (dict(d=96), -4),
    (dict(window=0), -12), (dict(window=-1), -12), (dict(sinks=-1), -12), (dict(q=P(0x10008)), -8),
    (dict(out=P(0x10008)), -8),
])
def test_window_refusals(lib, kw, status):
    assert _window(lib, **kw) == status


def _tables(lib, old=A[0], new=A[1], B=4, table=A[2], max_pages=8, free=A[3], cap=10, count=A[4], most=16, slots=A[5],
            pos=A[6], starts=A[7], out=A[8], status=A[9]):
    return lib.apa_cache_tables(old, new, B, table, max_pages, free, cap, count, most, slots, pos, starts, out, status, None)


@pytest.mark.parametrize("kw,status", [
    (dict(old=None), -1), (dict(new=None), -1), (dict(table=None), -1), (dict(free=None), -1), (dict(count=None), -1),
    (dict(slots=None), -1), (dict(pos=None), -1), (dict(starts=None), -1), (dict(out=None), -1), (dict(status=None), -1),
    (dict(B=0), -2), (dict(B=8193), -2), (dict(max_pages=0), -2), (dict(max_pages=1 << 25), -2), (dict(cap=0), -2),
    (dict(most=-1), -2), (dict(most=(1 << 30) + 1), -2),
])
def test_tables_refusals(lib, kw, status):
    assert _tables(lib, **kw) == status


def _write(lib, k=A[0], v=A[1], dtype=0, H=2, T=3, d=64, ks_h=192, ks_t=64, vs_h=192, vs_t=64, slots=A[2], pages=A[3],
           num_pages=5, sk=A[4], sv=A[5]):
    return lib.apa_cache_write(k, v, dtype, H, T, d, ks_h, ks_t, vs_h, vs_t, slots, pages, num_pages, sk, sv, None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(slots=None), -1), (dict(pages=None), -1), (dict(sk=None), -1),
    (dict(sv=None), -1), (dict(H=0), -2), (dict(T=-1), -2), (dict(num_pages=0), -2), (dict(num_pages=1 << 25), -2),
    (dict(d=32), -4), (dict(dtype=2), -11), (dict(dtype=-1), -11), (dict(k=P(0x10008)), -8), (dict(pages=P(0x10008)), -8),
    (dict(ks_h=100), -8), (dict(ks_t=65), -8), (dict(vs_h=4), -8), (dict(vs_t=-7), -8), (dict(T=0, k=None, v=None), 0),
])
def test_write_refusals(lib, kw, status):
    assert _write(lib, **kw) == status


def _read(lib, pages=A[0], num_pages=5, dtype=0, H=2, T=3, d=64, slots=A[1], sk=A[2], sv=A[3], k=A[4], v=A[5]):
    return lib.apa_cache_read(pages, num_pages, dtype, H, T, d, slots, sk, sv, k, v, None)


@pytest.mark.parametrize("kw,status", [
    (dict(pages=None), -1), (dict(slots=None), -1), (dict(sk=None), -1), (dict(sv=None), -1), (dict(k=None), -1),
    (dict(v=None), -1), (dict(H=0), -2), (dict(T=-1), -2), (dict(num_pages=0), -2), (dict(d=512), -4), (dict(dtype=7), -11),
    (dict(k=P(0x10004)), -8), (dict(T=0, k=None, v=None), 0),
])
def test_read_refusals(lib, kw, status):
    assert _read(lib, **kw) == status


def _attend(lib, q=A[0], dtype=0, sb=512, sh=64, sr=256, pages=A[1], num_pages=5, table=A[2], max_pages=4, lens=A[3],
            sk=A[4], sv=A[5], B=2, Hq=4, Hkv=2, Nq=2, d=64, window=0, sinks=0, out=A[6], ws=A[7], nbytes=1 << 40):
    return lib.apa_attention_cache(q, dtype, sb, sh, sr, pages, num_pages, table, max_pages, lens, sk, sv, B, Hq, Hkv, Nq, d,
                                   window, sinks, out, None, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), -1), (dict(pages=None), -1), (dict(table=None), -1), (dict(lens=None), -1), (dict(sk=None), -1),
    (dict(sv=None), -1), (dict(out=None), -1), (dict(B=0), -2), (dict(B=8193), -2), (dict(Hq=3), -2), (dict(Nq=0), -2),
    (dict(num_pages=0), -2), (dict(max_pages=0), -2), (dict(max_pages=1 << 28), -2), (dict(Nq=1 << 20), -2),
    (dict(d=80), -4), (dict(dtype=3), -11), (dict(window=-1), -12), (dict(sinks=-1), -12), (dict(q=P(0x10002)), -8),
    (dict(sr=12), -8), (dict(nbytes=16), -6), (dict(ws=P(0x10010)), -6),
])
def test_attention_cache_refusals(lib, kw, status):
    assert _attend(lib, **kw) == status


def test_sizes(lib):
    # 2.25 bytes per pair of values: codes and scales of K and V
    assert lib.apa_cache_page_bytes(8, 128) == 8 * 64 * 128 * 2 * 9 // 16
    assert lib.apa_cache_page_bytes(0, 128) == 0 and lib.apa_cache_page_bytes(8, 100) == 0
    one = lib.apa_attention_cache_workspace_bytes(1, 24, 8, 1, 128)
    assert one > 0 and one % 4 == 0
    # it grows with the rows that share a head's keys, not with the sequences (but for 4 bytes each)
    assert lib.apa_attention_cache_workspace_bytes(8192, 24, 8, 1, 128) <= one + 4 * 8192 + 256
    assert lib.apa_attention_cache_workspace_bytes(1, 24, 8, 2, 128) > one
    assert lib.apa_attention_cache_workspace_bytes(1, 5, 2, 1, 128) == 0
    assert lib.apa_attention_cache_workspace_bytes(1, 24, 8, 1, 96) == 0
    assert _lib.status_string(-11) != "unknown status" and _lib.status_string(-12) != "unknown status"


def test_bindings_refuse_host_tensors_and_other_types():
    import torch

    import mixed_precision_attention_gb300 as apa
    i32, f32 = torch.zeros(2, dtype=torch.int32), torch.ones(2)
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    pages = apa.cache_pages(3, 2, 64, device="cpu")
    assert pages.shape == (3, 2, 72 * 64) and pages.dtype is torch.uint8
    with pytest.raises(ValueError):
        apa.cache_pages(3, 2, 96, device="cpu")
    with pytest.raises(ValueError):
        apa.cache_tables(i32, i32, i32[None], i32, i32[:1], 4)
    with pytest.raises(ValueError):
        apa.cache_write(k, k, i32, pages, f32, f32)
    with pytest.raises(ValueError):
        apa.cache_read(pages, i32, f32, f32)
    with pytest.raises(ValueError):
        apa.attention_cache(k[None], pages, i32[None], i32[:1], f32, f32)
    with pytest.raises(ValueError):
        apa.attention_window(k[None], k[None], k[None], 4)
    for bad in (k.float(), k[0], None):
        with pytest.raises(TypeError):
            apa.cache_write(bad, k, i32, pages, f32, f32)
