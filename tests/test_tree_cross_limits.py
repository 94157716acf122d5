"""Refusals of drafted trees and cross attention at the ends of their ranges, on the host (CPU only: the fake pointers below
are never dereferenced, and what is not refused ends at the launch, without a GPU)."""
import pytest
import torch

from .test_tree_cross_abi import A, P, _accept, _cross, _draft, _tree, lib  # noqa: F401 (lib: the fixture)

W = 4  # bytes of a word


@pytest.mark.parametrize("of", ["lens", "nodes", "counts", "path", "table"])
@pytest.mark.parametrize("B,shift", [(2, 0), (2, 1), (2, -1), (300, 299), (300, -299)])
def test_accept_refuses_new_lens_inside_what_it_reads(lib, of, B, shift):  # noqa: F811
    """Other CTAs of a sequence may read these when its first has written new_lens."""
    at = dict(lens=A[2], nodes=A[3], counts=A[5], path=A[4], table=A[1])[of].value
    assert _accept(lib, B=B, new=P(at + W * shift)) == -2


@pytest.mark.parametrize("of,words", [("lens", 2), ("nodes", 2), ("counts", 2), ("path", 2 * 3), ("table", 2 * 4)])
def test_accept_takes_new_lens_next_to_what_it_reads(lib, of, words):  # noqa: F811
    at = dict(lens=A[2], nodes=A[3], counts=A[5], path=A[4], table=A[1])[of].value
    if torch.cuda.is_available():
        pytest.skip("would run on made-up pointers")
    for new in (at + W * words, at - W * 2):
        assert _accept(lib, new=P(new)) == -5
    assert _accept(lib, new=P(at + W * (words - 1))) == -2


def test_an_early_kernel_takes_tensor_memory_behind_its_wait():
    """A kernel that is launched while the one before it runs, and takes tensor memory before it waits for that, may keep it
    from ending: in every kernel text the wait comes first, and what follows is let in only when the columns are taken."""
    import glob
    import os
    import re

    from mixed_precision_attention_gb300 import build
    found = 0
    for path in glob.glob(os.path.join(build.CSRC, "*.cu*")):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for body in text.split("__global__")[1:]:
            wait, let = body.find('"griddepcontrol.wait;"'), body.find('"griddepcontrol.launch_dependents;"')
            take = body.find("tmem_alloc(")
            if take >= 0 and wait >= 0:
                found += 1
                assert wait < take, path
            if take >= 0 and let >= 0:
                assert take < let, path
    assert found == 1  # rows_kernel


# ------------------------------------------------------------------ lengths past 32 bits
LONG = 2 ** 32 + 2  # its lower 32 bits alone would be a size that is taken


def _bind(monkeypatch, module):
    """The binding without a GPU: what it hands on to the library."""
    got = []
    monkeypatch.setattr(module, "_empty", lambda *a, **k: torch.empty(4, dtype=torch.uint8))
    monkeypatch.setattr(module, "_enqueue", lambda index, name, *a: got.append(a))
    for name in ("_need_rows", "_need"):
        monkeypatch.setattr(module, name, lambda *a: 0)
    return got


@pytest.mark.parametrize("axis", [None, "B", "Hq", "Nq", "Hkv", "Nkv"])
def test_cross_binding_refuses_lengths_past_32_bits(lib, monkeypatch, axis):  # noqa: F811
    from mixed_precision_attention_gb300 import cross
    got = _bind(monkeypatch, cross)
    n = dict(dict(B=2, Hq=4, Nq=2, Hkv=2, Nkv=8), **({axis: LONG} if axis else {}))
    q = torch.empty_strided((n["B"], n["Hq"], n["Nq"], 64), (8, 8, 8, 1), dtype=torch.bfloat16, device="meta")
    k = torch.empty_strided((n["B"], n["Hkv"], n["Nkv"], 64), (8, 8, 8, 1), dtype=torch.bfloat16, device="meta")
    if axis:
        with pytest.raises(ValueError):
            cross.attention_cross(q, k, k)
    else:
        cross.attention_cross(q, k, k)
    assert len(got) == (0 if axis else 1)


@pytest.mark.parametrize("axis", [None, "B", "Hq", "Nq", "Hkv", "num_pages"])
def test_tree_binding_refuses_lengths_past_32_bits(lib, monkeypatch, axis):  # noqa: F811
    from mixed_precision_attention_gb300 import tree
    got = _bind(monkeypatch, tree)
    n = dict(dict(B=2, Hq=4, Nq=2, Hkv=2, num_pages=3), **({axis: LONG} if axis else {}))
    monkeypatch.setattr(tree, "_need_pool", lambda *a: (n["num_pages"], n["Hkv"], 64))
    monkeypatch.setattr(tree, "_need_tree", lambda *a: 0)
    q = torch.empty_strided((n["B"], n["Hq"], n["Nq"], 64), (8, 8, 8, 1), dtype=torch.bfloat16, device="meta")
    x = torch.empty(n["B"], 1, device="meta")
    if axis:
        with pytest.raises(ValueError):
            tree.attention_tree(q, x, x, x, None, x, x, x)
    else:
        tree.attention_tree(q, x, x, x, None, x, x, x)
    assert len(got) == (0 if axis else 1)


# ------------------------------------------------------------------ the sizes that the header names
def _taken(status):
    """Not refused: there is no GPU to launch on."""
    return status == -5


gpu_free = pytest.mark.skipif(torch.cuda.is_available(), reason="would run on made-up pointers")
ONE = dict(Hq=1, Hkv=1, Nq=1)  # (G * Nq + 255) / 128 = 2


@gpu_free
@pytest.mark.parametrize("kw,last,past", [
    (dict(ONE, B=32), dict(max_pages=2 ** 24 - 1), dict(max_pages=2 ** 24)),                          # B * max_pages
    (dict(ONE, B=1), dict(max_pages=2 ** 25 - 1), dict(max_pages=2 ** 25)),
    (dict(ONE, B=1), dict(num_pages=2 ** 25 - 1), dict(num_pages=2 ** 25)),
    (dict(B=64, Hq=257, Hkv=1, Nq=1), dict(max_pages=2 ** 23 - 17), dict(max_pages=2 ** 23 - 16)),     # U = 2^31: factor 4
    (dict(B=64, Hq=128, Hkv=128, Nq=1), dict(max_pages=2 ** 23 - 17), dict(max_pages=2 ** 23 - 16)),   # U * Hkv = 2^37
    (dict(B=1, Hkv=1, Nq=1024), dict(Hq=1024), dict(Hq=1025)),                                         # G * Nq = 2^20
    (dict(B=1, Nq=1), dict(Hq=2 ** 16, Hkv=2 ** 16), dict(Hq=2 ** 16 + 1, Hkv=2 ** 16 + 1)),
    (dict(Hq=2 ** 16, Hkv=2 ** 16, Nq=1), dict(B=8192), dict(B=8193)),
    (dict(Hq=2 ** 16, Hkv=2 ** 16, Nq=1023), dict(B=32), dict(B=33)),                                  # B * Hq * Nq
])
def test_tree_sizes(lib, kw, last, past):  # noqa: F811
    assert _taken(_tree(lib, **dict(kw, **last)))
    assert _tree(lib, **dict(kw, **past)) == -2


@gpu_free
@pytest.mark.parametrize("kw,last,past", [
    (dict(ONE, B=8192), dict(Nkv=64 * (2 ** 17 - 17)), dict(Nkv=64 * (2 ** 17 - 17) + 1)),             # U = 2^31
    (dict(B=4096, Hq=128, Hkv=128, Nq=1), dict(Nkv=64 * (2 ** 17 - 17)), dict(Nkv=64 * (2 ** 17 - 17) + 1)),
    (dict(ONE, B=1), dict(Nkv=2 ** 30), dict(Nkv=2 ** 30 + 1)),
    (dict(B=1), dict(Nq=2 ** 19), dict(Nq=2 ** 19 + 1)),                                               # G * Nq = 2^20
    (dict(Nq=2 ** 19), dict(B=1023), dict(B=1024)),                                                    # B * Hq * Nq
    (dict(ONE), dict(B=8192), dict(B=8193)),
    (dict(B=1, Nq=1), dict(Hq=2 ** 16, Hkv=2 ** 16), dict(Hq=2 ** 16 + 1, Hkv=2 ** 16 + 1)),
])
def test_cross_sizes(lib, kw, last, past):  # noqa: F811
    assert _taken(_cross(lib, **dict(kw, **last)))
    assert _cross(lib, **dict(kw, **past)) == -2


@gpu_free
def test_cross_strides(lib):  # noqa: F811
    assert _taken(_cross(lib, ks=(2 ** 39 - 8, 64, 128))) and _cross(lib, ks=(2 ** 39, 64, 128)) == -8
    assert _taken(_cross(lib, vs=(64, 2 ** 39 - 8, 128))) and _cross(lib, vs=(64, 2 ** 39, 128)) == -8


@gpu_free
@pytest.mark.parametrize("last,past", [
    (dict(layers=65535), dict(layers=65536)), (dict(Hkv=2 ** 16), dict(Hkv=2 ** 16 + 1)), (dict(most=1024), dict(most=1025)),
    (dict(num_pages=2 ** 25 - 1), dict(num_pages=2 ** 25))])
def test_accept_sizes(lib, last, past):  # noqa: F811
    assert _taken(_accept(lib, **last)) and _accept(lib, **past) == -2


@gpu_free
def test_draft_sizes_and_alignment(lib):  # noqa: F811
    assert _taken(_draft(lib, Nq=1024)) and _draft(lib, Nq=1025) == -2
    assert all(_draft(lib, Nq=n, mask=P(A[1].value + 4)) == -8 for n in (1, 5, 128))
