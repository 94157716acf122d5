"""Drafted trees and cross attention at the ends of their ranges: the largest block tables, keys that are no numbers in a
part of a split walk, scores far from 0, sizes past 32 bits, and a product of matrices right before the call."""
import math

import numpy as np
import pytest

from .test_gpu_cache import _cache, _torch, _types
from .test_gpu_tree import _attend, _i32, _parents
from .test_gpu_tree_cross_edges import _cross_inputs, _same, _step

pytestmark = pytest.mark.gpu

MOST_PAGES = (1 << 25) - 1  # of a block table


# ------------------------------------------------------------------ the largest tables
@pytest.mark.parametrize("Nq", [1, 63, 64, 130])
def test_tree_window_holds_under_the_largest_table(Nq):
    """64 * max_pages + Nq passes 2^31: the window and the sinks are those of a small table, bit for bit."""
    import torch

    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(Nq)
    a, _, _ = _step(rng, 1, 1, 1, Nq, 64, [1000], [Nq])
    table = torch.zeros(1, MOST_PAGES, dtype=torch.int32, device="cuda")
    table[:, : a["block_table"].shape[1]] = a["block_table"]
    for window, sinks in ((100, 4), (3, 0), (5000, 2), (0, 0)):
        want = apa.attention_tree(**a, window=window, sinks=sinks)
        got = apa.attention_tree(**dict(a, block_table=table), window=window, sinks=sinks)
        apa.check_error()
        assert _same(got, want), (window, sinks)
    assert not _same(apa.attention_tree(**a, window=100, sinks=4), apa.attention_tree(**a))


@pytest.mark.parametrize("Nq,nodes", [(1, 1), (64, 64), (130, 130), (1024, 64)])
def test_tree_of_a_full_largest_table(Nq, nodes):
    """A context up to the last key of the largest table, 2^31 - 64 keys: positions of nodes pass 2^31 where depths are any.
    Pages repeat, so a short context whose windows and sinks hold the same keys gives the same bits."""
    import torch

    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(Nq)
    held = 40
    a, _, _ = _step(rng, 1, 2, 1, Nq, 64, [64 * held - nodes], [nodes])
    if nodes < Nq:  # depths of no tree
        a["depths"] = _i32(rng.integers(0, Nq, (1, Nq)))
    table = torch.full((1, MOST_PAGES), -1, dtype=torch.int32, device="cuda")
    table[:, :held // 2] = a["block_table"][:, :held // 2]
    table[:, MOST_PAGES - held // 2:] = a["block_table"][:, held - held // 2:held]
    full = dict(a, block_table=table, lens=_i32([64 * MOST_PAGES]))
    for window, sinks in ((200, 70), (1, 0), (3, 1), (900, 1), (64, 64 * 15)):
        want = apa.attention_tree(**a, window=window, sinks=sinks)
        got = apa.attention_tree(**full, window=window, sinks=sinks)
        apa.check_error()  # (no page but those that hold visible keys is read: the others are -1)
        assert _same(got, want), (window, sinks)


def test_tree_sinks_past_every_position_of_the_largest_table():
    import torch

    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(1)
    a, _, _ = _step(rng, 1, 1, 1, 64, 64, [1000], [64])
    table = torch.zeros(1, MOST_PAGES, dtype=torch.int32, device="cuda")
    table[:, : a["block_table"].shape[1]] = a["block_table"]
    want = apa.attention_tree(**a)
    for sinks in (1064, 2 ** 31 - 64, 2 ** 31 - 1, 2 ** 40):
        assert _same(apa.attention_tree(**dict(a, block_table=table), window=2, sinks=sinks), want), sinks
    apa.check_error()


# ------------------------------------------------------------------ no numbers in a part of a split walk
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Nq", [1, 90, 150])
@pytest.mark.parametrize("at", [0, 300, 576])
def test_cross_a_key_that_is_no_number_reaches_every_row(d, Nq, at):
    """Every row sees it, so by the formula every output is NaN; key 576 is alone in the last of ten tiles, which a CTA of
    its own takes, and whose part has a sum but no maximum."""
    import mixed_precision_attention_gb300 as apa
    q, k, v = _cross_inputs(1, 4, 2, Nq, 577, d, seed=at)
    k[0, :, at, 3] = math.nan
    out, lse = apa.attention_cross(q, k, v)
    apa.check_error()
    assert out.isnan().all() and lse.isnan().all()
    want = apa.attention_cross(q[:, :2], k[:, :1], v[:, :1])
    k[0, 1, at, 3] = 0  # head 1 has numbers again, head 0 keeps its own
    got = apa.attention_cross(q, k, v)
    assert not got[0][:, 2:].isnan().any() and got[0][:, :2].isnan().all() and want[0].isnan().all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Nq", [3, 40])
@pytest.mark.parametrize("page", [0, 4, 9])
def test_tree_a_page_of_keys_that_are_no_numbers_reaches_the_rows_that_see_it(d, Nq, page):
    import torch

    import mixed_precision_attention_gb300 as apa
    a, _, _ = _step(np.random.default_rng(d + page), 1, 4, 1, Nq, d, [640], [Nq])
    want = apa.attention_tree(**a, window=200, sinks=1)
    pool = a["pages"][int(a["block_table"][0, page])].view(1, 4, 18 * d)
    pool[:, :, 16 * d: 17 * d] = 0x7F  # K's scales
    out, lse = apa.attention_tree(**a)
    apa.check_error()
    assert out.isnan().all() and lse.isnan().all()
    out, lse = apa.attention_tree(**a, window=200, sinks=1)  # page 4 lies between the sink and every window
    if page == 4:
        assert _same((out, lse), want)
    else:
        assert out.isnan().all() and lse.isnan().all()
