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


# ------------------------------------------------------------------ scores far from 0
def _far(out, lse, ref, ref_lse, size, half, limit, reach):
    """Rows whose largest score (ref_lse, but for the log of a sum of few weights) is beyond the limit, in log2 units, are
    NaN; of the others all are right but those with any score beyond it (reach: the largest magnitude), which may be NaN.
    What is rounded is the weights (half a step of 16 bits at most), their FP32 sums and the output; scores, sums of up to
    256 FP32 terms, are off by 256 * 2^-24 = 2^-16 of their size at most, and so is the lse.  Weights that the formula has
    below 2^-149 are 0 here: 2^-126 covers what they bring to an output."""
    ln2 = math.log(2)
    beyond = ref_lse.abs() >= limit * ln2 * 1.01
    within = ref_lse.abs() <= limit * ln2 * 0.99
    assert bool(out[beyond].isnan().all()) and bool(lse[beyond].isnan().all())
    tol = size * (half + 2 ** -14) + ref.abs() * half + 2.0 ** -126
    right = ((out.double() - ref).abs() <= tol).all(-1)
    may = within & (reach >= limit * ln2 * 0.99) & out.isnan().all(-1)
    assert bool((right | may)[within].all())
    assert bool(((lse.double() - ref_lse).abs() <= ref_lse.abs() * 2 ** -16 + 2 ** -14)[within & right].all())
    return int(beyond.sum()), int((within & right).sum())


LIMIT = {"bf16": 2.0 ** 29, "fp16": 2.0 ** 24}  # by the type of the weights


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("power", [3, 6, 9, 12, 14])
@pytest.mark.parametrize("sign", [1, -1])
def test_cross_scores_far_from_zero(dtype, d, power, sign):
    """q.k / sqrt(d) of up to 2^32 or from -2^31: the largest scores win and equal ones share, up to the stated limit."""
    import torch

    import mixed_precision_attention_gb300 as apa
    from .test_gpu_cross import formula
    t = _types()[dtype]
    g = torch.Generator(device="cuda")
    g.manual_seed(power)
    N, Nq = 700, 40
    step = torch.randint(1, 4, (1, 2, N, 1), device="cuda", generator=g).double()   # a key's size, 1 .. 3 eighths below
    for at in (2, 5, 77, 500, 699):                                                # the ones of the largest score
        step[:, :, at] = 0 if sign > 0 else 4
    u = 1 - 2 * torch.randint(0, 2, (1, 1, 1, d), device="cuda", generator=g).double()
    k = (u * sign * 2.0 ** power * (1 - step / 8)).to(t).expand(1, 2, N, d).contiguous()
    q = (u * 2.0 ** power).to(t).expand(1, 4, Nq, d).contiguous()
    v = torch.randn(1, 2, N, d, device="cuda", generator=g).to(t)
    out, lse = apa.attention_cross(q, k, v)
    apa.check_error()
    if power > 3:  # (below, more keys than the largest have weight, which formula() counts as well)
        w = torch.softmax(q[0, 0, :1].double() @ k[0, 0].double().T / math.sqrt(d), -1)
        assert int((w > 2.0 ** -100).sum()) == 5
    ref, ref_lse, size = formula(q, k, v, [N])
    most = (q[:, :, :1].double() @ k.repeat_interleave(2, 1).double().transpose(2, 3)).abs().max() / math.sqrt(d)
    beyond, right = _far(out, lse, ref, ref_lse, size, torch.finfo(t).eps / 2, LIMIT[dtype], most)
    assert beyond + right == lse.numel() and (power < 10 or dtype == "bf16" and power < 13 or beyond == lse.numel())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Nq", [3, 60])
@pytest.mark.parametrize("up", [8, 20, 30, 60])
def test_tree_scores_far_from_zero(d, Nq, up):
    """Keys scaled up by powers of two, through their head scales."""
    import torch

    import mixed_precision_attention_gb300 as apa
    a, kv, parents = _step(np.random.default_rng(d + up), 2, 4, 2, Nq, d, [500, 70], [Nq, Nq])
    scale = 2.0 ** up
    a["k_scale"] = a["k_scale"] * scale
    a["q"] = a["q"].round() * 16  # (whole numbers)
    from .test_gpu_tree import _tree
    sees, depths = _tree(parents, [Nq, Nq])
    q = a["q"].double().cpu().numpy()
    lens = [500 + Nq, 70 + Nq]
    far = [np.stack([x[0] * scale, x[1]]) for x in kv]
    ref, ref_lse, mag = _attend(q, far, lens, [Nq, Nq], sees, depths, 0, 0)
    out, lse = apa.attention_tree(**a)
    apa.check_error()
    # a row counts where its largest score leaves the next different one 200 behind after an error of 2^-15 of it
    sure, reach = np.zeros(ref_lse.shape, bool), np.zeros(ref_lse.shape)
    for b in range(2):
        vis = np.ones((Nq, lens[b]), bool)
        vis[:, lens[b] - Nq:] = sees[b]
        for h in range(4):
            s = np.where(vis, q[b, h] @ far[b][0][h // 2].T / math.sqrt(d), -np.inf)
            top = s.max(1, keepdims=True)
            sure[b, h] = ~((s < top) & (s > top - 200 - np.abs(top) * 2.0 ** -15)).any(1)
            reach[b, h] = np.where(vis, np.abs(s), 0).max(1)
    at = np.nonzero(sure)
    pick = lambda x: _torch(x[at]) if isinstance(x, np.ndarray) else x[tuple(_torch(i) for i in at)]  # noqa: E731
    beyond, right = _far(pick(out), pick(lse), pick(ref), pick(ref_lse), pick(mag), 2.0 ** -8, LIMIT["fp16"], pick(reach))
    assert beyond > 0 if up >= 20 else beyond == 0 and right > 0


# ------------------------------------------------------------------ the accepted path
@pytest.mark.parametrize("layers,H,B,Nq,most", [(6, 6, 300, 9, 5), (1, 20, 1500, 6, 6), (2, 257, 40, 20, 4)])
def test_cache_accept_several_heads_of_a_cta(layers, H, B, Nq, most):
    """Where layers, sequences and heads are many a CTA takes two, four or more heads, the last one what is left."""
    import mixed_precision_attention_gb300 as apa
    from .test_gpu_tree import _accept
    rng = np.random.default_rng(B)
    base = rng.integers(0, 64, B)
    nodes = rng.integers(1, Nq + 1, B)
    lens = base + nodes
    held = (lens + 63) // 64
    table, at = np.full((B, 2), -1), np.cumsum(held) - held
    ids = rng.permutation(int(held.sum()))
    for b in range(B):
        table[b, :held[b]] = ids[at[b]:at[b] + held[b]]
    counts = np.minimum(rng.integers(0, most + 1, B), nodes)
    path = np.full((B, most), 7)
    for b in range(B):
        path[b, :counts[b]] = np.sort(rng.choice(nodes[b], counts[b], replace=False))
    pages = rng.integers(0, 256, (layers, len(ids), H, 72 * 64), dtype=np.uint8)
    want = _accept(pages, table, base, path, counts)
    p = _torch(pages)
    new = apa.cache_accept(p, _i32(table), _i32(lens), _i32(nodes), _i32(path), _i32(counts))
    apa.check_error()
    assert np.array_equal(new.cpu().numpy(), base + counts)
    assert np.array_equal(p.cpu().numpy(), want)


# ------------------------------------------------------------------ behind a product of matrices
@pytest.mark.parametrize("d,Nq", [(64, 20), (128, 20), (128, 60), (256, 20)])
def test_calls_right_behind_products_of_matrices(d, Nq):
    """As a layer makes them: q out of a projection just before, the output into one just behind, many times without a
    wait, and captured."""
    import torch

    import mixed_precision_attention_gb300 as apa
    B, Hq, H, N = 3, 4, 2, 300
    a, _, _ = _step(np.random.default_rng(d + Nq), B, Hq, H, Nq, d, [500, 3, 70], [Nq, 1, Nq])
    _, k, v = _cross_inputs(B, Hq, H, Nq, N, d)
    wide = Hq * d
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    w1, w2 = (torch.randn(wide, wide, device="cuda", generator=g).div_(math.sqrt(wide)).bfloat16() for _ in range(2))
    x = torch.randn(B, Nq, wide, device="cuda", generator=g).bfloat16()
    rows = lambda y: y.view(B, Nq, Hq, d).transpose(1, 2)  # noqa: E731
    flat = lambda y: y.transpose(1, 2).reshape(B, Nq, wide)  # noqa: E731

    def layer(x, wait=lambda: None):
        y = x @ w1
        wait()
        t, _ = apa.attention_tree(**dict(a, q=rows(y)))
        wait()
        y = flat(t) @ w2
        wait()
        c, _ = apa.attention_cross(rows(y), k, v)
        wait()
        return flat(c) @ w1

    want = x
    for _ in range(4):
        want = layer(want, torch.cuda.synchronize)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()

    def run():
        y = x
        for _ in range(4):
            y = layer(y)
        return y

    with torch.cuda.stream(side):
        eager = run()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        captured = run()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    apa.check_error()
    assert torch.equal(eager, want) and torch.equal(captured, want)


# ------------------------------------------------------------------ sizes past 32 bits
def test_cross_refuses_sizes_past_32_bits():
    """An expanded axis may be longer than 2^32: its length does not lose its upper bits on the way."""
    import mixed_precision_attention_gb300 as apa
    q, k, v = _cross_inputs(1, 4, 1, 3, 40, 64)
    apa.attention_cross(q, k.expand(1, 2, 40, 64), v.expand(1, 2, 40, 64))
    for heads in (2 ** 32 + 1, 2 ** 32 + 2, 2 ** 31):
        with pytest.raises(ValueError):
            apa.attention_cross(q, k.expand(1, heads, 40, 64), v.expand(1, heads, 40, 64))
    apa.check_error()


# ------------------------------------------------------------------ short lists
@pytest.mark.parametrize("B,Hq,H,Nq,N,d", [(1, 24, 8, 1, 1500, 128), (1, 24, 8, 64, 1500, 128), (1, 8, 8, 100, 700, 256),
                                           (1, 24, 8, 26, 1026, 64), (3, 6, 2, 333, 1021, 256), (1, 1, 1, 1, 64, 128)])
def test_cross_lists_that_leave_ctas_without_a_tile(B, Hq, H, Nq, N, d):
    import mixed_precision_attention_gb300 as apa
    from .test_gpu_cross import check
    q, k, v = _cross_inputs(B, Hq, H, Nq, N, d, seed=N)
    lens = [N, max(1, N // 3), N][:B]
    got = apa.attention_cross(q, k, v, _i32(lens))
    apa.check_error()
    check(q, k, v, lens, got)
    assert _same(got, apa.attention_cross(q, k, v, _i32(lens)))


@pytest.mark.parametrize("Hq,H,Nq,d,base", [(24, 8, 26, 128, 1000), (24, 8, 60, 128, 1400), (8, 8, 100, 256, 600), (16, 4, 5, 64, 700)])
def test_tree_lists_that_leave_ctas_without_a_tile(Hq, H, Nq, d, base):
    import mixed_precision_attention_gb300 as apa
    from .test_gpu_cache import _near
    from .test_gpu_tree import _tree
    a, kv, parents = _step(np.random.default_rng(Nq), 1, Hq, H, Nq, d, [base], [Nq])
    got = apa.attention_tree(**a)
    apa.check_error()
    sees, depths = _tree(parents, [Nq])
    _near(*got, _attend(a["q"].double().cpu().numpy(), kv, [base + Nq], [Nq], sees, depths, 0, 0), "bf16")
    assert _same(got, apa.attention_tree(**a))
