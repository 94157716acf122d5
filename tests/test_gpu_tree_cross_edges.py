"""Drafted trees and cross attention where they can go wrong: hidden values that are no numbers, strides and shared axes,
lengths out of range, reruns, streams and graphs, sizes past 32 bits, and a whole step of both together."""
import math

import numpy as np
import pytest

from .test_gpu_cache import _cache, _near, _quantize, _torch, _types, _value
from .test_gpu_tree import _attend, _i32, _parents, _tree, _words

pytestmark = pytest.mark.gpu


def _cross_inputs(B, Hq, H, Nq, N, d, seed=0, dtype=None):
    from .test_gpu_cross import BF16, inputs
    return inputs(B, Hq, H, Nq, N, d, dtype or BF16, seed)


def _same(a, b):
    import torch
    return all(torch.equal(x.view(torch.int16 if x.dtype.itemsize == 2 else torch.int32),
                           y.view(torch.int16 if y.dtype.itemsize == 2 else torch.int32)) for x, y in zip(a, b))


# ------------------------------------------------------------------ cross attention
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Nq", [1, 90])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_cross_keys_behind_the_end_are_never_used(d, Nq, what):
    import mixed_precision_attention_gb300 as apa
    lens = [130, 1, 64, 0, 63, 300]
    q, k, v = _cross_inputs(6, 4, 2, Nq, 300, d)
    want = apa.attention_cross(q, k, v, _i32(lens))
    for b, n in enumerate(lens):
        k[b, :, n:] = what
        v[b, :, n:] = what
    got = apa.attention_cross(q, k, v, _i32(lens))
    apa.check_error()
    assert _same(got, want) and not got[0].isnan().any()


def test_cross_what_is_no_number_stays_in_its_rows():
    import torch

    import mixed_precision_attention_gb300 as apa
    q, k, v = _cross_inputs(2, 4, 2, 5, 200, 128, seed=3)
    want = apa.attention_cross(q, k, v)
    q[0, 1, 2, 7] = math.nan
    out, lse = apa.attention_cross(q, k, v)
    hit = torch.zeros(2, 4, 5, dtype=torch.bool, device="cuda")
    hit[0, 1, 2] = True
    assert out[hit].isnan().all() and lse[hit].isnan().all()
    assert torch.equal(out[~hit], want[0][~hit]) and torch.equal(lse[~hit], want[1][~hit])
    q, k, v = _cross_inputs(2, 4, 2, 5, 200, 128, seed=3)
    v[1, 0, 199, 3] = math.nan  # a key that heads 0 and 1 of sequence 1 see
    out, lse = apa.attention_cross(q, k, v)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[1, :2, :, 3] = True
    assert torch.equal(out.isnan(), hit) and torch.equal(lse, want[1])
    assert torch.equal(out[~hit], want[0][~hit])


@pytest.mark.parametrize("d", [64, 128, 256])
def test_cross_strides_and_shared_axes(d):
    """Any strides that are multiples of 8, k and v of their own; one encoder for all sequences; one head for all."""
    import torch

    import mixed_precision_attention_gb300 as apa
    B, Hq, H, Nq, N = 3, 6, 2, 20, 150
    lens = _i32([150, 77, 64])
    q, k, v = (x.contiguous() for x in _cross_inputs(B, Hq, H, Nq, N, d, seed=d))
    want = apa.attention_cross(q, k, v, lens)

    def spread(x, order, pad):  # x with its axes laid out in another order, rows pad elements apart
        y = torch.full([x.shape[i] for i in order] + [d + pad], math.nan, dtype=x.dtype, device="cuda")
        back = [order.index(i) for i in range(3)]
        y = y[..., :d].permute(back + [3])
        y.copy_(x)
        return y

    for oq, ok, ov, pad in (((2, 0, 1), (1, 2, 0), (0, 2, 1), 8), ((0, 1, 2), (2, 1, 0), (2, 0, 1), 24), ((1, 0, 2), (0, 1, 2), (1, 0, 2), 0)):
        assert _same(apa.attention_cross(spread(q, oq, pad), spread(k, ok, pad), spread(v, ov, 2 * pad), lens), want)
    one = apa.attention_cross(q, k[:1].expand(B, H, N, d), v[:1].expand(B, H, N, d), lens)
    each = apa.attention_cross(q, k[:1].repeat(B, 1, 1, 1), v[:1].repeat(B, 1, 1, 1), lens)
    assert _same(one, each)
    one = apa.attention_cross(q, k[:, :1].expand(B, H, N, d), v, lens)
    each = apa.attention_cross(q, k[:, :1].repeat(1, H, 1, 1), v, lens)
    assert _same(one, each)
    # strides of axes of length 1 are not looked at
    q1, k1, v1 = q[:1, :1, :1], k[:1, :1, :1], v[:1, :1, :1]
    want = apa.attention_cross(q1.contiguous(), k1.contiguous(), v1.contiguous())
    odd = [torch.as_strided(x, (1, 1, 1, d), (3, 5, 7, 1)) for x in (q1, k1, v1)]
    assert _same(apa.attention_cross(*odd), want)
    with pytest.raises(apa.ApaError):  # a token stride of 0
        apa.attention_cross(q, k[:, :, :1].expand(B, H, N, d), v, lens)
    with pytest.raises(apa.ApaError):
        apa.attention_cross(spread(q, (0, 1, 2), 4), k, v, lens)


def test_cross_lengths_out_of_range_are_clamped_and_reported():
    import mixed_precision_attention_gb300 as apa
    q, k, v = _cross_inputs(3, 4, 2, 3, 100, 64)
    want = apa.attention_cross(q, k, v, _i32([100, 0, 7]))
    for bad in ([101, 0, 7], [100, -1, 7], [2 ** 31 - 1, -2 ** 31, 7]):
        got = apa.attention_cross(q, k, v, _i32(bad))
        with pytest.raises(apa.ApaError):
            apa.check_error()
        assert _same(got, want)
    apa.check_error()


def test_cross_refusals_of_the_binding():
    import torch

    import mixed_precision_attention_gb300 as apa
    q, k, v = _cross_inputs(2, 4, 2, 3, 10, 64)
    ok = dict(q=q, k=k, v=v)
    for kw, err in ((dict(k=k.half()), ValueError), (dict(v=v[:, :, :5]), ValueError), (dict(q=q[:1]), ValueError),
                    (dict(k=k[..., :32], v=v[..., :32]), ValueError), (dict(lens=_i32([1])), ValueError),
                    (dict(lens=torch.tensor([1, 2], device="cuda")), TypeError), (dict(lens=torch.tensor([1, 2], dtype=torch.int32)), ValueError),
                    (dict(q=q.transpose(2, 3)), ValueError), (dict(q=q.double()), TypeError), (dict(k=k[:, :0], v=v[:, :0]), Exception),
                    (dict(q=q[:, :3]), apa.ApaError), (dict(q=q[:, :, :0]), apa.ApaError), (dict(k=k[:, :, :0], v=v[:, :, :0]), apa.ApaError),
                    (dict(workspace=torch.empty(1000, dtype=torch.uint8, device="cuda")), apa.ApaError)):
        with pytest.raises(err):
            apa.attention_cross(**dict(ok, **kw))
    out, lse = apa.attention_cross(q, k, v, return_lse=False)
    assert lse is None and torch.equal(out, apa.attention_cross(q, k, v)[0])


@pytest.mark.parametrize("B,Hq,H,Nq,N,d", [(8192, 1, 1, 1, 40, 64), (3000, 4, 2, 1, 70, 128), (1, 128, 1, 3, 9000, 128),
                                           (1, 4, 1, 5000, 130, 64), (2, 3, 1, 1000, 700, 128), (1, 8, 1, 300, 2000, 256)])
def test_cross_many_sequences_rows_and_keys(B, Hq, H, Nq, N, d):
    import torch

    import mixed_precision_attention_gb300 as apa
    q, k, v = _cross_inputs(B, Hq, H, Nq, N, d, seed=B)
    rng = np.random.default_rng(B)
    lens = rng.integers(0, N + 1, B)
    lens[0] = N
    got = apa.attention_cross(q, k, v, _i32(lens))
    assert _same(got, apa.attention_cross(q, k, v, _i32(lens)))  # bit for bit
    apa.check_error()
    from .test_gpu_cross import check
    pick = torch.arange(B)[:: max(1, B // 40)]
    sub = lambda x: x[pick.to(x.device)]  # noqa: E731
    check(sub(q), sub(k), sub(v), lens[pick.numpy()].tolist(), tuple(sub(x) for x in got))


def test_cross_keys_past_32_bits():
    import torch

    import mixed_precision_attention_gb300 as apa
    from .test_gpu_cross import check
    H, N, d = 8, 2_200_000, 128  # 2.25e9 elements
    k, v = (torch.empty(1, H, N, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for x in (k, v):
        for h in range(H):
            x[0, h].normal_()
    q = torch.randn(1, H, 1, d, dtype=torch.bfloat16, device="cuda") * 3
    got = apa.attention_cross(q, k, v)
    apa.check_error()
    for h in (0, H - 1):
        check(q[:, h:h + 1], k[:, h:h + 1], v[:, h:h + 1], [N], tuple(x[:, h:h + 1] for x in got))


# ------------------------------------------------------------------ trees
def _step(rng, B, Hq, H, Nq, d, base, nodes, dtype="bf16", most=None):
    import mixed_precision_attention_gb300 as apa
    lens = np.array(base) + np.array(nodes)
    pages, table, ks, vs, kv = _cache(rng, B, H, d, lens, most or int(max(lens)) // 64 + 2)
    parents = _parents(rng, B, Nq, "tree")
    t = apa.draft_tree(_i32(parents), _i32(nodes))
    q = _torch(rng.standard_normal((B, Hq, Nq, d)) * 2, _types()[dtype])
    return dict(q=q, pages=pages, block_table=table, lens=_i32(lens), nodes=_i32(nodes), mask=t["mask"], k_scale=_torch(ks),
                v_scale=_torch(vs), depths=t["depths"]), kv, parents


@pytest.mark.parametrize("d,Nq", [(64, 20), (128, 20), (128, 45), (256, 20)])
def test_tree_any_mask(d, Nq):
    """Bits that are no tree's: later nodes, none at all; rows that see nothing; one mask for all sequences."""
    import torch

    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(d + Nq)
    base, nodes = np.array([0, 130, 50]), np.array([Nq, Nq - 3, 1])
    a, kv, _ = _step(rng, 3, 8, 2, Nq, d, base, nodes)
    sees = rng.integers(0, 3, (1, Nq, Nq)) == 0
    sees[:, 4] = False
    sees[:, 5] = True
    depths = rng.integers(0, Nq, (1, Nq))
    a.update(mask=_torch(_words(sees)), depths=_i32(depths))
    for window, sinks in ((0, 0), (9, 0), (60, 2)):
        out, lse = apa.attention_tree(**a, window=window, sinks=sinks)
        apa.check_error()
        ref = _attend(a["q"].double().cpu().numpy(), kv, base + nodes, nodes, np.repeat(sees, 3, 0), np.repeat(depths, 3, 0), window, sinks)
        _near(out, lse, ref, "bf16")
        each = apa.attention_tree(**dict(a, mask=a["mask"].expand(3, -1, -1).contiguous(), depths=a["depths"].expand(3, -1)),
                                  window=window, sinks=sinks)
        assert _same((out, lse), each)
    assert torch.isneginf(lse[0, :, 4]).all() and not out[0, :, 4].any()


def test_tree_of_a_chain_is_causal_attention():
    """A chain's rows are those of attention_cache; the two differ by their roundings."""
    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(5)
    lens = np.array([300, 64, 9, 1000])
    pages, table, ks, vs, kv = _cache(rng, 4, 2, 128, lens, 17)
    q = _torch(rng.standard_normal((4, 6, 9, 128)), _types()["fp16"])
    chain = apa.draft_tree(_i32(_parents(rng, 1, 9, "chain")))
    sees, depths = _tree(_parents(rng, 4, 9, "chain"), [9] * 4)
    for window, sinks in ((0, 0), (5, 0), (70, 4)):
        a = apa.attention_tree(q, pages, table, _i32(lens), None, chain["mask"], _torch(ks), _torch(vs), depths=chain["depths"],
                               window=window, sinks=sinks)
        b = apa.attention_cache(q, pages, table, _i32(lens), _torch(ks), _torch(vs), window=window, sinks=sinks)
        ref = _attend(q.double().cpu().numpy(), kv, lens, [9] * 4, sees, depths, window, sinks)
        _near(*a, ref, "fp16")
        _near(*b, ref, "fp16")
    apa.check_error()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 3)])
def test_tree_keys_that_no_row_sees(d, window, sinks):
    """Pages behind the end, keys behind it in the last page, and keys between the sinks and every window: NaN there
    changes nothing."""
    import torch

    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(d)
    a, _, _ = _step(rng, 2, 4, 2, 12, d, [400, 30], [12, 7])
    want = apa.attention_tree(**a, window=window, sinks=sinks)
    if window:
        lo, hi = sinks, 400 - window + 1  # of sequence 0: hidden from its root, and so from all
        for j in range(lo, hi):
            page, i = int(a["block_table"][0, j // 64]), j % 64
            blk, at = i // 16 * 18 * d, i % 16
            t = torch.arange(d // 16, device="cuda")
            a["pages"][page, :, blk + 16 * d + at * (d // 16) + t] = 0x7F
            a["pages"][page, :, blk + 17 * d + 4 * ((at // 4) * (d // 16) + t) + at % 4] = 0x7F
    got = apa.attention_tree(**a, window=window, sinks=sinks)
    apa.check_error()
    assert _same(got, want) and not want[0].isnan().any()


def test_tree_lengths_and_pages_out_of_range():
    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(8)
    a, _, _ = _step(rng, 2, 4, 2, 6, 64, [100, 40], [6, 4], most=2)
    for kw, as_if in ((dict(lens=_i32([1000, 44])), dict(lens=_i32([128, 44]))), (dict(lens=_i32([-3, 44])), dict(lens=_i32([0, 44]), nodes=_i32([0, 4]))),
                      (dict(nodes=_i32([7, 4])), dict(nodes=_i32([6, 4]))), (dict(nodes=_i32([-1, 4])), dict(nodes=_i32([0, 4]))),
                      (dict(lens=_i32([3, 44])), dict(lens=_i32([3, 44]), nodes=_i32([3, 4])))):
        got = apa.attention_tree(**dict(a, **kw))
        with pytest.raises(apa.ApaError):
            apa.check_error()
        # (the page behind the end that the first reads holds NaN scales; nothing faults)
        want = apa.attention_tree(**dict(a, **as_if))
        apa.check_error()
        assert _same(got, want)
    table = a["block_table"].clone()
    table[0, 1] = 10 ** 6
    got = apa.attention_tree(**dict(a, block_table=table))
    with pytest.raises(apa.ApaError):
        apa.check_error()
    assert got[0].shape == a["q"].shape


def test_tree_refusals_of_the_binding():
    import torch

    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(9)
    a, _, _ = _step(rng, 2, 4, 2, 40, 64, [100, 40], [40, 4])
    for kw, err in ((dict(q=a["q"].float()), TypeError), (dict(mask=a["mask"].long()), TypeError), (dict(mask=a["mask"][:, :39]), ValueError),
                    (dict(mask=a["mask"][..., :1]), ValueError), (dict(mask=a["mask"].transpose(1, 2).contiguous().transpose(1, 2)), ValueError),
                    (dict(depths=a["depths"][:, 1:]), ValueError), (dict(depths=a["depths"].cpu()), ValueError),
                    (dict(depths=None, window=4), ValueError), (dict(lens=a["lens"][:1]), ValueError), (dict(nodes=a["nodes"][:1]), ValueError),
                    (dict(window=-1), apa.ApaError), (dict(sinks=-2 ** 40), apa.ApaError), (dict(q=a["q"][:, :3]), apa.ApaError),
                    (dict(q=a["q"][..., :32]), ValueError), (dict(pages=a["pages"][:, :, 1:]), ValueError),
                    (dict(workspace=torch.empty(4096, dtype=torch.uint8, device="cuda")), apa.ApaError)):
        with pytest.raises(err):
            apa.attention_tree(**dict(a, **kw))
    assert apa.attention_tree(**a, return_lse=False)[1] is None
    for window, sinks in ((2 ** 32 + 1, 0), (2 ** 31, 7), (1, 2 ** 32)):  # past every position
        assert _same(apa.attention_tree(**a, window=window, sinks=sinks), apa.attention_tree(**a))
    path, counts = _i32([[0, 1], [0, 1]]), _i32([1, 1])
    args = (a["pages"], a["block_table"], a["lens"], a["nodes"], path, counts)
    for i, x in ((0, a["pages"].float()), (0, a["pages"][:, :, ::2]), (1, a["block_table"][:1]), (2, a["lens"].long()), (3, None), (4, path[0]),
                 (4, path[:1]), (5, counts.cpu())):
        with pytest.raises((TypeError, ValueError)):
            apa.cache_accept(*(x if k == i else y for k, y in enumerate(args)))


@pytest.mark.parametrize("B,Hq,H,Nq,d", [(8192, 1, 1, 2, 64), (2000, 4, 1, 5, 128), (1, 32, 1, 1024, 64), (1, 3, 1, 1024, 128), (1, 2, 1, 600, 256)])
def test_tree_many_sequences_and_nodes(B, Hq, H, Nq, d):
    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(B + Nq)
    base, nodes = rng.integers(0, 70, B), rng.integers(0, Nq + 1, B)
    nodes[0] = Nq
    a, kv, parents = _step(rng, B, Hq, H, Nq, d, base, nodes)
    got = apa.attention_tree(**a)
    assert _same(got, apa.attention_tree(**a))  # bit for bit
    apa.check_error()
    pick = np.arange(0, B, max(1, B // 30))
    rows = np.arange(0, Nq, max(1, Nq // 60))
    sees, depths = _tree(parents[pick], nodes[pick])
    q = a["q"][_torch(pick)].double().cpu().numpy()
    if Nq > 100:  # the reference's rows, a few of them
        sees = np.where(np.isin(np.arange(Nq), rows)[None, :, None], sees, False)
    ref = _attend(q, [kv[b] for b in pick], (base + nodes)[pick], nodes[pick], sees, depths, 0, 0)
    sub = lambda x, r: x[_torch(pick)][:, :, _torch(r)]  # noqa: E731
    _near(sub(got[0], rows), sub(got[1], rows), tuple(x[:, :, rows] for x in ref), "bf16")


def test_tree_a_pool_past_32_bits():
    import torch

    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(11)
    P, H, d, base, nodes = 60000, 8, 128, 200, 9  # 4.4e9 bytes
    pages = torch.full((P, H, 72 * d), 0x7F, dtype=torch.uint8, device="cuda")
    small, table, ks, vs, kv = _cache(rng, 1, H, d, [base + nodes], 5)
    far = table.clone()
    for e in range(4):
        far[0, e] = P - 1 - e
        pages[P - 1 - e] = small[int(table[0, e])]
    parents = _parents(rng, 1, nodes, "tree")
    t = apa.draft_tree(_i32(parents))
    q = _torch(rng.standard_normal((1, 2 * H, nodes, d)), torch.bfloat16)
    args = (_i32([base + nodes]), None, t["mask"], _torch(ks), _torch(vs))
    assert _same(apa.attention_tree(q, pages, far, *args), apa.attention_tree(q, small, table, *args))
    move = (_i32([base + nodes]), _i32([nodes]), _i32([[0, 4, 8]]), _i32([3]))
    apa.cache_accept(pages, far, *move)
    apa.cache_accept(small, table, *move)
    apa.check_error()
    for e in range(4):
        assert torch.equal(pages[P - 1 - e], small[int(table[0, e])])


# ------------------------------------------------------------------ together
def test_two_streams_at_once():
    import torch

    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(12)
    steps = [_step(rng, 3, 6, 2, Nq, d, [700, 64, 1], [Nq, 3, 1])[0] for d, Nq in ((64, 11), (128, 50))]
    cross = [_cross_inputs(4, 6, 2, n, 500, 128, seed=n) for n in (1, 70)]
    lens = _i32([500, 3, 64, 0])
    run = lambda i: (*apa.attention_tree(**steps[i]), *apa.attention_cross(*cross[i], lens))  # noqa: E731
    want = [run(0), run(1)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(i))
    torch.cuda.synchronize()
    apa.check_error()
    assert all(_same(x, want[i]) for i in range(2) for x in got[i])


def test_speculative_steps_in_a_graph():
    """Steps of a decoder with drafts and an encoder, captured once and replayed: tables grow by the drafted tokens, their
    keys are written, the tree is attended to and the encoder read, the accepted keys move, tables shrink."""
    import torch

    import mixed_precision_attention_gb300 as apa
    rng = np.random.default_rng(21)
    B, Hq, H, Nq, d, N, pool = 3, 6, 2, 24, 128, 90, 24
    i32 = lambda a: _i32(np.asarray(a))  # noqa: E731
    free, count = i32(np.arange(pool)[::-1].copy()), i32([pool])
    table, pages = i32(np.full((B, 6), -1)), torch.zeros(2, pool, H, 72 * d, dtype=torch.uint8, device="cuda")
    ks = vs = _torch(np.full(H, 4 / 2688, np.float32))
    base, lens, nodes = i32([0] * B), i32([0] * B), i32([0] * B)
    parents, path, counts = i32(np.full((B, Nq), -1)), i32(np.zeros((B, 5))), i32([0] * B)
    kn, vn = (torch.zeros(H, B * Nq, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(B, Hq, Nq, d, dtype=torch.bfloat16, device="cuda")
    _, ek, ev = _cross_inputs(B, Hq, H, 1, N, d, seed=4)
    enc = i32([90, 17, 64])

    def check_drafts():
        lens.copy_(base + nodes)
        tree = apa.draft_tree(parents, nodes)
        t = apa.cache_tables(base, lens, table, free, count, B * Nq, free_count_out=count)
        for layer in range(2):
            apa.cache_write(kn, vn, t["slots"], pages[layer], ks, vs)
        out, lse = apa.attention_tree(q, pages[1], table, lens, nodes, tree["mask"], ks, vs)
        return out, lse, apa.attention_cross(out, ek, ev, enc), t

    def keep():
        new = apa.cache_accept(pages, table, lens, nodes, path, counts)
        apa.cache_tables(lens, new, table, free, count, 0, free_count_out=count)
        base.copy_(new)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0], stream=side):
        out, lse, (cout, clse), t = check_drafts()
    with torch.cuda.graph(graphs[1], stream=side):
        keep()
    from .test_gpu_cross import check
    # per sequence, what the cache stands for, and what reading it in FP16 gives
    kept, seen = ([np.zeros((2, H, 0, d)) for _ in range(B)] for _ in range(2))
    scale = ks.double().cpu().numpy()[:, None, None]
    for step in range(6):
        n = rng.integers(1, Nq + 1, B)
        p = _parents(rng, B, Nq, "tree")
        nodes.copy_(i32(n))
        parents.copy_(i32(p))
        for x in (kn, vn, q):
            x.copy_(_torch(rng.standard_normal(x.shape), torch.bfloat16))
        graphs[0].replay()
        torch.cuda.synchronize()
        apa.check_error()
        had = [k.shape[2] for k in kept]
        drafted, read, at = [], [], 0
        for b in range(B):  # the drafted tokens' values
            part = slice(at, at + int(n[b]))
            drafted.append(np.stack([_value(*_quantize(x[:, part].double().cpu().numpy(), scale)) * scale for x in (kn, vn)]))
            read.append(np.stack([x.double().cpu().numpy() for x in apa.cache_read(pages[1], t["slots"][part], ks, vs, dtype=torch.float16)]))
            at += int(n[b])
        kv = [np.concatenate([kept[b], drafted[b]], 2) for b in range(B)]
        sees, depths = _tree(p, n)
        ref = _attend(q.double().cpu().numpy(), kv, [had[b] + int(n[b]) for b in range(B)], n, sees, depths, 0, 0)
        _near(out, lse, ref, "bf16")
        check(out, ek, ev, [90, 17, 64], (cout, clse))
        c = np.array([rng.integers(1, min(5, x) + 1) for x in n])
        chosen = np.zeros((B, 5), int)
        for b in range(B):
            chosen[b, :c[b]] = np.sort(rng.choice(n[b], c[b], replace=False))
            kept[b] = np.concatenate([kept[b], drafted[b][:, :, chosen[b, :c[b]]]], 2)
            seen[b] = np.concatenate([seen[b], read[b][:, :, chosen[b, :c[b]]]], 2)
        path.copy_(i32(chosen))
        counts.copy_(i32(c))
        graphs[1].replay()
        torch.cuda.synchronize()
        apa.check_error()
        assert base.tolist() == [k.shape[2] for k in kept]
        for b in range(B):
            pos = np.arange(kept[b].shape[2])
            slots = i32(table[b].cpu().numpy()[pos // 64] * 64 + pos % 64)
            for layer in range(2):
                got = apa.cache_read(pages[layer], slots, ks, vs, dtype=torch.float16)
                assert all(np.array_equal(g.double().cpu().numpy(), w) for g, w in zip(got, seen[b]))
    held = sum((k.shape[2] + 63) // 64 for k in kept)
    assert int(count) == pool - held


@pytest.mark.parametrize("before", ["copy from the host", "fill", "kernel", "joined stream", "its own call"])
def test_cross_sees_what_the_work_before_it_wrote(before):
    """The kernel begins before the work before it has ended: queries and lengths written just before, of every kind of
    work that a stream holds, run at once and captured and replayed, give the bits of a call after a synchronize."""
    import torch

    import mixed_precision_attention_gb300 as apa
    B, N = 16, 500
    q, k, v = _cross_inputs(B, 4, 2, 30, N, 128, seed=8)
    rng = np.random.default_rng(8)
    lens, host, big = _i32([0] * B), torch.zeros(B, dtype=torch.int32).pin_memory(), torch.ones(1 << 27, device="cuda")
    src, other = _i32([0] * B), torch.cuda.Stream()
    x = torch.empty_like(q)

    def run():
        x.fill_(0)
        lens.fill_(0)
        big.mul_(1.0)  # what is before it takes some time
        if before == "copy from the host":
            x.copy_(q)
            lens.copy_(host, non_blocking=True)
        elif before == "fill":
            lens.fill_(321)
            x.copy_(q)
            x[:, 1].zero_()
        elif before == "kernel":
            torch.mul(q, 1, out=x)
            torch.add(src, 0, out=lens)
        elif before == "joined stream":
            now = torch.cuda.current_stream()
            other.wait_stream(now)
            with torch.cuda.stream(other):
                big.mul_(1.0)
                lens.copy_(src)
                x.copy_(q)
            big[:1000].mul_(1.0)
            now.wait_stream(other)
        else:
            lens.copy_(src)
            x.copy_(apa.attention_cross(q, k, v, lens)[0])
            return apa.attention_cross(apa.attention_cross(x, k, v, lens)[0], k, v, lens)
        return apa.attention_cross(x, k, v, lens)

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        captured = run()
    for _ in range(3):
        n = rng.integers(0, N + 1, B).astype(np.int32)
        q.copy_(_torch(rng.standard_normal(q.shape), torch.bfloat16))
        host.copy_(torch.from_numpy(n))
        src.copy_(host)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        with torch.cuda.stream(side):
            eager = run()
        torch.cuda.synchronize()
        a = q.clone()
        at = _i32([321] * B) if before == "fill" else _i32(n)
        if before == "fill":
            a[:, 1] = 0
        want = apa.attention_cross(a, k, v, at)
        if before == "its own call":
            for _ in range(2):
                torch.cuda.synchronize()
                want = apa.attention_cross(want[0], k, v, at)
        torch.cuda.synchronize()
        assert _same(got, want) and _same(eager, want)
    apa.check_error()


def test_an_empty_batch_is_refused():
    import mixed_precision_attention_gb300 as apa
    a, _, _ = _step(np.random.default_rng(9), 2, 4, 2, 40, 64, [100, 40], [40, 4])
    none = {k: a[k][:0] for k in ("q", "block_table", "lens", "nodes", "mask", "depths")}
    for kw in (none, dict(none, mask=a["mask"][:1], depths=a["depths"][:1])):
        with pytest.raises((ValueError, apa.ApaError)):
            apa.attention_tree(**dict(a, **kw))
    q, k, v = _cross_inputs(2, 4, 2, 5, 20, 64)
    with pytest.raises((ValueError, apa.ApaError)):
        apa.attention_cross(q[:0], k[:0], v[:0])
