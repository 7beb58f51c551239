"""Attention of drafted token trees over a paged cache against a float64
implementation: types, head groupings, page sizes, layouts, lengths of zero
and one, pages and tiles that end inside a context, masks that leave nothing,
and what stands in places that no token sees."""
import math

import numpy as np
import pytest
import torch

import gemm_w4a16_group_gb300 as w4

from tree_helpers import BF16, E4M3, Step, attention_bound

pytestmark = pytest.mark.gpu


def run(s, mask=True, **kw):
    out = w4.tree_attention(s.q, s.k, s.v, s.table, s.lengths, s.starts, s.mask if mask else None, s.max_tree,
                            k_scale=s.ks, v_scale=s.vs, **kw)
    torch.cuda.synchronize()
    assert w4.kernel_status() == 0
    return out


def check(s, out, chain=False, scale=None):
    ref, mag = s.attention(scale=scale, chain=chain)
    err = (out.double() - ref).abs()
    bad = ~(err <= attention_bound(ref, mag))
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, first {bad.nonzero()[:3].tolist()}"


SHAPES = [  # lengths, sizes
    ([1], [1]),
    ([0], [1]),
    ([0, 5, 0], [3, 0, 0]),
    ([17], [16]),
    ([63, 64, 65, 1], [1, 2, 7, 33]),
    ([300, 0, 1000], [64, 64, 5]),
    ([2049], [12]),
]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lengths,sizes", SHAPES)
def test_lengths_and_types(dim, e4m3, lengths, sizes):
    s = Step(lengths, sizes, 6, 2, dim, 16, e4m3=e4m3, seed=len(lengths) + dim)
    check(s, run(s))


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (4, 4), (5, 1), (40, 8), (24, 4), (64, 1), (7, 7), (36, 3)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_head_groupings(heads, kv_heads, e4m3):
    s = Step([130, 77], [9, 4], heads, kv_heads, 128, 32, e4m3=e4m3, seed=heads)
    check(s, run(s))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "kv"])
@pytest.mark.parametrize("e4m3", [False, True])
def test_pages_and_layouts(page, layout, e4m3):
    """NHD pages, and keys and values side by side in one allocation."""
    s = Step([page * 3 - 1, page, 3 * page + 5, 400], [3, 1, 8, 20], 8, 2, 64, page, e4m3=e4m3, layout=layout, seed=page)
    check(s, run(s))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("size", [1, 3, 7, 16, 40, 64])
@pytest.mark.parametrize("e4m3", [False, True])
def test_every_key_counts_once(dim, size, e4m3):
    """q = 0 weighs every seen key alike, and value rows are unit vectors: the output counts keys, and one key
    missed or taken twice shows at any of these lengths."""
    lengths = [0, 1, 31, 127, 128, 1000, 4095, 5000]
    s = Step(lengths, [size] * len(lengths), 4, 2, dim, 64, e4m3=e4m3, seed=size)
    s.q.zero_()
    s.v.zero_()
    for b, n in enumerate(lengths):
        ids, rows = s.slots(b, n + size)
        one = torch.nn.functional.one_hot(torch.arange(n + size, device="cuda") % dim, dim).to(BF16)
        if e4m3:
            s.v.view(torch.uint8)[ids, :, rows] = one[:, None].to(E4M3).view(torch.uint8).expand(-1, 2, -1)
        else:
            s.v[ids, :, rows] = one[:, None].expand(-1, 2, -1)
    out = run(s).double()
    if e4m3:
        out = out / s.vs.double().repeat_interleave(2)[None, :, None]
    for b, n in enumerate(lengths):
        sees = s.sees(b)
        for i in range(size):
            count = torch.bincount(sees[i].nonzero()[:, 0] % dim, minlength=dim).double()
            want = (count / count.sum()).expand(4, dim)
            # one rounding to bf16, and two float32 ones where 8-bit scales come in
            assert (out[int(s.starts_h[b]) + i] - want).abs().le(want * (2.0 ** -8 + 2.0 ** -20)).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("size", [1, 16, 64])
def test_one_key_outweighs_all(size, e4m3):
    """A key that a head's query matches gets all the weight: at the ends of pages, tiles and contexts."""
    n, dim = 3000, 128
    for at in [0, 15, 16, 63, 64, 127, 128, 255, 256, 1023, 1500, 2047, 2048, 2999, 3000]:
        s = Step([n], [size], 5, 1, dim, 32, e4m3=e4m3, seed=at)
        ids, rows = s.slots(0, n + size)
        s.q[:] = 4.0
        s.k.view(torch.uint8)[:] = 0  # every other score is 0
        hot = torch.full((dim,), 448.0 if e4m3 else 4.0, device="cuda").to(s.k.dtype)
        s.k.view(torch.uint8)[ids[at], 0, rows[at]] = hot.view(torch.uint8)
        if e4m3:
            s.ks[:] = 1 / 112
        out = run(s)
        want = s.v[ids[at], 0, rows[at]].float() * (1 if s.vs is None else s.vs)
        # the other weights are e^(-16 * 128 / sqrt(128)) = e^-181: nothing
        seen = s.sees(0)[:, at]
        assert torch.equal(out[seen], want.to(BF16).expand(int(seen.sum()), 5, dim))


@pytest.mark.parametrize("size", [3, 14, 64])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_what_nobody_sees_does_not_matter(size, e4m3, dim):
    """NaN and infinities past the context's end, in unused pages and table entries, and in drafted tokens that a
    token does not see."""
    lengths = [0, 70, 129]
    rng = np.random.default_rng(size)
    words = np.concatenate([np.array([1 << i for i in range(size)], np.uint64)] * 3)  # each sees itself alone
    dark = [int(rng.integers(0, size)) for _ in lengths]
    for b in range(3):  # a node that nobody sees
        words[b * size + dark[b]] = 0
    s = Step(lengths, [size] * 3, 6, 2, dim, 16, e4m3=e4m3, seed=3, masks=words, width_more=2)
    want, mag = s.attention()
    if e4m3:
        bad_k = torch.tensor([0x7F, 0xFF] * (dim // 2), dtype=torch.uint8, device="cuda")
        kb, vb = s.k.view(torch.uint8), s.v.view(torch.uint8)
    else:
        bad_k = torch.tensor([math.nan, math.inf, -math.inf, math.nan] * (dim // 4), dtype=BF16, device="cuda")
        kb, vb = s.k, s.v
    used = torch.zeros((s.pool, 16), dtype=torch.bool, device="cuda")
    for b, n in enumerate(lengths):
        ids, rows = s.slots(b, n + size)
        used[ids, rows] = True
        used[ids[n + dark[b]], rows[n + dark[b]]] = False
    for c in (kb, vb):
        c.copy_(torch.where(used[:, None, :, None], c, bad_k))
    out = run(s)
    assert torch.isfinite(out.float()).all()
    err = (out.double() - want).abs()
    assert (err <= attention_bound(want, mag)).all()


def test_a_node_with_nan_spoils_only_those_who_see_it():
    size = 20
    s = Step([200], [size], 8, 2, 128, 32, seed=5)
    want, mag = s.attention()
    ids, rows = s.slots(0, 200 + size)
    node = 3
    s.v[ids[200 + node], :, rows[200 + node]] = math.nan
    out = run(s)
    seen = s.sees(0)[:, 200 + node]
    assert seen.any() and not seen.all()
    assert torch.isnan(out[seen].float()).all()
    assert ((out[~seen].double() - want[~seen]).abs() <= attention_bound(want, mag)[~seen]).all()
    # infinite values: infinite where seen, unseen elsewhere
    s.v[ids[200 + node], :, rows[200 + node]] = math.inf
    out = run(s)
    assert torch.isposinf(out[seen].float()).all()
    assert ((out[~seen].double() - want[~seen]).abs() <= attention_bound(want, mag)[~seen]).all()


def test_rows_that_see_nothing_are_zero():
    words = np.array([0, 1, 0, 0], np.uint64)
    s = Step([0, 0], [3, 1], 4, 2, 64, 16, seed=1, masks=words)
    out = run(s, out=torch.full((4, 4, 64), 7.0, dtype=BF16, device="cuda"))
    for t in (0, 2, 3):
        assert (out[t] == 0).all()
    ids, rows = s.slots(0, 1)
    assert torch.equal(out[1], s.v[ids[0], :, rows[0]].repeat_interleave(2, 0))


@pytest.mark.parametrize("size", [1, 5, 33, 64])
def test_chain_without_mask(size):
    s = Step([100, 0], [size, size], 6, 3, 128, 64, seed=size)
    check(s, run(s, mask=False), chain=True)


def test_mask_bits_past_the_row_are_ignored():
    s = Step([50], [5], 4, 1, 64, 32, seed=9)
    a = run(s)
    s.mask |= ~31  # bits 5 .. 63
    assert torch.equal(a, run(s))


@pytest.mark.parametrize("size", [2, 20, 64])
def test_large_scores(size):
    """Scores up to thousands: the maximum is subtracted before any exponential."""
    s = Step([700], [size], 8, 2, 128, 64, seed=size)
    s.q.mul_(64)
    check(s, run(s))
    check(s, run(s, scale=3.0), scale=3.0)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("size", [1, 6, 30, 64])
@pytest.mark.parametrize("every", [16, 64, 128])
def test_a_maximum_that_keeps_growing(dim, size, every):
    """Scores that rise by 9 powers of two every so many keys, values that fall as fast: each stretch counts as much as
    the last, and what was summed before has to be scaled down in time, once, and whole. (13 stretches: the first weight
    is 2^-108, within float32's normal numbers.)"""
    n = 13 * every - size
    s = Step([n], [size], 8, 2, dim, 32, seed=every)
    ids, rows = s.slots(0, n + size)
    step = torch.arange(n + size, device="cuda") // every
    s.q.zero_()
    s.q[:, :, 0] = 4.0
    s.k.zero_()
    s.k[ids, :, rows, 0] = (step * (9 * math.log(2) / 4))[:, None].to(BF16)
    s.v[ids, :, rows] = (s.v[ids, :, rows].float() * 2.0 ** (72 - 9 * step)[:, None, None]).to(BF16)
    check(s, run(s, scale=1.0), scale=1.0)


@pytest.mark.parametrize("size", [4, 30])
def test_views_and_side_streams(size):
    """q a slice of a fused query/key/value product; the call on another stream, into given buffers."""
    s = Step([333, 12], [size, size], 10, 2, 128, 16, seed=2)
    check(s, run(s))
    want = run(s)
    fused = torch.zeros((s.tokens, 14, 128), dtype=BF16, device="cuda")
    fused[:, 2:12] = s.q
    s.q = fused[:, 2:12]
    out = torch.zeros_like(want)
    ws = torch.empty(w4.tree_attention_workspace_bytes(10, 2, 128, size), dtype=torch.uint8, device="cuda").fill_(255)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    w4.tree_attention(s.q, s.k, s.v, s.table, s.lengths, s.starts, s.mask, s.max_tree, out=out, workspace=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("size", [1, 13, 64])
@pytest.mark.parametrize("e4m3", [False, True])
def test_same_bits_every_time_and_in_a_graph(size, e4m3):
    s = Step([5000, 100, 0, 4000], [size] * 4, 8, 2, 128, 64, seed=4, e4m3=e4m3)
    out = torch.empty_like(s.q)
    ws = torch.empty(w4.tree_attention_workspace_bytes(8, 2, 128, s.max_tree), dtype=torch.uint8, device="cuda")
    want = run(s, out=out, workspace=ws).clone()
    for _ in range(5):
        assert torch.equal(run(s, out=out, workspace=ws), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4.tree_attention(s.q, s.k, s.v, s.table, s.lengths, s.starts, s.mask, s.max_tree, k_scale=s.ks, v_scale=s.vs,
                          out=out, workspace=ws)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    # the graph follows the lengths on the device
    s.lengths[0] = 17
    s.lengths_h = np.array([17, 100, 0, 4000])
    g.replay()
    torch.cuda.synchronize()
    check(s, out)


@pytest.mark.parametrize("dim,size,heads", [(64, 1, 1), (128, 3, 4), (128, 20, 1), (128, 64, 3), (256, 30, 1)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_one_item_over_every_share(dim, size, heads, e4m3):
    """One kv head and a long context: more partial results than are joined at a time."""
    s = Step([40000], [size], heads, 1, dim, 64, e4m3=e4m3, seed=dim + size)
    check(s, run(s))


def test_outputs_are_handed_out_once():
    s = Step([40, 7], [1, 1], 8, 2, 64, 16)
    outs, q = [], s.q.clone()
    for i in range(70):  # small outputs are made some dozens at a time
        s.q.copy_(q * (i + 1))
        outs.append(run(s))
    assert len({o.data_ptr() for o in outs}) == 70
    for i in (0, 31, 32, 69):
        s.q.copy_(q * (i + 1))
        assert torch.equal(outs[i], run(s, out=torch.empty_like(outs[i])))


def test_padding_tokens_are_left_alone():
    s = Step([20, 30], [2, 3], 4, 2, 64, 16, seed=6)
    want = run(s)
    s.q = torch.cat([s.q, s.q[:3]])
    s.mask = torch.cat([s.mask, s.mask[:3]])
    out = torch.full((8, 4, 64), 5.0, dtype=BF16, device="cuda")
    run(s, out=out)
    assert torch.equal(out[:5], want) and (out[5:] == 5).all()


@pytest.mark.parametrize("size", [3, 64])
def test_offsets_past_32_bits(size):
    """Pages 2^27 elements apart: the last ones start past 2^32 bytes and 2^31 elements."""
    pages = 24
    s = Step([16 * (pages - 6)], [size], 4, 1, 64, 16, seed=8, spare=0)
    far = lambda c: torch.empty((s.pool << 27,), dtype=BF16, device="cuda").as_strided(c.shape, (1 << 27, 16 * 64, 64, 1))  # noqa: E731
    k, v = far(s.k), far(s.v)
    k.copy_(s.k)
    v.copy_(s.v)
    s.k, s.v = k, v
    check(s, run(s))


@pytest.mark.parametrize("size", [4, 50])
def test_bad_indices_are_skipped_and_reported(size):
    s = Step([100, 100, 40], [size] * 3, 4, 2, 64, 16, seed=7)
    want = run(s)
    table = s.table.clone()
    table[0, 2] = s.pool + 5  # keys 32 .. 47 of row 0 are not there
    table[1, 1] = -1
    out = w4.tree_attention(s.q, s.k, s.v, table, s.lengths, s.starts, s.mask, s.max_tree)
    torch.cuda.synchronize()
    assert w4.kernel_status() == -6 and w4.kernel_status() == 0
    assert torch.isfinite(out.float()).all()
    assert torch.equal(out[2 * size:], want[2 * size:])
    # row 1 without its keys 16 .. 31 is a shorter row
    keep = [*range(0, 16), *range(32, 100 + size)]
    ids, rows = s.slots(1, 100 + size)
    sees = s.sees(1)
    for i in (0, size - 1):
        w = torch.zeros(100 + size, dtype=torch.bool, device="cuda")
        w[keep] = True
        w &= sees[i]
        for h in range(4):
            k, v = s.k[ids, h // 2, rows][w].double(), s.v[ids, h // 2, rows][w].double()
            p = torch.softmax(k @ s.q[size + i, h].double() / 8, 0)
            assert ((out[size + i, h].double() - p @ v).abs() <= attention_bound(p @ v, p @ v.abs())).all()
    # a row with more new tokens than max_tree says, starts that descend, a negative length
    for starts, lengths in (([0, size, 3 * size, 3 * size], None), ([0, size, size - 1, 3 * size], None), (None, [100, -1, 40])):
        st = s.starts if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
        ln = s.lengths if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
        out = w4.tree_attention(s.q, s.k, s.v, s.table, ln, st, s.mask, s.max_tree)
        torch.cuda.synchronize()
        assert w4.kernel_status() == -6
        # row 0 as before; where starts descend, row 2 lays claim to its last token too
        n = size if starts is None or starts[2] >= size else size - 1
        assert torch.equal(out[:n], want[:n])
