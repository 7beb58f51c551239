"""The paged cache around the attention: append, acceptance, compaction, and
the page table's free, fork and reserve, against loops on the host. Everything
here moves values or counts, so results are equal, not near."""
import math

import numpy as np
import pytest
import torch

import gemm_w4a16_group_gb300 as w4

from tree_helpers import BF16, E4M3, Step, Table, greedy, new_cache, page_table, random_tree

pytestmark = pytest.mark.gpu


def ok():
    torch.cuda.synchronize()
    return w4.kernel_status()


def bits(t):
    return t.view(torch.uint8) if t.element_size() == 1 else t.view(torch.int16)


@pytest.mark.parametrize("dim,kv,page", [(64, 1, 16), (128, 8, 64), (256, 3, 32), (128, 2, 256)])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "kv"])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("sizes", [[1], [5, 0, 17, 1], [300, 0, 0, 33]])
def test_append(dim, kv, page, layout, e4m3, sizes):
    lengths = [0, 7, 100, 63][:len(sizes)]
    s = Step(lengths, sizes, kv, kv, dim, page, e4m3=e4m3, layout=layout, masks=np.zeros(sum(sizes), np.uint64))
    n = sum(sizes)
    rows = torch.randn((n + 2, 2 * kv + 1, dim), device="cuda").to(BF16)  # two padding tokens behind
    if e4m3:
        rows[0, 1, :6] = torch.tensor([math.nan, math.inf, -math.inf, 1e30, -1e-30, 0.0])
    k, v = rows[:, 1:kv + 1], rows[:, kv + 1:]
    want_k, want_v = s.k.clone(), s.v.clone()
    for b, size in enumerate(sizes):
        for i in range(size):
            pos = lengths[b] + i
            t, id_ = int(s.starts_h[b]) + i, int(s.table_h[b, pos // page])
            for want, x, scale in ((want_k, k, s.ks), (want_v, v, s.vs)):
                x = x[t]
                if e4m3:
                    x = (x.float() / scale[:, None]).clamp(-448, 448).to(E4M3)
                bits(want)[id_, :, pos % page] = bits(x)
    w4.kv_append(k, v, s.k, s.v, s.table, s.lengths, s.starts, k_scale=s.ks, v_scale=s.vs)
    assert ok() == 0
    for got, want in ((s.k, want_k), (s.v, want_v)):
        got, want = bits(got), bits(want)
        if e4m3:  # a NaN code's sign is free
            got, want = (torch.where(x & 0x7F == 0x7F, 0x7F, x) for x in (got, want))
        assert torch.equal(got, want)


@pytest.mark.parametrize("dim,kv,rows", [(64, 5, 70), (256, 20, 33), (128, 33, 4), (64, 1, 1100), (128, 2, 1025)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_append_many_rows_and_heads(dim, kv, rows, e4m3):
    """More rows than a warp looks at, heads off a block's threads, rows without tokens in between."""
    rng = np.random.default_rng(rows)
    sizes, lengths = rng.choice([0, 0, 1, 2, 40], rows).tolist(), rng.integers(0, 50, rows).tolist()
    n = sum(sizes)
    s = Step(lengths, sizes, kv, kv, dim, 16, e4m3=e4m3, masks=np.zeros(n, np.uint64))
    k, v = (torch.randn((n, kv, dim), device="cuda").to(BF16) for _ in range(2))
    want_k, want_v = s.k.clone(), s.v.clone()
    row = np.repeat(np.arange(rows), sizes)
    pos = np.asarray(lengths)[row] + np.arange(n) - np.asarray(s.starts_h)[row]
    ids, at = (torch.from_numpy(x.astype(np.int64)).cuda() for x in (np.asarray(s.table_h)[row, pos // 16], pos % 16))
    for want, x, scale in ((want_k, k, s.ks), (want_v, v, s.vs)):
        if e4m3:
            x = (x.float() / scale[:, None]).clamp(-448, 448).to(E4M3)
        bits(want)[ids, :, at] = bits(x)
    w4.kv_append(k, v, s.k, s.v, s.table, s.lengths, s.starts, k_scale=s.ks, v_scale=s.vs)
    assert ok() == 0
    for got, want in ((s.k, want_k), (s.v, want_v)):
        got, want = bits(got), bits(want)
        if e4m3:  # a NaN code's sign is free
            got, want = (torch.where(x & 0x7F == 0x7F, 0x7F, x) for x in (got, want))
        assert torch.equal(got, want)


def test_append_every_e4m3_rounding():
    """Each code, the halfway points between codes and their bf16 neighbours, at two scales."""
    codes = torch.arange(256, dtype=torch.uint8).view(E4M3).float()
    fin = codes[torch.isfinite(codes)].sort().values
    mid = (fin[1:] + fin[:-1]) / 2
    x = torch.cat([fin, mid]).to(BF16)
    x = torch.cat([x, (x.view(torch.int16) + 1).view(BF16), (x.view(torch.int16) - 1).view(BF16)])
    x = x[torch.isfinite(x.float())]
    n = -(-x.numel() // 64)
    x = torch.nn.functional.pad(x, (0, n * 64 - x.numel())).view(n, 1, 64).cuda()
    for scale in (1.0, 0.0173):
        s = Step([0], [n], 1, 1, 64, 64, e4m3=True, masks=np.zeros(n, np.uint64))
        s.ks[:], s.vs[:] = scale, scale
        w4.kv_append(x, x, s.k, s.v, s.table, s.lengths, s.starts, k_scale=s.ks, v_scale=s.vs)
        assert ok() == 0
        want = (x.float() / torch.tensor(scale, device="cuda")).clamp(-448, 448).to(E4M3)
        ids, rows = s.slots(0, n)
        assert torch.equal(s.k.float()[ids, :, rows], want.float()) and torch.equal(s.v.float()[ids, :, rows], want.float())


def test_append_skips_what_has_no_place():
    s = Step([10, 20, 30], [4, 4, 4], 2, 2, 64, 16, masks=np.zeros(12, np.uint64))
    k = torch.randn((12, 2, 64), device="cuda").to(BF16)
    table = s.table.clone()
    table[1, 1] = s.pool  # positions 16 .. 31 of row 1
    lengths = torch.tensor([10, 20, 16 * s.table.shape[1] - 2], dtype=torch.int32, device="cuda")
    table[2, :] = s.table[2, 0]  # its last page is a page of its own row
    before = s.k.clone()
    w4.kv_append(k, k, s.k, s.v, table, lengths, s.starts)
    assert ok() == -6
    want = before.clone()
    for i in range(4):
        want[int(s.table_h[0, 0]), :, 10 + i] = k[i]
    for i in range(2):  # the two that the table still holds
        want[int(s.table_h[2, 0]), :, 14 + i] = k[8 + i]
    assert torch.equal(s.k, want)


def accept_case(rng, sizes, vocab):
    words = np.concatenate([random_tree(rng, n) for n in sizes] + [np.zeros(0, np.uint64)])
    draft, target = (rng.integers(0, vocab, len(words)) for _ in range(2))
    return words, draft, target


@pytest.mark.parametrize("sizes", [[1], [0, 3, 0], [64, 33, 32, 31, 2], [16] * 40])
@pytest.mark.parametrize("vocab", [1, 2, 5, 1 << 40])
def test_accept(sizes, vocab):
    """Small vocabularies make equal siblings and long walks; one token accepts a child everywhere."""
    rng = np.random.default_rng(len(sizes) + vocab)
    words, draft, target = accept_case(rng, sizes, vocab)
    starts = np.concatenate([[0], np.cumsum(sizes)])
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    path, count, token = w4.tree_accept(to(target), to(draft), to(words.view(np.int64)), to(starts.astype(np.int32)), max(sizes))
    assert ok() == 0
    for b, n in enumerate(sizes):
        lo = starts[b]
        p = greedy(words[lo:lo + n], draft[lo:lo + n], target[lo:lo + n])
        assert path[b].tolist() == p + [-1] * (max(sizes) - len(p))
        assert int(count[b]) == len(p) and int(token[b]) == (target[lo + p[-1]] if p else -1)


def test_accept_chain_and_forests():
    to = lambda *a: torch.tensor(a, device="cuda")  # noqa: E731
    starts = to(0, 5).int()
    draft, target = to(9, 1, 2, 3, 4), to(1, 2, 3, 7, 8)
    path, count, token = w4.tree_accept(target, draft, None, starts, 5)
    assert ok() == 0 and path[0].tolist() == [0, 1, 2, 3, -1] and int(count) == 4 and int(token) == 7
    # node 1 is a second root: not a child of node 0, so never reached; node 2 hangs under it
    words = to(1, 2, 6, 9, 25)
    path, count, token = w4.tree_accept(to(3, 2, 0, 4, 8), to(0, 3, 2, 3, 4), words, starts, 5)
    assert ok() == 0 and path[0].tolist() == [0, 3, 4, -1, -1] and int(token) == 8
    # more new tokens than max_tree
    path, count, token = w4.tree_accept(target, draft, None, starts, 4)
    assert ok() == -6 and int(count) == 0 and int(token) == -1 and path[0].tolist() == [-1] * 4


@pytest.mark.parametrize("dim,kv,page,layers", [(64, 1, 16, 1), (128, 8, 16, 3), (256, 2, 64, 2)])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "kv"])
@pytest.mark.parametrize("e4m3", [False, True])
def test_compact(dim, kv, page, layers, layout, e4m3):
    rng = np.random.default_rng(dim)
    lengths, tree = np.array([0, 15, 100, 33, 7, 64]), 64
    paths = [[0], list(range(64)), sorted(rng.permutation(64)[:40].tolist()), [], [0, 1, 2, 5, 6, 60], [63]]
    held = -(-(lengths + tree) // page)
    table = page_table(rng, held, int(held.max()), int(held.sum()))
    gen = torch.Generator().manual_seed(1)
    k, v, _, _ = new_cache((layers, int(held.sum()), kv, page, dim), e4m3, layout, gen, "cuda")
    if layers == 1:
        k, v = k[0], v[0]
    path = np.full((6, tree), -1, np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    want = [bits(x).clone() for x in (k, v)]
    for w in want:
        if layers == 1:
            w = w[None]
        for b, p in enumerate(paths):
            at = [(int(table[b, (lengths[b] + i) // page]), int(lengths[b] + i) % page) for i in range(tree)]
            rows = [w[:, at[i][0], :, at[i][1]].clone() for i in p]
            for i, r in enumerate(rows):
                w[:, at[i][0], :, at[i][1]] = r
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).int().cuda()  # noqa: E731
    count = np.array([len(p) for p in paths])
    out = w4.kv_compact(k, v, to(table), to(lengths), to(path), to(count))
    assert ok() == 0
    assert torch.equal(bits(k), want[0]) and torch.equal(bits(v), want[1])
    assert out.tolist() == (lengths + count).tolist()


def test_compact_refuses_paths_that_do_not_ascend():
    s = Step([20, 20, 20, 20], [8] * 4, 2, 2, 64, 16)
    path = torch.tensor([[0, 2, 1, 5], [1, 1, 2, 3], [0, 9, 0, 0], [0, 2, 3, 3]], dtype=torch.int32, device="cuda")
    count = torch.tensor([3, 2, 2, 3], dtype=torch.int32, device="cuda")
    k, v = s.k.clone(), s.v.clone()
    out = w4.kv_compact(k, v, s.table, s.lengths, path, count)
    assert ok() == -6 and out.tolist() == [20, 20, 20, 23]
    ids, rows = s.slots(3, 28)
    want = s.k.clone()
    want[ids[21], :, rows[21]] = s.k[ids[22], :, rows[22]]
    want[ids[22], :, rows[22]] = s.k[ids[23], :, rows[23]]
    assert torch.equal(k, want)


class Pool:
    """A table of `rows` rows over `pool` pages on the device and, as Table, on the host."""

    def __init__(self, rng, rows, width, pool, page, lengths, layers=2, kv=2, dim=64, e4m3=False, layout="hnd"):
        held = -(-np.asarray(lengths) // page)
        table = page_table(rng, held, width, pool)
        refs = np.zeros(pool, np.int32)
        np.add.at(refs, table[table >= 0], 1)
        self.host = Table(table, np.asarray(lengths, np.int32), refs, page)
        to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).int().cuda()  # noqa: E731
        self.to = to
        self.table, self.lengths, self.refs = to(table), to(lengths), to(refs)
        self.k, self.v, _, _ = new_cache((layers, pool, kv, page, dim), e4m3, layout, torch.Generator().manual_seed(2), "cuda")

    def same(self):
        assert self.table.tolist() == self.host.table.tolist()
        assert self.lengths.tolist() == self.host.lengths.tolist()
        assert self.refs.tolist() == self.host.refs.tolist()

    def fork(self, src, dst):
        want = [bits(x).clone() for x in (self.k, self.v)]
        copies = self.host.fork(src, dst)
        for w in want:
            for a, b, n in copies or []:
                w[:, b, :, :n] = w[:, a, :, :n]
        got = w4.kv_fork(self.k, self.v, self.table, self.lengths, self.refs, self.to(src), self.to(dst))
        assert int(got) == (copies is not None)
        assert torch.equal(bits(self.k), want[0]) and torch.equal(bits(self.v), want[1])


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "kv"])
@pytest.mark.parametrize("e4m3", [False, True])
def test_fork_free_reserve_in_turn(page, layout, e4m3):
    rng = np.random.default_rng(page)
    lengths = [0, 1, page, page + 1, 5 * page - 1, 0, 0, 0, 0, 0, 0, 0]
    p = Pool(rng, 12, 8, 40, page, lengths, e4m3=e4m3, layout=layout)
    p.fork([4, 4, 2, 0, 3], [6, 5, 11, 7, 9])
    p.same()
    for rows, want in (([6, 9], [6 * page, 2 * page + 1]), ([0, 1, 8], [1, page, 0])):
        assert int(w4.kv_reserve(p.table, p.refs, p.to(rows), p.to(want), page)) == p.host.reserve(rows, want) == 1
        p.same()
    w4.kv_free(p.table, p.lengths, p.refs, p.to([4, 6, 8]))
    p.host.free([4, 6, 8])
    p.same()
    p.fork([5, 3], [6, 4])  # of a branch, into pages just freed
    p.same()
    assert ok() == 0


@pytest.mark.parametrize("pool", [1, 40, 1024, 1025, 5000])
def test_many_rows_and_pools(pool):
    """Pools off the scan's width, more rows than a block has threads, and all or nothing at the last page."""
    rng = np.random.default_rng(pool)
    rows = 1500 if pool == 5000 else 8
    p = Pool(rng, rows, 4, pool, 16, [0] * rows, layers=1, kv=1)
    names = rng.permutation(rows)[:rows // 2 + 1]
    want = rng.integers(0, 65, len(names))
    for target in (want, want * 0 + 64):
        assert int(w4.kv_reserve(p.table, p.refs, p.to(names), p.to(target), 16)) == int(p.host.reserve(names, target))
        p.same()
    left = int((p.host.refs == 0).sum())
    empty = [b for b in range(rows) if p.host.table[b, 0] < 0]
    if left and empty:  # one row takes what is left, page by page; the next page is refused
        n = min(left, 4)
        assert int(w4.kv_reserve(p.table, p.refs, p.to(empty[:1]), p.to([16 * n]), 16)) == p.host.reserve(empty[:1], [16 * n]) == 1
    p.same()
    w4.kv_free(p.table, p.lengths, p.refs, p.to(names))
    p.host.free(names)
    p.same()
    assert ok() == 0


def test_fork_without_room_changes_nothing():
    p = Pool(np.random.default_rng(0), 6, 4, 5, 16, [20, 40, 0, 0, 0, 0])
    assert (p.host.refs == 0).sum() == 0
    p.fork([0], [2])
    p.same()
    p.fork([0, 1], [3, 4])
    p.same()
    w4.kv_free(p.table, p.lengths, p.refs, p.to([0]))
    p.host.free([0])
    p.fork([1, 1], [3, 4])  # two pages free, two needed
    p.same()
    p.fork([1, 3], [5, 0])
    p.same()
    assert ok() == 0


def test_bad_rows_are_reported_and_change_nothing():
    p = Pool(np.random.default_rng(1), 6, 4, 12, 16, [20, 40, 0, 0, 0, 0])
    for src, dst in (([0], [6]), ([-1], [2]), ([0], [1]), ([0, 0], [2, 2]), ([0, 2], [2, 3]), ([0], [0])):
        got = w4.kv_fork(p.k, p.v, p.table, p.lengths, p.refs, p.to(src), p.to(dst))
        assert int(got) == 0 and ok() == -6
        p.same()
    for rows, want in (([6], [1]), ([0, 0], [1, 1]), ([0], [65]), ([0], [-1])):
        assert int(w4.kv_reserve(p.table, p.refs, p.to(rows), p.to(want), 16)) == 0 and ok() == -6
        p.same()
    w4.kv_free(p.table, p.lengths, p.refs, p.to([1, 6, -1, 1]))  # row 1 once; the rest reported
    p.host.free([1])
    p.same()
    assert ok() == -6


def test_on_another_stream():
    p = Pool(np.random.default_rng(3), 4, 4, 12, 16, [20, 0, 0, 0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    src, dst, want = p.to([0]), p.to([2]), p.to([40])
    w4.kv_fork(p.k, p.v, p.table, p.lengths, p.refs, src, dst, stream=s)
    w4.kv_reserve(p.table, p.refs, dst, want, 16, stream=s)
    w4.kv_free(p.table, p.lengths, p.refs, src, stream=s)
    assert ok() == 0
    p.host.fork([0], [2])
    p.host.reserve([2], [40])
    p.host.free([0])
    p.same()


def test_outputs_are_new_each_time():
    """Small outputs share allocations, never memory: each keeps its values while others are made, in and out of order."""
    to = lambda *a: torch.tensor(a, device="cuda")  # noqa: E731
    starts, draft = to(0, 3).int(), to(9, 1, 2)
    kept = []
    for i in range(100):
        out = w4.tree_accept(to(1, 2, 100 + i), draft, None, starts, 3 + i % 2)
        if i % 3:
            kept.append((i, out))
    assert ok() == 0
    for i, (path, count, token) in kept:
        assert path[0].tolist() == [0, 1, 2] + [-1] * (i % 2) and int(count) == 3 and int(token) == 100 + i
    at = sorted((t.data_ptr(), t.nbytes) for _, out in kept for t in out)
    assert all(a + n <= b for (a, n), (b, _) in zip(at, at[1:]))
