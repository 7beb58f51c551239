"""tree_sample against exact fractions: chains and trees, drawn and picked
children, borders of the drawn token, rows that leave nothing, odd widths."""
import numpy as np
import pytest
import torch

import gemm_w4a16_group_gb300 as w4
from sample_helpers import sampled, tree

pytestmark = pytest.mark.gpu


def dist(rng, n, vocab, sharp=2.0, zeros=0.0):
    x = np.exp(sharp * rng.standard_normal((n, vocab)))
    x[rng.random((n, vocab)) < zeros] = 0.0
    x[:, 0] += 1e-3
    return (x / x.sum(-1, keepdims=True)).astype(np.float32)


def call(p, q, draft, words, sizes, u, max_tree=None, mask=True):
    starts = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    got = w4.tree_sample(up(p), None if q is None else up(q), up(draft.astype(np.int64)),
                         up(words.view(np.int64)) if mask else None, up(starts), up(u.astype(np.float32)),
                         max_tree or max(1, int(max(sizes))))
    return [t.cpu().numpy() for t in got]


def check(p, q, draft, words, sizes, u, exact=True, **kw):
    path, count, token = call(p, q, draft, words, sizes, u, **kw)
    at = 0
    for b, n in enumerate(sizes):
        s = slice(at, at + n)
        want, tok = sampled(p[s], None if q is None else q[s], draft[s], words[s], u[s], exact)
        assert path[b, :len(want)].tolist() == want and (path[b, len(want):] == -1).all(), (b, path[b], want)
        assert count[b] == len(want)
        assert token[b] == tok, (b, token[b], tok)
        at += n
    assert w4.kernel_status() == 0


def problem(seed, sizes, vocab, width, drawn, sharp=1.0, noise=0.6):
    rng = np.random.default_rng(seed)
    words = np.concatenate([tree(rng, n, width) for n in sizes])
    n = len(words)
    logits = sharp * rng.standard_normal((n, vocab))
    soft = lambda x: (np.exp(x) / np.exp(x).sum(-1, keepdims=True)).astype(np.float32)  # noqa: E731
    p, q = soft(logits), soft(logits + noise * rng.standard_normal((n, vocab)))
    draft = np.zeros(n, np.int64)
    at = 0
    for size in sizes:
        for i in range(1, size):
            above = int(words[at + i]) & ((1 << i) - 1)
            row = q[at + above.bit_length() - 1].astype(np.float64)
            draft[at + i] = rng.choice(vocab, p=row / row.sum()) if drawn else np.argsort(-row)[rng.integers(0, min(vocab, 3))]
        at += size
    u = rng.random(n).astype(np.float32)
    return p, q if drawn else None, draft, words, sizes, u


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("vocab,width,sizes", [
    (1, 1, [1, 2]), (2, 2, [3, 1, 4]), (3, 64, [64, 5, 0, 17]), (7, 3, [9] * 8), (64, 1, [1] * 5), (257, 4, [16, 1, 0, 12]),
    (1000, 2, [8, 8, 3]), (1003, 5, [20, 6]), (4099, 3, [6, 2]),
])
def test_walks(drawn, vocab, width, sizes):
    for seed in range(3):
        check(*problem(seed, sizes, vocab, width, drawn))


@pytest.mark.parametrize("drawn", [True, False])
def test_many_children_refused(drawn):
    """A root with 63 children of which most are refused."""
    rng = np.random.default_rng(5)
    vocab, n = 300, 64
    words = np.array([1] + [1 | 1 << i for i in range(1, n)], np.uint64)
    p, q = dist(rng, n, vocab, 2.0), dist(rng, n, vocab, 2.0)
    draft = rng.integers(0, 40, n)  # many twins
    for shift in (0.0, 0.3, 0.7, 0.999):
        u = np.full(n, 0.98, np.float32)
        u[0] = shift
        check(p, q if drawn else None, draft, words, [n], u)


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("vocab", [32000, 32001, 128003, 248320, 262147, 600001])
def test_large_vocabularies(vocab, drawn):
    """Against float64 sums: no draw may differ."""
    sizes = [1, 6, 4, 8]
    p, q, draft, words, sizes, u = problem(vocab, sizes, vocab, 2, drawn, sharp=2.5)
    for k in range(4):
        check(p, q, draft, words, sizes, np.roll(u, k), exact=False)


def test_tokens_at_the_borders():
    """Probabilities that are multiples of 2^-6, numbers that fall on their running sums."""
    vocab = 64
    p = np.full((1, vocab), 2.0 ** -6, np.float32)
    p[0, 5], p[0, 6], p[0, 63], p[0, 62] = 0.0, 2.0 ** -5, 0.0, 2.0 ** -5
    edge = np.concatenate([np.arange(64) / 64.0, np.arange(64) / 64.0 + 2.0 ** -24, [0.0, 1 - 2.0 ** -24]]).astype(np.float32)
    n = len(edge)
    check(np.repeat(p, n, 0), None, np.zeros(n, np.int64), np.ones(n, np.uint64), [1] * n, edge)


def test_acceptance_at_its_border():
    """u q(x) = p(x) refuses, the next smaller u accepts."""
    vocab, n = 8, 2
    p = np.full((2 * n, vocab), 0.125, np.float32)
    q = p.copy()
    p[:, 0], p[:, 1] = 0.0625, 0.1875
    q[:, 0], q[:, 1] = 0.125, 0.125
    words = np.array([1, 3] * n, np.uint64)
    u = np.array([0.3, 0.5, 0.3, np.nextafter(np.float32(0.5), np.float32(0))], np.float32)
    draft = np.zeros(2 * n, np.int64)
    path, count, _ = call(p, q, draft, words, [2, 2], u)
    assert count.tolist() == [1, 2]
    check(p, q, draft, words, [2, 2], u)


def test_rows_that_leave_nothing():
    vocab = 40
    rng = np.random.default_rng(0)
    p = dist(rng, 6, vocab)
    q = p.copy()
    p[1] = 0.0                       # no probability at all: no token
    p[2] = 0.0
    p[2, 7] = 1.0
    q[2] = 0.0
    q[2, 7] = 1.0                    # the same one-hot
    words = np.array([1, 1, 1, 3, 1, 3], np.uint64)
    draft = np.array([0, 0, 0, 9, 0, 3])
    sizes = [1, 1, 2, 2]
    u = np.array([0.5, 0.5, 0.2, 0.5, 0.4, 0.999], np.float32)
    for drawn in (q, None):
        check(p, drawn, draft, words, sizes, u)
    # p = q: everything is accepted
    path, count, _ = call(p[4:], p[4:], draft[4:], words[4:], [2], u[4:])
    assert count.tolist() == [2]
    # a picked child that has all of p, refused by a number of 1 (which is not below 1): nothing is left, so p itself
    one = np.zeros((2, vocab), np.float32)
    one[:, 11] = 1.0
    path, count, token = call(one, None, np.array([0, 11]), np.array([1, 3], np.uint64), [2], np.array([0.9, 1.0]))
    assert count.tolist() == [1] and token.tolist() == [11]


def test_values_that_are_none():
    """NaN, negative and infinite probabilities count as 0, 0 and 1; numbers outside [0, 1) as its ends."""
    rng = np.random.default_rng(3)
    vocab = 50
    p, q = dist(rng, 6, vocab), dist(rng, 6, vocab)
    p[:, 3], p[:, 4], q[:, 5], q[:, 6] = np.nan, -1.0, np.nan, -np.inf
    p[2, 9] = np.inf
    words = np.array([1, 3, 5] * 2, np.uint64)
    draft = np.array([0, 8, 5, 0, 3, 9])
    for u0 in (-1.0, 0.0, 2.0):
        u = np.array([u0, 0.9, 0.9, u0, 0.5, 0.8], np.float32)
        for d in (q, None):
            check(p, d, draft, words, [3, 3], u)
    u[0] = u[3] = np.nan
    assert all(0 <= t < vocab for t in call(p, q, draft, words, [3, 3], u)[2])


def test_chain_and_masks_that_leave_out():
    p, q, draft, words, sizes, u = problem(11, [6, 1, 4], 100, 1, True)
    chain = np.concatenate([np.array([(1 << i + 1) - 1 for i in range(n)], np.uint64) for n in sizes])
    a = call(p, q, draft, chain, sizes, u, mask=False)
    b = call(p, q, draft, chain, sizes, u)
    assert all((x == y).all() for x, y in zip(a, b))
    check(p, q, draft, chain, sizes, u)
    # nodes without an ancestor are never reached; a word's own and later bits say nothing
    words = chain.copy()
    words[2] = 0
    words[4] |= np.uint64(0xFFFFFFFFFFFFFFE0)
    check(p, q, draft, words, sizes, u)


def test_strided_rows_and_alignment():
    p, q, draft, words, sizes, u = problem(4, [5, 3], 1001, 2, True)
    want = call(p, q, draft, words, sizes, u)
    starts = torch.tensor([0, 5, 8], dtype=torch.int32, device="cuda")
    rest = [torch.from_numpy(a).cuda() for a in (draft, words.view(np.int64))]
    uu = torch.from_numpy(u).cuda()
    for lead, width in ((0, 1004), (4, 1008), (1, 1003), (3, 1201)):
        for q_lead, q_width in ((lead, width), (0, 1001)):
            big = torch.full((8, lead + width), 9.0, device="cuda")
            big[:, lead:lead + 1001] = torch.from_numpy(p).cuda()
            other = torch.full((8, q_lead + q_width), 9.0, device="cuda")
            other[:, q_lead:q_lead + 1001] = torch.from_numpy(q).cuda()
            got = w4.tree_sample(big[:, lead:lead + 1001], other[:, q_lead:q_lead + 1001], rest[0], rest[1], starts, uu, 5)
            assert all((g.cpu().numpy() == w).all() for g, w in zip(got, want))
    for at, q_at in ((1, 1), (2, 2), (3, 3), (1, 3), (5, 2)):  # packed rows that begin off 16 bytes
        room = [torch.full((8 * 1001 + 8,), 9.0, device="cuda") for _ in range(2)]
        pp, qq = (r[k:k + 8 * 1001].view(8, 1001) for r, k in zip(room, (at, q_at)))
        pp.copy_(torch.from_numpy(p))
        qq.copy_(torch.from_numpy(q))
        got = w4.tree_sample(pp, qq, rest[0], rest[1], starts, uu, 5)
        assert all((g.cpu().numpy() == w).all() for g, w in zip(got, want))


def test_bad_indices_are_skipped_and_reported():
    p, q, draft, words, sizes, u = problem(2, [4, 4, 4], 60, 3, True)
    bad = draft.copy()
    bad[2], bad[6] = 60, -5
    got = call(p, q, bad, words, sizes, u)
    assert w4.kernel_status() == -6
    at = 0
    for b, n in enumerate(sizes):
        s = slice(at, at + n)
        want, tok = sampled(p[s], q[s], bad[s], words[s], u[s])
        assert got[0][b, :len(want)].tolist() == want and got[2][b] == tok
        at += n
    # offsets that cannot be: the row has no tokens
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    for starts in ([0, 8, 4, 12], [-3, 4, 8, 12], [0, 4, 8, 13]):
        path, count, token = w4.tree_sample(up(p), up(q), up(draft), up(words.view(np.int64)),
                                            torch.tensor(starts, dtype=torch.int32, device="cuda"), up(u), 4)
        assert w4.kernel_status() == -6
        assert (count == 0).any() and token[count == 0].eq(-1).all() and path[count == 0].eq(-1).all()
    # a row with more tokens than max_tree
    path, count, token = w4.tree_sample(up(p), up(q), up(draft), None, torch.tensor([0, 4, 12], dtype=torch.int32, device="cuda"), up(u), 4)
    assert w4.kernel_status() == -6 and count.tolist()[1] == 0 and count.tolist()[0] > 0


def test_padding_is_not_read():
    p, q, draft, words, sizes, u = problem(8, [3, 2, 4], 90, 2, True)
    want = call(p, q, draft, words, sizes, u)
    pad = lambda a, v: np.concatenate([a, np.full((3, *a.shape[1:]), v, a.dtype)])  # noqa: E731
    got = call(pad(p, np.nan), pad(q, np.nan), pad(draft, -1), pad(words, 0), sizes, pad(u, np.nan), max_tree=4)
    assert w4.kernel_status() == 0
    assert all((a == b).all() for a, b in zip(got, want))


@pytest.mark.parametrize("drawn", [True, False])
def test_accepted_and_drawn_tokens_are_distributed_as_the_target(drawn):
    """40,000 rows of one tree: the first token after the root (accepted, or drawn at the root) has the distribution
    p(root). A share of n draws is off by more than 5.5 sqrt(p (1 - p) / n) once in 26 million."""
    rng = np.random.default_rng(9)
    n, vocab = 40000, 6
    p1 = np.array([0.30, 0.05, 0.25, 0.02, 0.28, 0.10], np.float32)
    q1 = np.array([0.10, 0.30, 0.05, 0.25, 0.10, 0.20], np.float32)
    words = np.tile(np.array([1, 3, 5, 9], np.uint64), n)  # a root with three children
    draft = np.zeros((n, 4), np.int64)
    draft[:, 1:] = rng.choice(vocab, (n, 3), p=q1.astype(np.float64) / q1.astype(np.float64).sum()) if drawn else [4, 1, 2]
    p, q = np.tile(p1, (4 * n, 1)), np.tile(q1, (4 * n, 1))
    u = rng.random(4 * n).astype(np.float32)
    path, count, token = call(p, q if drawn else None, draft.reshape(-1), words, [4] * n, u)
    first = np.where(count > 1, draft[np.arange(n), np.maximum(path[:, 1], 0)], token)
    assert (count > 1).mean() > 0.4 and (count == 1).mean() > 0.05
    for j in range(vocab):
        share = float((first == j).mean())
        assert abs(share - p1[j]) <= 5.5 * (p1[j] * (1 - p1[j]) / n) ** 0.5, (j, share, p1[j])


@pytest.mark.parametrize("vocab", [64, 65, 300, 4097, 32000, 248320])
@pytest.mark.parametrize("drawn", [True, False])
def test_rows_that_sum_to_64_have_no_token_and_are_reported(vocab, drawn):
    """Rows of ones: their sums would wrap at 256. The rows beside them, and nodes before them, stay as they are."""
    rng = np.random.default_rng(vocab)
    for size, words in ((1, [1]), (3, [1, 3, 7]), (3, [1, 3, 5])):
        p, q = dist(rng, 3 * size, vocab), dist(rng, 3 * size, vocab)
        draft, u = rng.integers(0, vocab, 3 * size), np.full(3 * size, 0.4, np.float32)
        words = np.array(words * 3, np.uint64)
        q[:, draft] = 1e-6  # children are accepted where p has anything there
        last = size + (2 if list(words[:3]) == [1, 3, 7] else 1 if size > 1 else 0)
        p[last] = 1.0  # the node at which the middle row's walk ends
        path, count, token = call(p, q if drawn else None, draft, words, [size] * 3, np.where(np.arange(3 * size) % size, 0.0, u))
        assert w4.kernel_status() == -6
        for b in range(3):
            s = slice(b * size, (b + 1) * size)
            want, tok = sampled(p[s], q[s] if drawn else None, draft[s], words[s], np.where(np.arange(size), 0.0, u[s]).astype(np.float32), False)
            assert path[b, :count[b]].tolist() == want
            assert token[b] == (-1 if b == 1 else tok)


def test_sums_up_to_64_are_kept():
    """Rows that are no distributions, below that: by the rules all the same."""
    vocab = 127
    rng = np.random.default_rng(7)
    p, q = np.full((9, vocab), 0.5, np.float32), dist(rng, 9, vocab)
    words = np.array([1, 3, 5, 9] + [1] * 5, np.uint64)
    draft = rng.integers(0, vocab, 9)
    sizes = [4, 1, 1, 1, 1, 1]
    u = np.array([0.9, 0.0, 1.0, 1.0, 0.0, 0.25, 0.5, 0.75, 0.99], np.float32)
    for drawn in (q, None):
        for first in (0.0, 0.6, 1.0):
            u[1] = first
            check(p, drawn, draft, words, sizes, u)


def test_many_refusals_of_rows_that_sum_to_almost_2():
    """c grows by the row's sum with each child that q and p leave nothing: to 125, or past 128 where rows sum to more."""
    vocab, n = 70, 64
    p = np.full((n, vocab), 1.99 / 64, np.float32)
    p[:, 64:] = 0.0
    q = np.zeros((n, vocab), np.float32)
    words = np.array([1] + [1 | 1 << i for i in range(1, n)], np.uint64)
    draft = np.full(n, 66)
    u = np.full(n, 0.5, np.float32)
    check(p, q, draft, words, [n], u)
    path, count, token = call(p * 30, q, draft, words, [n], u)  # 59.7 a row
    assert w4.kernel_status() == -6 and count.tolist() == [1] and token.tolist() == [-1]
    for few in (2, 3):  # one or two refusals of such rows are counted
        check(p[:few] * 30, q[:few], draft[:few], words[:few], [few], u[:few])


def test_streams_graphs_and_repeats():
    p, q, draft, words, sizes, u = problem(6, [6, 2, 7], 2003, 3, True)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    args = (up(p), up(q), up(draft), up(words.view(np.int64)), torch.tensor([0, 6, 8, 15], dtype=torch.int32, device="cuda"), up(u), 7)
    want = [t.clone() for t in w4.tree_sample(*args)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        got = w4.tree_sample(*args, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = w4.tree_sample(*args)
    args[5].copy_(up(np.roll(u, 1)))
    graph.replay()
    torch.cuda.synchronize()
    again = w4.tree_sample(*args)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert w4.kernel_status() == 0
