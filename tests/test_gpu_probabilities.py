"""probabilities against a softmax in 64 bits: temperatures, floors, masked
logits, values that are not numbers, odd widths and strides."""
import math

import numpy as np
import pytest
import torch

import gemm_w4a16_group_gb300 as w4

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def reference(logits, temperature=None, floor=None):
    """float64 probabilities and their bounds. e^((l - m) / T): the exponential is off by 2^-21 (ex2.approx 2^-22, its
    factor), the difference l - m, rounded to float32, by 2^-24 of itself, and so is the argument's second part; the sum of
    up to 64 values of a thread, two at a time, 8 joinings and 16 slices by 2^-18, the division and the product by 2^-23. A
    power below 2^-126, the smallest normal number, becomes 0: relative to a sum of at least 1, so off by at most that."""
    x = logits.double().cpu()
    out, bound = torch.zeros_like(x), torch.zeros_like(x)
    for i in range(x.shape[0]):
        kept = torch.ones(x.shape[1], dtype=torch.bool) if floor is None else ~(x[i] < float(floor[i]))
        kept &= x[i] != -math.inf
        if not kept.any():
            continue
        t = 1.0 if temperature is None else float(temperature[i])
        m = x[i][kept].max()
        if t > 0:
            e = torch.exp((x[i][kept] - m) / t)
            out[i, kept] = e / e.sum()
            bound[i, kept] = out[i, kept] * (2.0 ** -17 + 2.0 ** -23 * (m - x[i][kept]) / t) + 2.0 ** -126
        else:
            out[i, int(torch.nonzero(kept & (x[i] == m))[0])] = 1.0
    return out, bound


def check(logits, temperature=None, floor=None, **kw):
    got = w4.probabilities(logits, temperature, floor, **kw)
    want, bound = reference(logits, temperature, floor)
    off = (got.double().cpu() - want).abs()
    assert (off <= bound).all(), float((off / bound.clamp(min=1e-300)).max())
    return got


def logits_of(seed, tokens, vocab, spread=4.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn((tokens, vocab), generator=gen) * spread).to(BF16).cuda()


@pytest.mark.parametrize("tokens,vocab", [(1, 1), (3, 2), (2, 5), (7, 31), (5, 1000), (4, 4097), (9, 16384), (3, 32001),
                                          (2, 65538), (1, 248320), (5, 248320), (2, 262147), (1, 600003), (300, 513)])
def test_softmax(tokens, vocab):
    x = logits_of(vocab, tokens, vocab)
    got = check(x)
    assert (got.double().sum(-1) - 1).abs().max() < 1e-5
    gen = torch.Generator().manual_seed(tokens)
    t = (torch.rand(tokens, generator=gen) * 2 + 0.1)
    t[::3] = 0.0
    check(x, t.cuda())
    k = min(vocab, 20)
    check(x, t.cuda(), torch.topk(x.float(), k).values[:, -1].contiguous())


def test_temperatures_at_the_ends():
    x = logits_of(0, 10, 777)
    x[:, 5] = x[:, 700] = 40.0  # two equal maxima
    t = torch.tensor([0.0, -1.0, 1e-38, 1e-30, 1e-6, 0.01, 100.0, 1e30, 3e38, math.nan], device="cuda")
    got = check(x, t)
    assert got[0, 5] == 1 and got[0, 700] == 0 and got[9, 5] == 1
    assert got[2, 5] == 0.5 and got[2, 700] == 0.5
    flat = w4.probabilities(x, torch.full((10,), math.inf, device="cuda"))
    assert ((flat - 1 / 777).abs() <= 2.0 ** -17 / 777).all()


def test_the_smallest_temperatures():
    """Logits as close together as their temperature is small, down to 2^-127; below that it counts as 2^-127.

    The exponent (l - m) a, a = log2(e) / T, in float32: log2(e) is off by 2^-26, and the quotient, the difference and the
    product are rounded once each, 3.25 2^-24 in all, which ln 2 log2(e) leaves as it is: less than 2^-22 (max - l) / T."""
    low = 2.0 ** -127
    got = w4.probabilities(torch.tensor([[0.0, -1e-31]], device="cuda").to(BF16), torch.tensor([1e-38], device="cuda"))
    assert got.tolist() == [[1.0, 0.0]]
    for t in (1e-20, 1e-30, 7e-31, 1e-35, 2.0 ** -126, 1e-38, low):
        x = (torch.randn((1, 3001), generator=torch.Generator().manual_seed(1)) * 4 * t).to(BF16).cuda()
        got = w4.probabilities(x, torch.tensor([t], device="cuda")).double()
        x, t = x.double(), float(np.float32(t))
        want = torch.softmax((x - x.max()) / t, -1)
        assert ((got - want).abs() <= want * (2.0 ** -17 + 2.0 ** -22 * (x.max() - x) / t) + 2.0 ** -126).all()
    x = torch.tensor([[0.0, -2.0 ** -133, -2.0 ** -130, -2.0 ** -126, -2.0 ** -120]], device="cuda").to(BF16)
    want = w4.probabilities(x, torch.tensor([low], device="cuda"))
    assert ((want.double() - torch.softmax(x.double() / low, -1)).abs() <= 2.0 ** -17).all()
    for t in (1e-39, 1e-42, 1.5e-45):
        assert torch.equal(w4.probabilities(x, torch.tensor([t], device="cuda")), want)


def test_masked_logits():
    """-inf and the type's lowest value as masks, rows that keep nothing or one token."""
    x = logits_of(1, 6, 900)
    low = torch.finfo(BF16).min
    x[0, ::2] = -math.inf
    x[1, ::2] = low
    x[2] = -math.inf
    x[3] = -math.inf
    x[3, 77] = -3.0
    x[4] = low
    for t in (None, torch.tensor([1.0, 0.7, 1.0, 0.0, 0.3, 0.0], device="cuda"), torch.zeros(6, device="cuda")):
        got = check(x, t)
        assert (got[2] == 0).all() and got[3, 77] == 1 and (got[0, ::2] == 0).all()
    # a floor above everything keeps nothing; a NaN floor drops nothing
    floor = torch.tensor([100.0, math.nan, -1.0, -2.0, -math.inf, 0.0], device="cuda")
    got = check(x, None, floor)
    assert (got[0] == 0).all() and (got[3] == 0).all()
    # -0 and 0 are equal, also to a floor
    z = torch.zeros((1, 9), dtype=BF16, device="cuda")
    z[0, 1::2] = -0.0
    assert torch.allclose(w4.probabilities(z, None, torch.zeros(1, device="cuda")), torch.full((1, 9), 1 / 9, device="cuda"))
    assert w4.probabilities(z.neg(), torch.zeros(1, device="cuda"))[0].tolist() == [1.0] + [0.0] * 8


def test_values_that_are_not_numbers():
    x = logits_of(2, 4, 500)
    x[0, 3], x[1, 7], x[2, 3] = math.nan, math.inf, math.nan
    x[0, 400:] = -math.inf
    got = w4.probabilities(x)
    assert got[0, :400].isnan().all() and (got[0, 400:] == 0).all()
    assert got[1].isnan().all() and got[2].isnan().all()
    want, bound = reference(x[3:])
    assert ((got[3:].double().cpu() - want).abs() <= bound).all()
    greedy = w4.probabilities(x, torch.zeros(4, device="cuda"))  # as the argmax: a NaN is the maximum
    assert greedy[0, 3] == 1 and greedy[1, 7] == 1 and greedy.sum().item() == 4
    assert torch.equal(greedy.argmax(-1), w4.topk(x.contiguous(), 1)[0][:, 0])


@pytest.mark.parametrize("vocab", [1001, 1004])
def test_strides_and_alignment(vocab):
    x = logits_of(3, 5, vocab)
    t = torch.tensor([0.5, 1.0, 0.0, 2.0, 1.0], device="cuda")
    want = check(x, t)
    for lead, width in ((0, vocab + 4), (4, vocab + 8), (1, vocab + 3), (3, vocab + 30)):
        big = torch.full((5, lead + width), 99.0, dtype=BF16, device="cuda")
        big[:, lead:lead + vocab] = x
        got = w4.probabilities(big[:, lead:lead + vocab], t)
        # (another alignment sums in another order)
        assert torch.allclose(got, want, rtol=2.0 ** -17, atol=0)
    for lead in (0, 1, 2):  # out that does not begin on 16 bytes, with its surroundings left alone
        room = torch.full((5 * vocab + 8,), 7.0, device="cuda")
        out = room[lead:lead + 5 * vocab].view(5, vocab)
        assert w4.probabilities(x, t, out=out) is out
        assert torch.allclose(out, want, rtol=2.0 ** -17, atol=0)
        assert (room[:lead] == 7).all() and (room[lead + 5 * vocab:] == 7).all()
    one = x[:1].expand(5, vocab)
    assert torch.allclose(w4.probabilities(one)[4], w4.probabilities(x[:1])[0], rtol=2.0 ** -17, atol=0)


@pytest.mark.parametrize("vocab", [5, 8, 1003, 16389, 33001, 262150])
def test_columns_of_a_wider_head(vocab):
    """Logits that begin anywhere, against every place of out; slices of one chunk and of more, masked and greedy rows."""
    x = logits_of(7, 6, vocab)
    t, floor = torch.tensor([0.5, 1.0, 0.0, 2.0, 1.0, 0.0], device="cuda"), x.float().mean(1)
    want = check(x, t), check(x, t, floor)
    for at in range(8):
        for width in (vocab, vocab + 1, vocab + 3, vocab + 61):
            store = torch.full((at + 6 * width + 3,), 99.0, dtype=BF16, device="cuda")  # (99: a maximum, were it read)
            view = store[at:at + 6 * width].view(6, width)[:, :vocab]
            view.copy_(x)
            room = torch.full((6 * vocab + 8,), 7.0, device="cuda")
            out = room[at // 2:at // 2 + 6 * vocab].view(6, vocab)
            for fl, w in zip((None, floor), want):
                w4.probabilities(view, t, fl, out=out)
                assert torch.allclose(out, w, rtol=2.0 ** -17, atol=0)
                assert (room[:at // 2] == 7).all() and (room[at // 2 + 6 * vocab:] == 7).all()


@pytest.mark.parametrize("vocab", [1, 2, 3, 4])
def test_a_few_columns_of_a_wider_head(vocab):
    """Rows without a whole quad, at every place of logits and out."""
    x = logits_of(vocab, 6, vocab)
    t = torch.tensor([0.5, 1.0, 0.0, 2.0, 1.0, 0.0], device="cuda")
    want, _ = reference(x, t)
    for at in range(8):
        for width in (vocab, vocab + 1, vocab + 2, vocab + 3, vocab + 4):
            store = torch.full((at + 6 * width + 3,), 99.0, dtype=BF16, device="cuda")
            view = store[at:at + 6 * width].view(6, width)[:, :vocab]
            view.copy_(x)
            for lead in range(4):
                room = torch.full((6 * vocab + 8,), 7.0, device="cuda")
                out = room[lead:lead + 6 * vocab].view(6, vocab)
                check(view, t, out=out)
                assert (room[:lead] == 7).all() and (room[lead + 6 * vocab:] == 7).all()
                assert torch.equal(out.double().cpu().argmax(1), want.argmax(1))


def test_streams_graphs_and_repeats():
    x = logits_of(4, 6, 30001)
    want = w4.probabilities(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        got = w4.probabilities(x, stream=side)
        side.synchronize()
        assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = w4.probabilities(x)
    x.copy_(logits_of(5, 6, 30001))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, w4.probabilities(x))


def test_many_rows():
    """More rows than a grid's second axis would hold."""
    x = logits_of(6, 70000, 8)
    got = w4.probabilities(x).double()
    want = torch.softmax(x.double(), -1)
    assert ((got - want).abs() <= want * 2.0 ** -17).all()
