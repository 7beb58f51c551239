"""lora_add against 64 bits: ranks, sizes, rows with shared, missing and bad
adapters, padding, strides, in place, other streams and graphs."""
import math

import numpy as np
import pytest
import torch

import gemm_w4a16_group_gb300 as w4
from sample_helpers import adapted, stored

pytestmark = pytest.mark.gpu


class Problem:
    def __init__(self, sizes, which, rank, inner, outer, store, seed=0, pad=0, scaled=True):
        gen = torch.Generator().manual_seed(seed)
        self.tokens = sum(sizes) + pad
        self.starts_h = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        self.which = [e for n, e in zip(sizes, which) for _ in range(n)] + [-1] * pad
        self.x, self.y = stored(gen, self.tokens, inner).cuda(), stored(gen, self.tokens, outer).cuda()
        self.a = stored(gen, store, rank, inner, std=inner ** -0.5).cuda()
        self.b = stored(gen, store, outer, rank, std=rank ** -0.5).cuda()
        self.scale = (torch.rand(store, generator=gen) + 0.5).cuda() if scaled else None
        self.adapter = torch.tensor(which, dtype=torch.int32, device="cuda")
        self.starts = torch.from_numpy(self.starts_h).cuda()
        self.live = sum(sizes)

    def run(self, **kw):
        return w4.lora_add(self.y, self.x, self.a, self.b, self.adapter, self.starts, self.scale, **kw)

    def check(self, out):
        want, bound = adapted(self.y, self.x, self.a, self.b, self.which, self.scale)
        off = (out.double().cpu() - want).abs()[:self.live]
        assert (off <= bound[:self.live]).all(), float((off / bound[:self.live].clamp(min=1e-300)).max())
        for t in range(self.live):
            if self.which[t] < 0:
                assert torch.equal(out[t].view(torch.int16), self.y[t].view(torch.int16))


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 72, 128])
@pytest.mark.parametrize("sizes,which,inner,outer", [
    ([1], [0], 64, 64), ([1, 2, 5], [1, -1, 1], 520, 250), ([16, 1, 0, 17], [2, 0, 1, 2], 1288, 1000),
    ([40, 33], [0, 1], 200, 333), ([1] * 20, [i % 3 for i in range(20)], 8, 1),
])
def test_few_tokens(rank, sizes, which, inner, outer):
    p = Problem(sizes, which, rank, inner, outer, 3, seed=rank)
    p.check(p.run())
    assert w4.kernel_status() == 0


@pytest.mark.parametrize("rank", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("sizes,which,inner,outer", [
    ([600], [0], 328, 515), ([300, 7, 513, 1], [1, -1, 0, 1], 1024, 264), ([65, 64, 63, 400], [0, 1, 0, 1], 96, 776),
    ([1200], [0], 328, 515), ([300, 7, 913, 1], [1, -1, 0, 1], 1024, 264), ([65, 64, 63, 1000], [0, 1, 0, 1], 96, 776),
    ([600, 80], [1, 0], 64, 8200), ([512], [1], 72, 40), ([513], [1], 72, 40), ([1023, 1], [1, 0], 72, 40), ([1024, 1], [1, 0], 72, 40),
    ([9, 1050], [0, 1], 8, 1), ([1100], [0], 16, 130), ([2100], [0], 328, 515), ([300, 7, 1913, 1], [1, -1, 0, 1], 1024, 264),
    ([65, 64, 63, 2000], [0, 1, 0, 1], 96, 776), ([9, 2050], [0, 1], 8, 1), ([2047, 1], [0, 1], 72, 40), ([2048, 1], [0, 1], 72, 40), ([3] * 700, [i % 2 for i in range(700)], 264, 140),
    ([128], [0], 64, 70000), ([129, 1], [0, 1], 64, 70000), ([100, 300], [1, 0], 8, 45001), ([3] * 350, [i % 2 for i in range(350)], 264, 140),
])
def test_prompts(rank, sizes, which, inner, outer):
    p = Problem(sizes, which, rank, inner, outer, 2, seed=rank + 1)
    p.check(p.run())
    assert w4.kernel_status() == 0


@pytest.mark.parametrize("tokens,rank", [(n, r) for n in (1, 17, 128) for r in (8, 16, 24, 64, 128)] + [(n, r) for n in (1100, 2500) for r in (8, 16, 24, 32)])
def test_all_bits_are_kept_between_the_products(tokens, rank):
    """x A^T next to the middle of two bf16 values: 1 + m 2^-7 + 2^-8 and 2^-k more or less, which is exact in float32, as are
    all sums here (B has one 1 a column). So the output is that value, rounded once."""
    rng = np.random.default_rng(rank)
    base, by = rng.integers(0, 128, rank), 2.0 ** -rng.integers(12, 22, rank) * rng.choice([-1, 1], rank)
    a = np.zeros((1, rank, 64))
    a[0, :, 3], a[0, :, 40], a[0, :, 9] = 1 + base / 128, 2.0 ** -8, by
    want = torch.from_numpy(a.sum(2)).to(torch.bfloat16)
    up = np.where(by > 0, base + 1, base)
    assert np.array_equal(want.double().numpy()[0], 1 + up / 128)
    a = torch.from_numpy(a).to(torch.bfloat16).cuda()
    x, y = torch.ones((tokens, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((tokens, rank), dtype=torch.bfloat16, device="cuda")
    b = torch.eye(rank, dtype=torch.bfloat16, device="cuda")[None].contiguous()
    out = w4.lora_add(y, x, a, b, torch.zeros(tokens, dtype=torch.int32, device="cuda"))
    assert torch.equal(out.cpu(), want.expand(tokens, rank))


@pytest.mark.parametrize("sizes,which,rank,inner,outer,store", [
    ([1], [3], 16, 5120, 5120, 8), ([1] * 48, [i % 12 for i in range(48)], 64, 5120, 2049, 12), ([8, 3, 1, 5], [0, 1, -1, 0], 32, 17408, 640, 2),
])
def test_model_sizes(sizes, which, rank, inner, outer, store):
    p = Problem(sizes, which, rank, inner, outer, store)
    p.check(p.run())


def test_a_token_a_row():
    p = Problem([1] * 37, [(i * 7) % 5 - 1 for i in range(37)], 16, 256, 300, 4, scaled=False)
    p.starts = None
    p.check(p.run())


def test_a_token_does_not_depend_on_the_others():
    p = Problem([3, 2, 9], [0, 1, 0], 16, 512, 512, 2)
    whole = p.run()
    for b in range(3):
        s = slice(int(p.starts_h[b]), int(p.starts_h[b + 1]))
        one = w4.lora_add(p.y[s], p.x[s], p.a, p.b, p.adapter[b:b + 1], torch.tensor([0, s.stop - s.start], dtype=torch.int32, device="cuda"), p.scale)
        off = (one.double() - whole[s].double()).abs()  # (K is split otherwise: a rounding of bf16 apart at most)
        assert (off <= 2.0 ** -7 * whole[s].double().abs() + 1e-5).all()
    assert torch.equal(p.run(), whole)


def test_in_place_and_padding():
    for sizes, which in (([3, 2, 4], [1, -1, 0]), ([200, 100, 300], [0, -1, 1]), ([400, 300, 600], [0, -1, 1]), ([900, 600, 800], [0, -1, 1])):
        p = Problem(sizes, which, 24, 320, 402, 2, pad=5)
        p.x[p.live:] = math.nan
        keep = p.y.clone()
        want = p.run(out=torch.full_like(p.y, 3.0))
        p.check(want)
        assert (want[p.live:] == 3).all()  # padding is left alone
        got = w4.lora_add(p.y, p.x, p.a, p.b, p.adapter, p.starts, p.scale, out=p.y)
        assert got is p.y and torch.equal(got[:p.live], want[:p.live]) and torch.equal(got[p.live:], keep[p.live:])


def test_columns_of_a_wider_product():
    """Query columns of a fused product, in place, at any alignment; the columns beside stay."""
    for lead, outer, width in ((0, 256, 512), (256, 128, 512), (8, 250, 264), (3, 101, 259), (0, 7, 7)):
        p = Problem([4, 1, 6], [0, 1, -1], 16, 128, outer, 2, seed=lead)
        wide = torch.randn((p.tokens, width + lead), device="cuda").to(torch.bfloat16)
        before = wide.clone()
        view = wide[:, lead:lead + outer]
        p.y = view.clone()
        w4.lora_add(view, p.x, p.a, p.b, p.adapter, p.starts, p.scale, out=view)
        p.check(view.contiguous())
        beside = torch.ones(wide.shape[1], dtype=torch.bool)
        beside[lead:lead + outer] = False
        assert torch.equal(wide[:, beside], before[:, beside])


@pytest.mark.parametrize("tokens", [21, 1100, 2100])
@pytest.mark.parametrize("outer", [31, 64, 300, 513])
def test_rows_that_begin_anywhere(tokens, outer):
    """y and out at every place after 16 bytes, alike and not, rows of one place and of many; what is beside them stays."""
    p = Problem([tokens - 12, 12], [0, 1], 16, 64, outer, 2, seed=outer)
    want = p.run()
    p.check(want)
    y = p.y
    for lead in range(9):
        for extra, out_lead, out_extra in ((0, lead, 0), (8, 0, 0), (3, 5, 16), (5, 7, 2)):
            p.y = torch.full((tokens * (outer + extra) + 16,), 9.0, dtype=torch.bfloat16, device="cuda")[
                lead:lead + tokens * (outer + extra)].view(tokens, outer + extra)[:, :outer]
            p.y.copy_(y)
            room = torch.full((tokens * (outer + out_extra) + 32,), 7.0, dtype=torch.bfloat16, device="cuda")
            out = room[out_lead:out_lead + tokens * (outer + out_extra)].view(tokens, outer + out_extra)
            assert torch.equal(p.run(out=out[:, :outer]), want)
            assert (out[:, outer:] == 7).all() and (room[:out_lead] == 7).all() and (room[out_lead + out.numel():] == 7).all()
            assert torch.equal(p.run(out=p.y), want)


@pytest.mark.parametrize("rank", [24, 40, 56, 72, 120])
@pytest.mark.parametrize("sizes,which,inner,outer", [
    ([300, 7, 1913, 1], [1, -1, 0, 1], 1024, 264), ([2100], [0], 328, 515), ([129, 1], [0, 1], 64, 70000), ([600, 80], [1, 0], 64, 8201),
])
def test_prompts_of_padded_ranks(rank, sizes, which, inner, outer):
    p = Problem(sizes, which, rank, inner, outer, 2, seed=rank)
    p.check(p.run())
    assert w4.kernel_status() == 0


@pytest.mark.parametrize("rank", [16, 40, 128])
@pytest.mark.parametrize("lead,outer,width", [(0, 256, 512), (256, 128, 512), (3, 101, 259), (7, 513, 640)])
def test_columns_of_a_wider_product_of_prompts(rank, lead, outer, width):
    """As test_columns_of_a_wider_product, for the kernels of prompts; rows without an adapter and padding stay too."""
    p = Problem([900, 600, 800], [0, -1, 1], rank, 128, outer, 2, seed=lead, pad=3)
    wide = torch.randn((p.tokens, width + lead), device="cuda").to(torch.bfloat16)
    before = wide.clone()
    view = wide[:, lead:lead + outer]
    p.y = view.clone()
    w4.lora_add(view, p.x, p.a, p.b, p.adapter, p.starts, p.scale, out=view)
    p.check(view.contiguous())
    beside = torch.ones(wide.shape[1], dtype=torch.bool)
    beside[lead:lead + outer] = False
    assert torch.equal(wide[:, beside], before[:, beside]) and torch.equal(wide[p.live:], before[p.live:])


def test_strided_inputs():
    p = Problem([4, 9], [1, 0], 32, 256, 200, 2)
    want = p.run()
    x = torch.empty((p.tokens, 300 + 4), dtype=torch.bfloat16, device="cuda")[:, 8:264]
    x.copy_(p.x)
    a = torch.empty((2, 32, 512), dtype=torch.bfloat16, device="cuda")[:, :, 128:384]
    a.copy_(p.a)
    b = torch.empty((200, 2, 48), dtype=torch.bfloat16, device="cuda").transpose(0, 1)[:, :, 16:]
    b.copy_(p.b)
    assert torch.equal(w4.lora_add(p.y, x, a, b, p.adapter, p.starts, p.scale), want)
    one = p.y[:1].expand(p.tokens, 200)
    p.y = one.contiguous()
    assert torch.equal(w4.lora_add(one, x, a, b, p.adapter, p.starts, p.scale), p.run())


def test_large_store_and_many_rows():
    """More adapters and rows than a block has threads; most of them idle."""
    rng = np.random.default_rng(0)
    store, rows = 1000, 700
    which = np.where(rng.random(rows) < 0.2, -1, rng.integers(0, store, rows)).tolist()
    sizes = rng.integers(0, 3, rows).tolist()
    p = Problem(sizes, which, 8, 64, 96, store)
    p.check(p.run())
    for rank in (8, 64, 128):
        p = Problem([1] * 300, [5] * 150 + [4095] * 150, rank, 16, 24, 4096)
        p.check(p.run())
        p = Problem([500, 0, 180], [4095, 3, 4000], rank, 16, 24, 4096)
        p.check(p.run())
        p = Problem([1500, 0, 180], [4095, 3, 4000], rank, 16, 24, 4096)
        p.check(p.run())
        p = Problem([2500, 0, 180], [4095, 3, 4000], rank, 16, 24, 4096)
        p.check(p.run())


def test_bad_indices_are_left_out_and_reported():
    p = Problem([2, 3, 4], [0, 2, -7], 16, 128, 128, 2)
    out = p.run()
    assert w4.kernel_status() == -6
    p.which = [0, 0] + [-1] * 7
    p.check(out)
    for starts in ([0, 5, 2, 9], [-1, 2, 5, 9], [0, 2, 5, 10]):
        q = Problem([2, 3, 4], [0, 1, -1], 16, 128, 128, 2)
        q.starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
        keep = torch.full_like(q.y, 5.0)
        q.run(out=keep)
        assert w4.kernel_status() == -6
        # (offsets that descend may give a token to two rows: it is either's)
        sound = [(s, t, e) for s, t, e in zip(starts, starts[1:], [0, 1, -1]) if 0 <= s <= t <= 9]
        for i in range(9):
            mine = [e for s, t, e in sound if s <= i < t]
            if not mine:
                assert (keep[i] == 5).all()
            elif len(mine) == 1:
                want, bound = adapted(q.y[i:i + 1], q.x[i:i + 1], q.a, q.b, mine, q.scale)
                assert ((keep[i].double().cpu() - want[0]).abs() <= bound[0]).all()


def test_descending_offsets_that_claim_tokens_many_times():
    """More tiles than a call of so many tokens has room for, and more tokens than 32 bits count."""
    for tokens, rows, top in ((1400, 200, 700), (2400, 300, 700), (2400, 65535, 2400), (70000, 65535, 70000)):
        gen = torch.Generator(device="cuda").manual_seed(rows)
        bf16 = lambda *shape: torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
        x, y, a, b = bf16(tokens, 16), bf16(tokens, 24), bf16(3, 8, 16), bf16(3, 24, 8)
        starts = torch.zeros(rows + 1, dtype=torch.int32, device="cuda")
        starts[1::2] = top  # 0, top, 0, top ..: every other row claims all of them
        adapter = torch.full((rows,), 1, dtype=torch.int32, device="cuda")
        for out in (torch.full_like(y, 5.0), y):
            before = y.clone()
            w4.lora_add(y, x, a, b, adapter, starts, out=out)
            assert w4.kernel_status() == -6
            want, bound = adapted(before, x, a, b, [1] * tokens, None)
            kept = out == (before if out is y else 5.0)
            assert (kept.cpu() | ((out.double().cpu() - want).abs() <= bound)).all() or out is y
            assert kept[top:].all()
            y.copy_(before)


def swapped(rows, each):
    """Offsets of `rows` rows, some of which have changed places with the next."""
    starts = np.arange(rows + 1) * each
    for i in (3, 255, 256, 300, rows - 2):
        starts[[i, i + 1]] = starts[[i + 1, i]]
    return starts.tolist()


@pytest.mark.parametrize("tokens,starts", [
    (9, [0, 5, 2, 9]), (9, [4, 9, 0, 6]), (40, [0, 10, 30, 20, 40, 35, 40]), (600, [0, 400, 100, 500, 300, 600]),
    (900, swapped(450, 2)), (2100, swapped(700, 3)), (4000, [0, 2000, 500, 4000]), (4000, [0, 1500, 4001, 1500, 4000]),
    (70000, [0, 30000, 70000, 70001] + [70000] * 65000),
])
@pytest.mark.parametrize("rank", [8, 32])
def test_offsets_in_no_order_cost_only_their_own_rows(tokens, starts, rank):
    """Every token goes with the first sound row that reaches it from behind all earlier ends, and no other is written."""
    gen = torch.Generator().manual_seed(tokens)
    x, y, a, b = stored(gen, tokens, 16), stored(gen, tokens, 24), stored(gen, 3, rank, 16, std=0.25), stored(gen, 3, 24, rank, std=0.3)
    adapter = torch.arange(len(starts) - 1) % 3 if len(starts) < 1000 else torch.arange(len(starts) - 1) % 2 + 1
    owner, end = [-2] * tokens, 0
    for s, t, e in zip(starts, starts[1:], adapter.tolist()):
        if 0 <= s < t <= tokens:
            for i in range(max(s, end), t):
                owner[i] = e
            end = max(end, t)
    written = torch.tensor([e >= 0 for e in owner])
    want, bound = adapted(y, x, a, b, owner, None)
    x, y, a, b = (v.cuda() for v in (x, y, a, b))
    args = x, a, b, adapter.int().cuda(), torch.tensor(starts, dtype=torch.int32, device="cuda")
    out = w4.lora_add(y, *args, out=torch.full_like(y, 5.0))
    assert w4.kernel_status() == -6
    assert ((out.double().cpu() - want).abs() <= bound)[written].all() and (out.cpu()[~written] == 5).all()
    before = y.clone()
    w4.lora_add(y, *args, out=y)
    assert w4.kernel_status() == -6
    assert torch.equal(y.cpu()[written], out.cpu()[written]) and torch.equal(y.cpu()[~written], before.cpu()[~written])


def test_values_that_are_not_finite_stay_with_their_tokens():
    p = Problem([3, 3, 3], [0, 1, -1], 16, 256, 128, 2)
    p.x[1, 5], p.x[7, 5] = math.inf, math.nan  # the second belongs to a row without an adapter
    p.y[4, 3], p.y[8, 9] = math.inf, math.nan
    p.a[1, 2, 3] = math.nan
    out = p.run()
    assert out[0].isfinite().all() and out[2].isfinite().all()
    assert not out[1].isfinite().any()
    assert out[3:6].isnan().all()
    assert torch.equal(out[6:].view(torch.int16), p.y[6:].view(torch.int16))


@pytest.mark.parametrize("tokens", [3, 1100, 2100])
@pytest.mark.parametrize("rank", [8, 24, 40, 72])
def test_an_infinite_input_times_positive_weights_is_infinite(tokens, rank):
    """Ranks are padded inside with zeros, and infinity times those would not be a number."""
    p = Problem([tokens], [1], rank, 72, 40, 2)
    p.a, p.b = p.a.abs() + 0.1, p.b.abs() + 0.1
    p.x[2, 7] = math.inf
    out = p.run()
    assert (out[2] == math.inf).all() and out[:2].isfinite().all() and out[3:].isfinite().all()


@pytest.mark.parametrize("tokens", [3, 150, 1100, 2500])
@pytest.mark.parametrize("rank", [8, 16, 40, 64, 128])
def test_an_infinite_weight_is_infinite(tokens, rank):
    """A value of x A^T goes on in parts, none of which may be 0 or of the other sign: infinity times that would not be a
    number. Values with 8 bits and with more, a large one, and an infinite one."""
    p = Problem([tokens], [1], rank, 72, 40, 2, scaled=False)
    p.x[:, 16:] = 0
    p.x[1, 5] = math.inf                 # x A^T is infinite
    p.x[2, :16] = 2.0 ** 60
    p.a[1, 3] = 0
    p.a[1, 3, 5], p.a[1, 3, 6] = 1.0, 0.01
    p.x[0, :16] = 0
    p.x[0, 5] = 1.5                      # 1.5, with nothing below
    low = p.x.double() @ p.a[1].double().T
    assert (low[:, 3] != 0).all()
    for column, value in ((7, math.inf), (9, -math.inf)):
        p.b[1, column] = 0
        p.b[1, column, 3] = value
    out = p.run()
    for column, sign in ((7, 1.0), (9, -1.0)):
        got = out[:, column].double()
        want = torch.sign(low[:, 3]) * sign * math.inf
        keep = torch.ones(tokens, dtype=torch.bool, device="cuda")
        keep[1] = False                  # (its other values are infinite too, times a weight of 0: not a number)
        assert torch.equal(got[keep], want[keep])
    beside = [c for c in range(40) if c not in (7, 9)]
    assert out[:, beside][keep].isfinite().all()


@pytest.mark.parametrize("tokens", [3, 1100, 2500])
@pytest.mark.parametrize("rank", [8, 24, 40, 72])
def test_an_infinite_scale_is_infinite(tokens, rank):
    """As an infinite input: the zeros that ranks are padded with are not multiplied by it."""
    p = Problem([tokens], [1], rank, 72, 40, 2)
    p.a, p.b, p.x = p.a.abs() + 0.1, p.b.abs() + 0.1, p.x.abs() + 0.1
    p.scale[1] = math.inf
    assert (p.run() == math.inf).all()
    p.scale[1] = -math.inf
    assert (p.run() == -math.inf).all()


@pytest.mark.parametrize("tokens", [3, 1100, 2500])
def test_values_next_to_the_largest(tokens):
    """x A^T between the largest bf16 value and the largest float32 value stays finite."""
    y = torch.zeros((tokens, 16), dtype=torch.bfloat16, device="cuda")
    x, a, b = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((tokens, 16), (1, 8, 16), (1, 16, 8)))
    x[:, :2] = 2.0 ** 100
    big = torch.finfo(torch.bfloat16).max
    a[0, 0, 0], a[0, 0, 1] = big / 2.0 ** 100, 2.0 ** 19  # big + 2^119: next to the middle between big and 2^128
    a[0, 0, 1] *= 1.5
    b[0, :, 0] = 2.0 ** -100
    out = w4.lora_add(y, x, a, b, torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([0, tokens], dtype=torch.int32, device="cuda"))
    want = torch.tensor((big + 1.5 * 2.0 ** 119) * 2.0 ** -100, dtype=torch.float64).to(torch.bfloat16)
    assert (out.cpu() == want).all()


def test_streams_graphs_and_repeats():
    for sizes, which in (([3, 1, 4], [0, 1, 0]), ([300, 300], [0, 1]), ([700, 400], [0, 1]), ([1700, 400], [0, 1])):
        p = Problem(sizes, which, 32, 512, 1000, 2)
        want = p.run()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(10):
            got = p.run(stream=side)
            mine = p.run()
            side.synchronize()
            assert torch.equal(got, want) and torch.equal(mine, want)
        one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(one):
            a = p.run()
        with torch.cuda.graph(two):
            b = p.run()
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(10):  # two graphs at once: each has a workspace of its own
            one.replay()
            with torch.cuda.stream(side):
                two.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(b, want)
        p.adapter.fill_(-1)
        one.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, p.y)


def test_behind_a_product():
    """gemm and lora_add in a row, as a decode step calls them: the second reads what the first has just written."""
    import synth
    M, N, K, G = 5, 384, 512, 128
    prob = synth.make_problem(M, N, K, G, True, seed=0)
    up = lambda v: torch.from_numpy(np.ascontiguousarray(v).view(np.int16) if v.dtype == np.uint16 else np.ascontiguousarray(v)).cuda()  # noqa: E731
    packed = w4.repack(up(prob["qweight"]), up(prob["scales"]).view(torch.bfloat16), None, N, K, G, True)
    x = up(prob["x"]).view(torch.bfloat16)
    p = Problem([2, 3], [1, 0], 16, K, N, 2)
    p.x = x
    p.y = w4.gemm(x, packed, N, K, G, True)
    torch.cuda.synchronize()
    want = p.run()
    p.check(want)
    for _ in range(50):
        y = w4.gemm(x, packed, N, K, G, True)
        assert torch.equal(w4.lora_add(y, x, p.a, p.b, p.adapter, p.starts, p.scale, out=y), want)
