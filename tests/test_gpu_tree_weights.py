"""Attention over a paged cache where the softmax weights lie far apart: many
keys that only count together, maxima that keep growing, weights that round
badly. Against float64."""
import math

import numpy as np
import pytest
import torch

import gemm_w4a16_group_gb300 as w4

from tree_helpers import Step, attention_bound

pytestmark = pytest.mark.gpu


def run(s, **kw):
    out = w4.tree_attention(s.q, s.k, s.v, s.table, s.lengths, s.starts, s.mask, s.max_tree, k_scale=s.ks, v_scale=s.vs, **kw)
    torch.cuda.synchronize()
    assert w4.kernel_status() == 0
    return out.double()


def put(c, ids, rows, x):
    """Values x [positions, ...] at positions of row 0, in the cache's type."""
    x = x.expand(len(ids), *c[0, :, 0].shape).to(c.dtype)
    if c.dtype == torch.bfloat16:
        c[ids, :, rows] = x
    else:
        c.view(torch.uint8)[ids, :, rows] = x.view(torch.uint8)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("size", [1, 16, 64])
@pytest.mark.parametrize("keys", [512, 4000])  # in one piece, and split
@pytest.mark.parametrize("gap", [14, 17, 20, 22.3, 24.3, 25.2, 26])
def test_small_weights_count(e4m3, dim, size, keys, gap):
    """Every 128th key outweighs the others by 2^gap, and its value is 0: the others alone make the output, together."""
    s = Step([keys - size], [size], 4, 1, dim, 16, e4m3=e4m3, seed=size + dim)
    rng = np.random.default_rng(size)
    ids, rows = s.slots(0, keys)
    heavy = (torch.arange(keys, device="cuda") % 128 == 0)[:, None]
    put(s.k, ids, rows, torch.where(heavy, 0.0, 1.0)[:, None].expand(-1, 1, dim))
    v = torch.rand((keys, 1, dim), generator=torch.Generator().manual_seed(7)).cuda() + 0.5
    put(s.v, ids, rows, torch.where(heavy[:, None], 0.0, v))
    s.q.zero_()
    s.q[:, :, 0] = torch.from_numpy(-(gap + rng.random((size, 4)) / 2) * math.log(2)).to(s.q)
    if e4m3:
        s.ks[:], s.vs[:] = 1.0, 1.0
    ref, mag = s.attention(scale=1.0)
    err = (run(s, scale=1.0) - ref).abs() / attention_bound(ref, mag)
    assert err.max() <= 1, f"{float(err.max())} of the bound"


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("size", [1, 6, 30, 64])
@pytest.mark.parametrize("every", [16, 64, 128])
@pytest.mark.parametrize("rise", [1, 2, 3, 4, 8])
def test_a_maximum_that_keeps_growing_in_eight_bits(dim, size, every, rise):
    """Scores that rise by `rise` powers of two every so many keys, values that fall as fast, over the range that 8-bit
    values have."""
    steps = 17 // rise
    n = steps * every
    if n < size:
        pytest.skip("more new tokens than keys")
    s = Step([n - size], [size], 8, 2, dim, 32, e4m3=True, seed=every)
    ids, rows = s.slots(0, n)
    step = torch.arange(n, device="cuda") // every
    s.q.zero_()
    s.q[:, :, 0] = 4.0
    put(s.k, ids, rows, step[:, None, None].float().expand(-1, 1, dim))
    sign = torch.randint(0, 2, (n, 2, dim), generator=torch.Generator().manual_seed(1)).cuda() * 2 - 1
    put(s.v, ids, rows, sign * 2.0 ** (8 - rise * step)[:, None, None])
    s.ks[:] = rise * math.log(2) / 4
    ref, mag = s.attention(scale=1.0)
    err = (run(s, scale=1.0) - ref).abs() / attention_bound(ref, mag)
    assert err.max() <= 1, f"{float(err.max())} of the bound"


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("keys", [400, 3000])
def test_both_parts_of_a_weight(dim, keys):
    """One query row per head of a bf16 cache: weights keep 15 bits, in two parts. All but one are just under half way between two
    bf16 numbers, so that one part alone would be off by nearly 2^-8, all the same way. The output's own rounding is
    2^-8; two parts, float32 scores, exponentials and sums stay below 2^-12."""
    a = (128 + torch.arange(128)).double() / 128  # bf16 in [1, 2)
    weight = torch.exp(-(a[:, None] * a[None, :]) / 4)  # k = -a / 4, q = a
    over = weight * 2.0 ** -torch.floor(torch.log2(weight)) - 1  # mantissa
    best = int((((over * 128) % 1 - 0.48).abs() + over).argmin())  # an ulp is 2^-7; a mantissa near 1 loses most
    qa, ka = float(a[best // 128]), -float(a[best % 128]) / 4
    s = Step([keys - 1], [1], 4, 2, dim, 64, seed=dim)
    ids, rows = s.slots(0, keys)
    heavy = (torch.arange(keys, device="cuda") == 5)[:, None, None]
    put(s.k, ids, rows, torch.where(heavy, 0.0, ka).expand(-1, 1, dim))
    v = torch.rand((1, 2, dim), generator=torch.Generator().manual_seed(3)).cuda() + 0.5
    put(s.v, ids, rows, torch.where(heavy, 0.0, v))
    s.q.zero_()
    s.q[:, :, 0] = qa
    ref, mag = s.attention(scale=1.0)
    err = (run(s, scale=1.0) - ref).abs()
    assert (err <= 2.0 ** -8 * ref.abs() + 2.0 ** -12 * mag).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("size", [1, 4, 20, 64])
@pytest.mark.parametrize("keys", [300, 3000])
def test_values_of_the_context_that_are_not_finite(dim, size, keys):
    """Every token sees them, with a weight above 0: an infinite value makes its element infinite, a NaN or two
    infinities of either sign make it NaN, and the other elements are as they were."""
    s = Step([keys - size], [size], 4, 2, dim, 32, seed=dim + size)
    ref, mag = s.attention()
    ids, rows = s.slots(0, keys)
    s.v[ids[7], :, rows[7], 3] = math.inf
    s.v[ids[150], :, rows[150], 5] = -math.inf
    s.v[ids[150], :, rows[150], 9] = math.inf
    s.v[ids[201], :, rows[201], 9] = -math.inf
    s.v[ids[keys - size - 1], :, rows[keys - size - 1], 11] = -math.inf  # in the tile that ends the context
    s.v[ids[77], :, rows[77], 20] = math.nan
    out = run(s)
    assert torch.isposinf(out[..., 3]).all()
    assert torch.isneginf(out[..., 5]).all() and torch.isneginf(out[..., 11]).all()
    assert torch.isnan(out[..., 9]).all() and torch.isnan(out[..., 20]).all()
    rest = torch.ones(dim, dtype=torch.bool)
    rest[[3, 5, 9, 11, 20]] = False
    assert ((out - ref).abs() <= attention_bound(ref, mag))[..., rest].all()
