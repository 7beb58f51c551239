"""The 8-bit codes that kv_append writes, code by code: x / scale in float32,
rounded to nearest and saturated, whatever stands beside a value."""
import numpy as np
import pytest
import torch

import gemm_w4a16_group_gb300 as w4

from tree_helpers import BF16, E4M3, Step

pytestmark = pytest.mark.gpu


def codes(x, scale):
    """Codes (uint8) of the bf16 values x [n, 64], as kv_append stores them."""
    n = x.shape[0]
    s = Step([0], [n], 1, 1, 64, 64, e4m3=True, masks=np.zeros(n, np.uint64))
    s.ks[:], s.vs[:] = scale, scale
    w4.kv_append(x[:, None], x[:, None], s.k, s.v, s.table, s.lengths, s.starts, k_scale=s.ks, v_scale=s.vs)
    torch.cuda.synchronize()
    assert w4.kernel_status() == 0
    ids, rows = s.slots(0, n)
    k, v = (c.view(torch.uint8)[ids, 0, rows] for c in (s.k, s.v))
    assert torch.equal(k, v)
    return k


def want(x, scale):
    return (x.float() / torch.tensor(scale, dtype=torch.float32, device="cuda")).clamp(-448, 448).to(E4M3).view(torch.uint8)


@pytest.mark.parametrize("scale", [1.0, 0.0173, 3.0e-7, 1e-25, 1e25])
@pytest.mark.parametrize("order", ["ascending", "mixed"])
def test_every_bf16_value(scale, order):
    """All 65,536 of them: both zeros keep their signs."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    if order == "mixed":
        x = x[torch.randperm(65536, generator=torch.Generator().manual_seed(1))]
    x = x.view(BF16).view(-1, 64).cuda()
    got, w = codes(x, scale), want(x, scale)
    nan = torch.isnan(x.float())
    assert torch.equal(got[~nan], w[~nan])
    assert ((got[nan] & 0x7F) == 0x7F).all()


@pytest.mark.parametrize("scale", [1.0, 0.0173])
@pytest.mark.parametrize("neighbour", [1.0, -0.0, 1e30])
def test_a_code_does_not_depend_on_its_neighbours(scale, neighbour):
    vals = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 0.3, -0.3, 500.0, -500.0], dtype=BF16, device="cuda")
    for at in range(8):
        x = torch.full((8, 64), neighbour, dtype=BF16, device="cuda")
        x[:, at::8] = vals[:, None]
        assert torch.equal(codes(x, scale), want(x, scale))
