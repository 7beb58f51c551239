"""Cache calls with nothing to do, on the GPU: nothing changes, and nothing is
reported."""
import pytest
import torch

import gemm_w4a16_group_gb300 as w4

from tree_helpers import BF16, Step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stream", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
def test_a_step_without_new_tokens(stream, e4m3):
    s = Step([20, 3], [2, 1], 4, 2, 64, 16, e4m3=e4m3)
    side = torch.cuda.Stream() if stream else None
    k, v, table, lengths = s.k.clone(), s.v.clone(), s.table.clone(), s.lengths.clone()
    torch.cuda.synchronize()
    none, starts = s.q[:0, :2], torch.zeros(3, dtype=torch.int32, device="cuda")
    ids = torch.zeros(0, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    w4.kv_append(none, none, s.k, s.v, s.table, s.lengths, starts, k_scale=s.ks, v_scale=s.vs, stream=side)
    out = w4.tree_attention(s.q[:0], s.k, s.v, s.table, s.lengths, starts, None, 4, k_scale=s.ks, v_scale=s.vs, stream=side)
    path, count, token = w4.tree_accept(ids, ids, ids, starts, 4, stream=side)
    after = w4.kv_compact(s.k, s.v, s.table, s.lengths, path, count, stream=side)
    no = torch.zeros(0, dtype=torch.int32, device="cuda")
    refs = torch.ones(s.pool, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    w4.kv_free(s.table, s.lengths, refs, no, stream=side)
    forked = w4.kv_fork(s.k, s.v, s.table, s.lengths, refs, no, no, stream=side)
    grown = w4.kv_reserve(s.table, refs, no, no, 16, stream=side)
    torch.cuda.synchronize()
    assert w4.kernel_status() == 0
    assert out.shape == (0, 4, 64) and out.dtype == BF16
    assert path.tolist() == [[-1] * 4] * 2 and count.tolist() == [0, 0] and token.tolist() == [-1, -1]
    assert after.tolist() == [20, 3] and forked.tolist() == [1] and grown.tolist() == [1] and (refs == 1).all()
    assert torch.equal(s.table, table) and torch.equal(s.lengths, lengths)
    assert torch.equal(s.k.view(torch.uint8), k.view(torch.uint8)) and torch.equal(s.v.view(torch.uint8), v.view(torch.uint8))
