"""Attention over tables of many rows, most of them idle: more rows than a
block has threads, so that a thread looks after several of them when the work
is shared out. Against float64."""
import numpy as np
import pytest
import torch

import gemm_w4a16_group_gb300 as w4

from tree_helpers import Step, attention_bound

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,active", [(160, 160), (161, 161), (161, 3), (385, 40), (513, 513), (700, 350), (4096, 25), (4096, 1)])
@pytest.mark.parametrize("size", [1, 12])  # 4 query rows per kv head, and up to 48
@pytest.mark.parametrize("e4m3", [False, True])
def test_many_rows(rows, active, size, e4m3):
    rng = np.random.default_rng(rows + active)
    lengths, sizes = rng.integers(0, 200, rows), np.zeros(rows, np.int64)
    on = rng.permutation(rows)[:active]
    sizes[on] = rng.integers(1, size + 1, active)
    sizes[on[0]] = size
    lengths[on[0]] = 1500  # a table wide enough for items to be split
    s = Step(lengths, sizes, 4, 1, 64, 16, e4m3=e4m3, seed=rows)
    out = w4.tree_attention(s.q, s.k, s.v, s.table, s.lengths, s.starts, s.mask, s.max_tree, k_scale=s.ks, v_scale=s.vs)
    torch.cuda.synchronize()
    assert w4.kernel_status() == 0
    ref, mag = s.attention()
    assert ((out.double() - ref).abs() <= attention_bound(ref, mag)).all()
