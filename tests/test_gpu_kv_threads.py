"""Two host threads on one stream: the attention of each has to be its own, bit
by bit, also where its items are split and a second launch joins them."""
import threading

import pytest
import torch

import gemm_w4a16_group_gb300 as w4

from tree_helpers import Step

pytestmark = pytest.mark.gpu


def run(s):
    return w4.tree_attention(s.q, s.k, s.v, s.table, s.lengths, s.starts, s.mask, s.max_tree, k_scale=s.ks, v_scale=s.vs)


@pytest.mark.parametrize("sizes", [(1, 1), (16, 16), (1, 40)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_two_threads_on_one_stream(sizes, e4m3):
    steps = [Step([3000 + 1000 * i, 700], [n, n], 8, 2, 128, 64, e4m3=e4m3, seed=i) for i, n in enumerate(sizes)]
    want = [run(s) for s in steps]
    torch.cuda.synchronize()
    got, errors = [[], []], []
    together = threading.Barrier(2)

    def work(i):
        try:
            together.wait()
            for _ in range(200):
                got[i].append(run(steps[i]))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and w4.kernel_status() == 0
    for i in range(2):
        assert len(got[i]) == 200 and all(torch.equal(o, want[i]) for o in got[i])
