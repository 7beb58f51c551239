"""probabilities, tree_sample and lora_add at the ends of their ranges: offsets
past 32 bits, many rows, host threads on one stream, outputs of their own."""
import math
import threading

import numpy as np
import pytest
import torch

import gemm_w4a16_group_gb300 as w4
from sample_helpers import adapted

pytestmark = pytest.mark.gpu


def soft(shape, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.softmax(torch.randn(shape, generator=gen, device="cuda"), -1)


def test_walk_over_rows_far_apart():
    """p and q rows 2^28 floats apart: the ninth begins past 2^31."""
    tokens, vocab, far = 12, 5000, 1 << 28
    store = torch.empty(tokens * far, device="cuda")
    p, q = store.as_strided((tokens, vocab), (far, 1), 3), store.as_strided((tokens, vocab), (far, 1), 1 << 20)
    p.copy_(soft((tokens, vocab), 0))
    q.copy_(soft((tokens, vocab), 1))
    draft = torch.randint(0, vocab, (tokens,), device="cuda")
    mask = torch.tensor([1 | 1 << i for i in range(6)] * 2, device="cuda")
    starts = torch.tensor([0, 6, 12], dtype=torch.int32, device="cuda")
    for seed in range(4):
        u = torch.rand(tokens, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")
        for drawn in (q, None):
            got = w4.tree_sample(p, drawn, draft, mask, starts, u, 6)
            want = w4.tree_sample(p.contiguous(), None if drawn is None else q.contiguous(), draft, mask, starts, u, 6)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    one = torch.arange(tokens + 1, dtype=torch.int32, device="cuda")
    assert torch.equal(w4.tree_sample(p, None, draft, None, one, u, 1)[2], w4.tree_sample(p.contiguous(), None, draft, None, one, u, 1)[2])


def test_probabilities_far_apart_and_many():
    vocab, far = 7000, 1 << 29
    store = torch.empty(6 * far, dtype=torch.bfloat16, device="cuda")
    x = store.as_strided((6, vocab), (far, 1), 4)
    x.copy_(torch.randn((6, vocab), device="cuda"))
    assert torch.equal(w4.probabilities(x), w4.probabilities(x.contiguous()))
    del store, x
    tokens, vocab = 8700, 250000  # 2.2 billion probabilities
    x = torch.zeros((tokens, vocab), dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, 4321, 8589, 8590, 8698, 8699]
    x[rows] = torch.randn((len(rows), vocab), device="cuda").to(torch.bfloat16)
    got = w4.probabilities(x)
    assert torch.equal(got[rows], w4.probabilities(x[rows]))
    assert float(got[8600, 0]) == float(got[8600, vocab - 1]) == np.float32(1) / np.float32(vocab)


@pytest.mark.parametrize("rows,each,far", [(2, 3, 1 << 29), (4, 275, (1 << 21) + 8), (3, 350, (1 << 21) + 5), (4, 520, (1 << 20) + 8), (3, 700, (1 << 20) + 5)])
def test_adapters_and_rows_far_apart(rows, each, far):
    """Tokens, adapters and columns of B past 2^31 elements, in place (few tokens, prompts, rows off 16 bytes)."""
    tokens, inner, outer, rank, store = rows * each, 64, 136, 16, 5
    space = torch.empty(tokens * far, dtype=torch.bfloat16, device="cuda")
    y = space.as_strided((tokens, outer), (far, 1), 0)
    x = torch.empty(tokens * ((far + 7) // 8 * 8), dtype=torch.bfloat16, device="cuda").as_strided((tokens, inner), ((far + 7) // 8 * 8, 1), 64)
    wide = torch.empty(store << 29, dtype=torch.bfloat16, device="cuda")
    a = wide.as_strided((store, rank, inner), (1 << 29, 1 << 12, 1), 0)
    b = wide.as_strided((store, outer, rank), (1 << 29, 1 << 16, 1), 1 << 20)
    for t, std in ((y, 1.0), (x, 1.0), (a, inner ** -0.5), (b, rank ** -0.5)):
        t.copy_(torch.randn(t.shape, device="cuda") * std)
    which = [4, -1, 3, 4][:rows]
    adapter, starts = torch.tensor(which, dtype=torch.int32, device="cuda"), torch.arange(0, tokens + 1, each, dtype=torch.int32, device="cuda")
    want, bound = adapted(y.contiguous(), x.contiguous(), a.contiguous(), b.contiguous(), [e for e in which for _ in range(each)], None)
    w4.lora_add(y, x, a, b, adapter, starts, out=y)
    assert ((y.double().cpu() - want).abs() <= bound).all()
    assert w4.kernel_status() == 0


def test_values_that_are_not_finite_stay_with_their_tokens_in_prompts():
    tokens, inner, outer = 2500, 128, 200
    gen = torch.Generator(device="cuda").manual_seed(0)
    bf16 = lambda *shape: torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    x, y, a, b = bf16(tokens, inner), bf16(tokens, outer), bf16(2, 16, inner), bf16(2, outer, 16)
    x[3, 5], x[2300, 7] = math.inf, math.nan  # the second belongs to a row without an adapter
    y[705, 9] = math.nan
    a[1, 2, 3] = math.nan
    adapter = torch.tensor([0, 1, -1], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 700, 1200, 2500], dtype=torch.int32, device="cuda")
    out = w4.lora_add(y, x, a, b, adapter, starts)
    assert out[:3].isfinite().all() and out[4:700].isfinite().all() and not out[3].isfinite().any()
    assert out[700:1200].isnan().all()
    assert torch.equal(out[1200:].view(torch.int16), y[1200:].view(torch.int16))


def test_as_many_rows_as_there_may_be():
    rows, vocab = 65535, 12
    p = soft((rows, vocab), 3)
    starts = torch.arange(rows + 1, dtype=torch.int32, device="cuda")
    u = torch.rand(rows, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    path, count, token = w4.tree_sample(p, None, torch.zeros(rows, dtype=torch.int64, device="cuda"), None, starts, u, 1)
    w = p.double().cpu().numpy()
    want = (np.cumsum(w, 1) > (u.double().cpu().numpy() * w.sum(1))[:, None]).argmax(1)
    assert (path == 0).all() and (count == 1).all() and (token.cpu().numpy() == want).all()
    mask = torch.full((rows,), 3, device="cuda")
    mask[::2] = 1  # trees of a root and one child
    starts = torch.tensor([*range(0, rows - 1, 2), rows - 1], dtype=torch.int32, device="cuda")
    path, count, _ = w4.tree_sample(p, None, torch.full((rows,), 5, device="cuda"), mask, starts, u, 2)
    taken = (u[1:-1:2] < p[0:-2:2, 5]).int()
    assert torch.equal(count, taken + 1) and torch.equal(path[:, 1], taken * 2 - 1)
    y, x = (torch.randn((rows, 24), device="cuda").to(torch.bfloat16) for _ in range(2))
    a, b = (torch.randn(s, device="cuda").to(torch.bfloat16) for s in ((7, 8, 24), (7, 24, 8)))
    which = torch.arange(rows, device="cuda") % 8 - 1
    out = w4.lora_add(y, x, a, b, which.int(), torch.arange(rows + 1, dtype=torch.int32, device="cuda"))
    want, bound = adapted(y, x, a, b, which.tolist(), None)
    assert ((out.double().cpu() - want).abs() <= bound).all()


def test_two_threads_on_one_stream():
    """Each thread's calls have two launches and a workspace in common with the other's, which grows."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    bf16 = lambda *shape: torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    a, b = bf16(3, 32, 512), bf16(3, 768, 32)
    jobs = []
    for sizes in ((1, 4, 9), (1700, 600, 50)):
        n, starts = sum(sizes), torch.tensor(np.cumsum((0,) + sizes), dtype=torch.int32, device="cuda")
        y, x, adapter = bf16(n, 768), bf16(n, 512), torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
        p, u, draft = soft((n, 300), 1), torch.rand(n, generator=gen, device="cuda"), torch.randint(0, 300, (n,), generator=gen, device="cuda")
        trees = torch.tensor([0, *range(2, n + 1, 3)], dtype=torch.int32, device="cuda")

        def run(y=y, x=x, adapter=adapter, starts=starts, p=p, u=u, draft=draft, trees=trees):
            return w4.lora_add(y, x, a, b, adapter, starts), w4.probabilities(y), *w4.tree_sample(p, p, draft, None, trees, u, 3)
        jobs.append(run)
    want = [run() for run in jobs]
    torch.cuda.synchronize()
    got, errors, together = [[], []], [], threading.Barrier(2)

    def work(i):
        try:
            together.wait()
            for _ in range(60):
                got[i].append(jobs[i]())
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
        assert len(got[i]) == 60 and all(torch.equal(o, w) for outs in got[i] for o, w in zip(outs, want[i]))


def test_outputs_are_plain_tensors_of_their_own():
    p, starts = soft((4, 50), 0), torch.arange(5, dtype=torch.int32, device="cuda")
    args = (p, None, torch.zeros(4, dtype=torch.int64, device="cuda"), None, starts, torch.rand(4, device="cuda"), 1)
    with torch.inference_mode():
        first = w4.tree_sample(*args)
    kept = [t.clone() for t in first]
    rest = [w4.tree_sample(*args) for _ in range(70)]
    for outs in rest:
        for t in outs:
            t.fill_(-9)
    for t, k in zip(first, kept):
        assert torch.equal(t, k) and not t._is_view() and not t.is_inference() and t._version == 0
    y, x, a, b = (torch.ones(s, dtype=torch.bfloat16, device="cuda") for s in ((2, 8), (2, 8), (1, 8, 8), (1, 8, 8)))
    outs = [w4.lora_add(y, x, a, b, torch.zeros(2, dtype=torch.int32, device="cuda")) for _ in range(70)]
    for t in outs[:-1]:
        t.zero_()
    assert (outs[-1] == 65).all() and not outs[-1]._is_view() and outs[-1]._version == 0
