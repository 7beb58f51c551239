"""Adapters, products, cache, probabilities and the sampled walk together, as a
decoding loop of a model that samples uses them."""
import importlib.util
import os
import sys

import numpy as np
import pytest
import torch

import gemm_w4a16_group_gb300 as w4
from sample_helpers import adapted, sampled

pytestmark = pytest.mark.gpu

EXAMPLES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")
STEPS = 12


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("sampled_step", os.path.join(EXAMPLES, "sampled_step.py"))
    module = importlib.util.module_from_spec(spec)
    before = list(sys.path)
    spec.loader.exec_module(module)
    sys.path[:] = before
    return module


@pytest.fixture(scope="module")
def model(ex):
    return ex.Adapted()


def prompts(ex):
    gen = torch.Generator().manual_seed(5)
    return [torch.randint(0, ex.VOCAB, (n,), generator=gen).cuda() for n in (37, 90, 12)]


def test_greedy_users_walk_as_tree_accept_does(ex, model, monkeypatch):
    """At temperature 0 the walk is tree_accept's over the same logits' maxima, whatever the drafter's q. (Not compared
    with a run of single tokens: products of other row counts round a logit to its neighbour, and two may be as large.)"""
    logits, calls = [], []

    def seen(x, *a, **kw):
        logits.append(x)
        return w4.__dict__["_probabilities"](x, *a, **kw)

    def walk(p, q, draft, mask, starts, u, max_tree):
        out = w4.__dict__["_tree_sample"](p, q, draft, mask, starts, u, max_tree)
        first = [int((row == row.max()).nonzero()[0, 0]) for row in logits[-1]]  # (of several equal ones the first)
        path, count, token = w4.tree_accept(torch.tensor(first, device="cuda"), draft,
                                            torch.ones_like(draft) if mask is None else mask, starts, max_tree)
        assert torch.equal(out[0], path) and torch.equal(out[1], count) and torch.equal(out[2], token)
        calls.append(int(count.max()))
        return out

    for name, checked in (("probabilities", seen), ("tree_sample", walk)):
        monkeypatch.setattr(w4, "_" + name, getattr(w4, name), raising=False)
        monkeypatch.setattr(w4, name, checked)
    said = [ex.decode(model, prompts(ex), which, 0.0, STEPS, trees)[0] for which, trees in (([0, 1, -1], True), ([-1, -1, -1], True), ([0, 1, -1], False))]
    assert len(calls) > 3 * STEPS // 2
    assert said[0][0] != said[1][0] and said[0][1] != said[1][1]  # the adapters are heard


def test_every_call_of_a_sampled_run(ex, model, monkeypatch):
    """Each operator's result where it is called, against 64 bits; and the same numbers make the same run."""
    seen = []

    def probabilities(logits, temperature=None, *a, **kw):
        out = w4.__dict__["_probabilities"](logits, temperature, *a, **kw)
        x = logits.double() / temperature.double()[:, None]
        x = (x - x.amax(1, keepdim=True)).exp()
        want = x / x.sum(1, keepdim=True)
        # (off by 2^-17 + 2^-23 (max - l) / T of itself; below 2^-126 it may be 0)
        away = (logits.double().amax(1, keepdim=True) - logits.double()) / temperature.double()[:, None]
        assert ((out.double() - want).abs() <= want * (2.0 ** -17 + 2.0 ** -23 * away) + 2.0 ** -126).all()
        return out

    def tree_sample(p, q, draft, mask, starts, u, max_tree):
        path, count, token = w4.__dict__["_tree_sample"](p, q, draft, mask, starts, u, max_tree)
        edge = starts.tolist()
        for b, (s, t) in enumerate(zip(edge, edge[1:])):
            words = [1] if mask is None else mask[s:t].tolist()
            way, drawn = sampled(p[s:t].cpu().numpy(), None if q is None else q[s:t].cpu().numpy(), draft[s:t].tolist(),
                                 words, u[s:t].cpu().numpy(), exact=False)
            assert path[b, :int(count[b])].tolist() == way and int(token[b]) == drawn
            seen.append(len(way))
        return path, count, token

    def lora_add(y, x, a, b, adapter, starts, scale, out):
        before = y.clone()
        w4.__dict__["_lora_add"](y, x, a, b, adapter, starts, scale, out=out)
        which = np.repeat(adapter.tolist(), np.diff(starts.tolist())).tolist()
        want, bound = adapted(before, x, a, b, which, scale)
        assert ((out.double().cpu() - want).abs() <= bound).all()

    for name, checked in (("probabilities", probabilities), ("tree_sample", tree_sample), ("lora_add", lora_add)):
        monkeypatch.setattr(w4, "_" + name, getattr(w4, name), raising=False)
        monkeypatch.setattr(w4, name, checked)
    said, _ = ex.decode(model, prompts(ex), [1, 0, -1], 2.0, STEPS, True)
    assert max(seen) > 1  # a drafted token was accepted
    monkeypatch.undo()
    assert ex.decode(model, prompts(ex), [1, 0, -1], 2.0, STEPS, True)[0] == said  # the same numbers, the same run
    assert ex.decode(model, prompts(ex), [1, 0, -1], 2.0, STEPS, True, seed=2)[0] != said


def test_a_step_in_a_graph(ex, model):
    """Adapters, head, probabilities and the walk captured once, replayed with other numbers."""
    rows = 3
    x = torch.randn((rows, ex.HIDDEN), device="cuda").to(torch.bfloat16)
    adapter, starts = ex.ints(0, -1, 1), ex.ints(0, 1, 2, 3)
    a, b = model.a[0], torch.randn((ex.STORE, ex.VOCAB, ex.RANK), device="cuda").to(torch.bfloat16)
    u, t = torch.rand(rows, device="cuda"), torch.full((rows,), 1.5, device="cuda")
    draft = torch.zeros(rows, dtype=torch.int64, device="cuda")

    def step():
        y = model.head_of(x)
        p = w4.probabilities(w4.lora_add(y, x, a, b, adapter, starts, model.scale, out=y), t)
        return p, w4.tree_sample(p, None, draft, None, starts, u, 1)[2]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p, token = step()
    for _ in range(20):
        u.uniform_()
        x.normal_()
        graph.replay()
        want_p, want = step()
        assert torch.equal(p, want_p) and torch.equal(token, want)
