"""The decoding loops of the examples report the status that a kernel left, which
reading clears (on CPU: the model's steps replaced by counted ones)."""
import importlib.util
import os
import sys

import pytest
import torch

import gemm_w4a16_group_gb300 as w4

EXAMPLES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")


def load(name):
    spec = importlib.util.spec_from_file_location(name, os.path.join(EXAMPLES, name + ".py"))
    module = importlib.util.module_from_spec(spec)
    before = list(sys.path)
    spec.loader.exec_module(module)
    sys.path[:] = before
    return module


@pytest.fixture
def status(monkeypatch):
    """A status of -6, once."""
    left = [-6]
    monkeypatch.setattr(w4, "kernel_status", lambda: left.pop() if left else 0)
    return left


def test_sampled_step(monkeypatch, status):
    ex = load("sampled_step")

    class Users:
        def __init__(self, *a):
            self.last = torch.zeros(1, dtype=torch.int64)

        def step(self):
            return [[7]]
    monkeypatch.setattr(ex, "Users", Users)
    with pytest.raises(RuntimeError, match="kernel status -6"):
        ex.decode(None, [None], [0], 1.0, 3, False)
    assert ex.decode(None, [None], [0], 1.0, 3, False) == ([[0, 7, 7]], 2)


def test_verify_step(monkeypatch, status):
    ex = load("verify_step")

    class Cache:
        k = v = table = lengths = refs = None

        def __init__(self, *a, **kw):
            pass
    monkeypatch.setattr(ex, "Cache", Cache)
    monkeypatch.setattr(ex, "prefill", lambda *a: 5)
    monkeypatch.setattr(ex, "ints", lambda *a: torch.tensor(a, dtype=torch.int32))
    monkeypatch.setattr(w4, "kv_fork", lambda *a: 1)
    monkeypatch.setattr(w4, "kv_free", lambda *a: None)
    with pytest.raises(RuntimeError, match="kernel status -6"):
        ex.speculative(None, [None], 1, [[]])
    assert ex.speculative(None, [None], 1, [[]]) == ([[5]], 0)
