"""Host threads that call the cache operators on one stream, on CPU: the
compute entry points are replaced by recorders that let go of the interpreter,
as the real ones do."""
import ctypes
import threading
import time

import pytest
import torch

import gemm_w4a16_group_gb300 as w4

BF = torch.bfloat16


class SlowLib:
    """tree_attention makes two launches that share the workspace: no other call may use it in between."""

    def __init__(self, real):
        self.real, self.using, self.clashes, self.used = real, set(), 0, []

    def w4a16_tree_attention(self, *args):
        workspace = args[-2]
        self.used.append(workspace)
        if workspace in self.using:
            self.clashes += 1
        self.using.add(workspace)
        time.sleep(0.001)
        self.using.discard(workspace)
        return 0

    def __getattr__(self, name):
        return getattr(self.real, name)


@pytest.fixture
def slow(monkeypatch):
    f = SlowLib(w4.lib())
    monkeypatch.setattr(w4, "lib", lambda auto_build=True: f)
    monkeypatch.setattr(w4, "_is_device_tensor", lambda t: True)
    monkeypatch.setattr(w4, "_stream", lambda stream, device=None: ctypes.c_void_p(stream or 0))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    w4._workspaces.clear()
    yield f
    w4._workspaces.clear()


def attention(max_tree=4, **kw):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    cache = torch.zeros(6, 2, 16, 64, dtype=BF)
    out = torch.zeros(5, 8, 64, dtype=BF)
    w4.tree_attention(torch.zeros(5, 8, 64, dtype=BF), cache, cache, i32(3, 2), i32(3), i32(4), None, max_tree, out=out, **kw)


def in_threads(n, call):
    errors = []

    def run():
        try:
            for _ in range(10):
                call()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run) for _ in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_one_call_at_a_time_uses_the_kept_workspace(slow):
    in_threads(4, attention)
    assert len(slow.used) == 40 and slow.clashes == 0


def test_a_given_workspace_waits_for_nobody(slow):
    def call():
        attention(workspace=torch.empty(w4.tree_attention_workspace_bytes(8, 2, 64, 4), dtype=torch.uint8))

    in_threads(2, call)
    assert slow.clashes == 0
    assert not w4._workspaces


def test_few_workspaces_are_kept(slow, monkeypatch):
    """One per stream, of the streams used last."""
    monkeypatch.setattr(w4, "_capturing", lambda stream: False)
    monkeypatch.setattr(w4, "_empty", lambda shape, dtype, like, stream: torch.empty(shape, dtype=dtype))
    for stream in range(1, 101):
        attention(stream=stream)
    assert 1 <= len(w4._workspaces) <= 16
    kept = {id(t) for t in w4._workspaces.values()}
    attention(stream=100)
    assert {id(t) for t in w4._workspaces.values()} == kept
