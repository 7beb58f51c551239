"""What callers get as outputs of the small cache calls, on CPU: plain new
tensors, whatever mode and thread earlier calls ran in."""
import threading

import pytest
import torch

import gemm_w4a16_group_gb300 as w4


@pytest.fixture(autouse=True)
def host(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    w4._small_outputs.clear()
    yield
    w4._small_outputs.clear()


def out(shape=(3,), dtype=torch.float32):
    return w4._small_out(shape, dtype, torch.zeros(1), -1, None, 0)


def test_after_a_call_in_inference_mode():
    """Outputs made then may be changed in place and saved for backward."""
    with torch.inference_mode():
        out().zero_()
    for _ in range(70):
        x = out().zero_()
        assert not x.is_inference()
        x += 1
        w = torch.ones(3, requires_grad=True)
        (w * x).sum().backward()
        assert torch.equal(w.grad, torch.ones(3))


def test_in_inference_mode_after_a_call_outside():
    out()
    with torch.inference_mode():
        x = out().zero_()
        x += 1
        assert torch.equal(x * 2, torch.full((3,), 2.0))


def test_changing_one_leaves_another_saved_for_backward():
    a, b = out().zero_(), out().zero_()
    w = torch.ones(3, requires_grad=True)
    y = (w * a).sum()
    b += 1
    assert b._version != a._version
    y.backward()
    assert torch.equal(w.grad, torch.zeros(3))


def test_a_tensor_that_needs_a_gradient_may_be_added_in_place():
    x = out().zero_()
    w = torch.ones(3, requires_grad=True)
    x += w
    x.sum().backward()
    assert torch.equal(w.grad, torch.ones(3))
    assert not out()._is_view()


def test_what_one_output_keeps_alive():
    """Up to 32 outputs of its size, and of larger ones none but itself."""
    for shape in ((1,), (64,), (4096,)):
        assert out(shape).untyped_storage().nbytes() <= 32 * 4 * shape[0] <= 512 * 1024
    assert out((4097,)).untyped_storage().nbytes() == 4 * 4097


def test_threads():
    """Each output is handed out once, and every call gets one."""
    got, errors = [], []
    together = threading.Barrier(4)

    def work():
        try:
            together.wait()
            got.extend([out((7,)) for _ in range(20000)])
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert len({x.data_ptr() for x in got}) == len(got) == 80000


def test_a_batch_that_another_thread_empties(monkeypatch):
    """The last output of a batch taken between the look at it and the taking."""
    first = out()

    class Emptied(list):
        def __bool__(self):
            return True  # as it was a moment ago

    for key in w4._small_outputs:
        w4._small_outputs[key] = Emptied()
    second = out()
    assert second.data_ptr() != first.data_ptr() and second.shape == first.shape


def test_the_stream_that_is_asked_about_capture(monkeypatch):
    """A captured stream's buffers come from the graph, also when it is given to the call and another one is current."""
    current, made = ["outer"], []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current.append(self.stream)

        def __exit__(self, *a):
            current.pop()

    def empty(shape, dtype, like, stream):
        made.append(stream)
        return torch.empty(shape, dtype=dtype)

    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: current[-1] == "captured")
    monkeypatch.setattr(w4, "_empty", empty)
    like = torch.zeros(1)
    w4._workspaces.clear()
    for _ in range(2):
        assert w4._workspace(100, like, -1, "captured", 5).numel() == 100
        assert w4._small_out((3,), torch.int32, like, -1, "captured", 5).untyped_storage().nbytes() == 12
    assert made == ["captured"] * 4 and not w4._workspaces and not w4._small_outputs
    w4._workspace(100, like, -1, "other", 6)
    w4._small_out((3,), torch.int32, like, -1, "other", 6)
    assert len(w4._workspaces) == len(w4._small_outputs) == 1
    w4._workspaces.clear()
