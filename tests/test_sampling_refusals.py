"""What the calls of the sampled verify step and of the adapters refuse before
anything is launched, and what they do when there is nothing to do, on CPU: the
C entry points' argument checks, and the binding's checks (the compute entry
points replaced by a recorder)."""
import ctypes

import pytest
import torch

import gemm_w4a16_group_gb300 as w4

INVALID, MISALIGNED = -1, -2
FAKE = 1 << 20  # an aligned non-null address; never dereferenced on these paths
FAR = 1 << 40
BF = torch.bfloat16


@pytest.fixture(scope="module")
def L():
    return w4.lib()


def check(call, good, invalid, misaligned):
    """`call` refuses each change of `good`, a dict of arguments in order."""
    for code, cases in ((INVALID, invalid), (MISALIGNED, misaligned)):
        for changes in cases:
            assert call(*{**good, **changes}.values()) == code, changes


def test_probabilities(L):
    good = dict(logits=FAKE, row=100, temperature=None, floor=None, tokens=3, vocab=100, out=FAKE, stream=None)
    check(L.w4a16_probabilities, good,
          [dict(logits=None), dict(out=None), dict(tokens=0), dict(tokens=-1), dict(tokens=1 << 27), dict(vocab=0), dict(vocab=1 << 27),
           dict(row=-1)],
          [dict(logits=FAKE + 1), dict(temperature=FAKE + 2), dict(floor=FAKE + 1), dict(out=FAKE + 2)])


def test_tree_sample(L):
    good = dict(p=FAKE, p_row=100, q=FAKE, q_row=100, vocab=100, draft=FAKE, mask=None, starts=FAKE, u=FAKE, rows=2, tokens=4,
                max_tree=4, path=FAKE, count=FAKE, token=FAKE, stream=None)
    check(L.w4a16_tree_sample, good,
          [{k: None} for k in ("p", "draft", "starts", "u", "path", "count", "token")] +
          [dict(p_row=-1), dict(q_row=-4), dict(vocab=0), dict(vocab=1 << 27), dict(rows=0), dict(rows=65536), dict(tokens=0),
           dict(tokens=1 << 27), dict(max_tree=0), dict(max_tree=65)],
          [dict(p=FAKE + 2), dict(q=FAKE + 1), dict(draft=FAKE + 4), dict(mask=FAKE + 4), dict(starts=FAKE + 2), dict(u=FAKE + 2),
           dict(path=FAKE + 2), dict(count=FAKE + 1), dict(token=FAKE + 4)])


LORA = dict(y=FAKE, y_row=64, x=FAKE, x_row=32, a=FAKE, a_adapter=512, a_row=32, b=FAKE, b_adapter=1024, b_row=16, scale=None,
            adapter=FAKE, starts=FAKE, rows=2, tokens=4, adapters=3, rank=16, inner=32, outer=64, out=FAR, out_row=64,
            workspace=FAKE, stream=None)


def test_lora_add(L):
    check(L.w4a16_lora_add, LORA,
          [{k: None} for k in ("y", "x", "a", "b", "adapter", "out", "workspace")] +
          [dict(rank=0), dict(rank=4), dict(rank=12), dict(rank=136), dict(rank=-8), dict(inner=0), dict(inner=36), dict(inner=-32),
           dict(outer=0), dict(outer=1 << 27), dict(tokens=0), dict(rows=0), dict(rows=65536), dict(adapters=0), dict(adapters=4097),
           dict(starts=None), dict(y_row=-64), dict(x_row=-32), dict(a_adapter=-8), dict(a_row=-8), dict(b_adapter=-8), dict(b_row=-8),
           dict(out_row=-64), dict(out_row=63), dict(y_row=1 << 30), dict(x_row=1 << 30), dict(out_row=1 << 30)],
          [dict(x=FAKE + 8), dict(a=FAKE + 8), dict(b=FAKE + 2), dict(workspace=FAKE + 128), dict(y=FAKE + 1), dict(out=FAR + 1),
           dict(scale=FAKE + 2), dict(adapter=FAKE + 2), dict(starts=FAKE + 2), dict(x_row=36), dict(a_adapter=516), dict(a_row=36),
           dict(b_adapter=1028), dict(b_row=20)])


def test_lora_add_outputs_that_overlap_y(L):
    """y itself and other columns of it may be written (the call goes on to look for a GPU); anything between is refused."""
    def rc(**k):
        return L.w4a16_lora_add(*{**LORA, **k}.values())

    wide = dict(y_row=200, out_row=200)
    free = [dict(out=FAKE), dict(out=FAKE + 128, **wide), dict(out=FAKE + 272, **wide), dict(out=FAKE + 3 * 400 + 128, **wide),
            dict(out=FAKE + 2 * (3 * 64 + 64)), dict(out=FAKE - 2 * (3 * 64 + 64)), dict(out=FAKE + 400 * 2 + 128, **wide),
            dict(out=FAKE + 128, tokens=1, y_row=1, out_row=5), dict(y_row=0, out=FAKE + 128)]
    for k in free:
        assert rc(**k) not in (INVALID, MISALIGNED), k
    for k in (dict(out=FAKE + 2), dict(out=FAKE + 128), dict(out=FAKE - 128), dict(out=FAKE + 126, **wide), dict(out=FAKE + 274, **wide),
              dict(out=FAKE, out_row=72), dict(out=FAKE + 16, y_row=200, out_row=64), dict(y_row=0, out=FAKE + 64), dict(y_row=0, out=FAKE),
              dict(out=FAKE + 64, tokens=1), dict(y_row=1 << 41)):
        assert rc(**k) == INVALID, k


def test_workspace_sizes(L):
    for bad in ((0, 16, 64), (1, 0, 64), (1, 12, 64), (1, 136, 64), (1, 16, 0), (1, 16, 36), (1 << 27, 16, 64)):
        assert w4.lora_workspace_bytes(*bad) == 0
    for tokens in (1, 15, 16, 17, 100, 512, 513, 5000, 100000):
        for rank, padded in ((8, 8), (16, 16), (24, 32), (64, 64), (72, 128)):
            for inner in (8, 64, 5120, 17408):
                n = w4.lora_workspace_bytes(tokens, rank, inner)
                assert n % 256 == 0 and n >= tokens * padded * 4
                assert n <= 32 * tokens * padded * 4 + 256 and n < 32 * 1024 * 1024 + 4 * tokens * padded * 4
    for rank, inner in ((8, 64), (16, 5120), (64, 17408), (128, 17408)):  # one for the largest call is enough for all
        sizes = [w4.lora_workspace_bytes(t, rank, inner) for t in range(1, 2100)]
        assert sizes == sorted(sizes)
        assert w4.lora_workspace_bytes(300, rank, inner) <= w4.lora_workspace_bytes(300, rank, inner + 512)
        assert w4.lora_workspace_bytes(300, rank - 8 or 8, inner) <= w4.lora_workspace_bytes(300, rank, inner)


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------
@pytest.fixture
def calls(monkeypatch):
    real, made = w4.lib(), []

    class Recorder:
        def __getattr__(self, name):
            if name.endswith("_bytes") or name == "w4a16_strerror":
                return getattr(real, name)
            return lambda *a: made.append((name, a)) or 0

    monkeypatch.setattr(w4, "lib", lambda auto_build=True: Recorder())
    monkeypatch.setattr(w4, "_is_device_tensor", lambda t: True)
    monkeypatch.setattr(w4, "_stream", lambda stream, device=None: ctypes.c_void_p(0))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    w4._small_outputs.clear()
    w4._workspaces.clear()
    yield made
    w4._small_outputs.clear()
    w4._workspaces.clear()


def test_tensors_must_be_on_the_gpu():
    with pytest.raises(ValueError, match="CUDA"):
        w4.probabilities(torch.zeros(2, 8, dtype=BF))
    with pytest.raises(ValueError, match="CUDA"):
        w4.tree_sample(torch.zeros(2, 8), None, torch.zeros(2, dtype=torch.int64), None, torch.zeros(2, dtype=torch.int32), torch.zeros(2), 2)
    with pytest.raises(ValueError, match="CUDA"):
        lora()


def test_probabilities_binding(calls):
    x = torch.zeros(3, 50, dtype=BF)
    out = w4.probabilities(x)
    assert out.shape == (3, 50) and out.dtype == torch.float32
    name, a = calls[-1]
    assert name == "w4a16_probabilities" and a[:6] == (x.data_ptr(), 50, None, None, 3, 50) and a[6] == out.data_ptr()
    t, f = torch.ones(3), torch.zeros(3)
    w4.probabilities(x[:, 5:20], t, f)
    assert calls[-1][1][:6] == (x.data_ptr() + 10, 50, t.data_ptr(), f.data_ptr(), 3, 15)
    n = len(calls)
    for bad, error in ((dict(logits=x.float()), TypeError), (dict(logits=x.view(-1)), ValueError), (dict(logits=x.T), ValueError),
                       (dict(temperature=t[:2]), ValueError), (dict(temperature=t.double()), TypeError), (dict(floor=torch.zeros(6)[::2]), ValueError),
                       (dict(floor=f.to(BF)), TypeError), (dict(out=torch.zeros(3, 49)), ValueError), (dict(out=x), TypeError)):
        with pytest.raises(error):
            w4.probabilities(**{"logits": x, **bad})
    assert len(calls) == n
    for shape in ((0, 50), (3, 0)):
        assert w4.probabilities(torch.zeros(shape, dtype=BF)).shape == shape
    assert len(calls) == n


def sample(**changes):
    a = dict(p=torch.zeros(4, 30), q=torch.zeros(4, 30), draft=torch.zeros(4, dtype=torch.int64), mask=torch.zeros(4, dtype=torch.int64),
             starts=torch.zeros(3, dtype=torch.int32), u=torch.zeros(4), max_tree=3)
    a.update(changes)
    return a, w4.tree_sample(**a)


def test_tree_sample_binding(calls):
    a, (path, count, token) = sample()
    name, got = calls[-1]
    assert name == "w4a16_tree_sample"
    assert got[:12] == (a["p"].data_ptr(), 30, a["q"].data_ptr(), 30, 30, a["draft"].data_ptr(), a["mask"].data_ptr(),
                        a["starts"].data_ptr(), a["u"].data_ptr(), 2, 4, 3)
    assert got[12:15] == (path.data_ptr(), count.data_ptr(), token.data_ptr())
    assert path.shape == (2, 3) and count.shape == (2,) and token.shape == (2,)
    assert (path.dtype, count.dtype, token.dtype) == (torch.int32, torch.int32, torch.int64)
    a, _ = sample(q=None, mask=None)
    assert calls[-1][1][2:4] == (None, 0) and calls[-1][1][6] is None
    n = len(calls)
    for bad, error in ((dict(p=torch.zeros(4, 30, dtype=BF)), TypeError), (dict(p=torch.zeros(30, 4).T), ValueError), (dict(p=torch.zeros(120)), ValueError),
                       (dict(q=torch.zeros(4, 31)), ValueError), (dict(q=torch.zeros(3, 30)), ValueError), (dict(q=torch.zeros(4, 30).double()), TypeError),
                       (dict(draft=torch.zeros(4, dtype=torch.int32)), TypeError), (dict(draft=torch.zeros(3, dtype=torch.int64)), ValueError),
                       (dict(mask=torch.zeros(5, dtype=torch.int64)), ValueError), (dict(starts=torch.zeros(3, dtype=torch.int64)), TypeError),
                       (dict(u=torch.zeros(4, dtype=torch.float64)), TypeError), (dict(u=torch.zeros(2)), ValueError),
                       (dict(path=torch.zeros(2, 4, dtype=torch.int32)), ValueError), (dict(count=torch.zeros(2, dtype=torch.int64)), TypeError),
                       (dict(token=torch.zeros(3, dtype=torch.int64)), ValueError)):
        with pytest.raises(error):
            sample(**bad)
    assert len(calls) == n


@pytest.mark.parametrize("rows,tokens", [(3, 0), (0, 0), (0, 2)])
def test_tree_sample_with_nothing_to_do(calls, rows, tokens):
    _, (path, count, token) = sample(p=torch.zeros(tokens, 30), q=None, draft=torch.zeros(tokens, dtype=torch.int64), mask=None,
                                     starts=torch.zeros(rows + 1, dtype=torch.int32), u=torch.zeros(tokens))
    assert path.tolist() == [[-1] * 3] * rows and count.tolist() == [0] * rows and token.tolist() == [-1] * rows
    with pytest.raises(w4.W4A16Error):
        sample(p=torch.zeros(tokens, 30), q=None, draft=torch.zeros(tokens, dtype=torch.int64), mask=None,
               starts=torch.zeros(rows + 1, dtype=torch.int32), u=torch.zeros(tokens), max_tree=65)
    assert calls == []


def lora(**changes):
    a = dict(y=torch.zeros(5, 24, dtype=BF), x=torch.zeros(5, 32, dtype=BF), a=torch.zeros(3, 16, 32, dtype=BF), b=torch.zeros(3, 24, 16, dtype=BF),
             adapter=torch.zeros(2, dtype=torch.int32), starts=torch.zeros(3, dtype=torch.int32), scale=torch.zeros(3))
    a.update(changes)
    return a, w4.lora_add(**a)


def test_lora_add_binding(calls):
    a, out = lora()
    name, got = calls[-1]
    assert name == "w4a16_lora_add" and out.shape == (5, 24) and out.dtype == BF
    assert got[:21] == (a["y"].data_ptr(), 24, a["x"].data_ptr(), 32, a["a"].data_ptr(), 512, 32, a["b"].data_ptr(), 384, 16,
                        a["scale"].data_ptr(), a["adapter"].data_ptr(), a["starts"].data_ptr(), 2, 5, 3, 16, 32, 24, out.data_ptr(), 24)
    a, out = lora(out=(y := torch.zeros(5, 24, dtype=BF)), y=y)
    assert out is y and calls[-1][1][19] == y.data_ptr() == calls[-1][1][0]
    lora(starts=None, adapter=torch.zeros(5, dtype=torch.int32), scale=None)
    assert calls[-1][1][10] is None and calls[-1][1][12] is None and calls[-1][1][13:15] == (5, 5)
    need = w4.lora_workspace_bytes(5, 16, 32)
    ws = torch.zeros(need, dtype=torch.uint8)
    lora(workspace=ws)
    assert calls[-1][1][21] == ws.data_ptr()
    n = len(calls)
    for bad, error in ((dict(y=torch.zeros(5, 24)), TypeError), (dict(y=torch.zeros(24, 5, dtype=BF).T), ValueError), (dict(y=torch.zeros(4, 24, dtype=BF)), ValueError),
                       (dict(x=torch.zeros(5, 40, dtype=BF)), ValueError), (dict(x=torch.zeros(5, 32)), TypeError), (dict(a=torch.zeros(16, 32, dtype=BF)), ValueError),
                       (dict(a=torch.zeros(3, 32, 16, dtype=BF).transpose(1, 2)), ValueError), (dict(b=torch.zeros(3, 24, 8, dtype=BF)), ValueError),
                       (dict(b=torch.zeros(2, 24, 16, dtype=BF)), ValueError), (dict(b=torch.zeros(3, 25, 16, dtype=BF)), ValueError),
                       (dict(starts=None), ValueError), (dict(starts=torch.zeros(4, dtype=torch.int32)), ValueError), (dict(scale=torch.zeros(2)), ValueError),
                       (dict(scale=torch.zeros(3, dtype=BF)), TypeError), (dict(adapter=torch.zeros(2, dtype=torch.int64)), TypeError),
                       (dict(out=torch.zeros(5, 25, dtype=BF)), ValueError), (dict(out=torch.zeros(5, 24)), TypeError),
                       (dict(workspace=ws[1:]), ValueError), (dict(workspace=ws.view(torch.int8)), TypeError),
                       (dict(a=torch.zeros(3, 12, 32, dtype=BF), b=torch.zeros(3, 24, 12, dtype=BF)), w4.W4A16Error),
                       (dict(x=torch.zeros(5, 36, dtype=BF), a=torch.zeros(3, 16, 36, dtype=BF)), w4.W4A16Error)):
        with pytest.raises(error):
            lora(**bad)
    assert len(calls) == n


@pytest.mark.parametrize("rows,tokens", [(3, 0), (0, 0), (0, 2)])
def test_lora_add_with_nothing_to_do(calls, rows, tokens):
    given = torch.ones(tokens, 24, dtype=BF)
    a = dict(y=torch.zeros(tokens, 24, dtype=BF), x=torch.zeros(tokens, 32, dtype=BF), adapter=torch.zeros(rows, dtype=torch.int32),
             starts=torch.zeros(rows + 1, dtype=torch.int32))
    assert lora(**a)[1].shape == (tokens, 24)
    assert lora(out=given, **a)[1] is given and (given == 1).all()
    assert calls == []


def test_one_workspace_for_all_calls_of_a_stream(calls):
    lora()
    lora(x=torch.zeros(5, 32, dtype=BF))
    assert calls[0][1][21] == calls[1][1][21] and len(w4._workspaces) == 1
