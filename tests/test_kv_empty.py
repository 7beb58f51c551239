"""Cache calls with nothing to do, on CPU: a step without new tokens, no rows
to free, branch or give room to. Arguments are checked as ever, nothing is
launched, and the outputs say that there was nothing."""
import ctypes

import pytest
import torch

import gemm_w4a16_group_gb300 as w4

BF = torch.bfloat16


@pytest.fixture
def calls(monkeypatch):
    """Names of the entry points called."""
    real, made = w4.lib(), []

    class Recorder:
        def __getattr__(self, name):
            if name.endswith("_bytes") or name == "w4a16_strerror":
                return getattr(real, name)
            return lambda *a: made.append(name) or 0

    monkeypatch.setattr(w4, "lib", lambda auto_build=True: Recorder())
    monkeypatch.setattr(w4, "_is_device_tensor", lambda t: True)
    monkeypatch.setattr(w4, "_stream", lambda stream, device=None: ctypes.c_void_p(0))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    w4._small_outputs.clear()
    yield made
    w4._small_outputs.clear()


def i32(*shape, fill=0):
    return torch.full(shape, fill, dtype=torch.int32)


def args(tokens=0, rows=3):
    return dict(q=torch.zeros(tokens, 8, 64, dtype=BF), k=torch.zeros(tokens, 2, 64, dtype=BF), v=torch.zeros(tokens, 2, 64, dtype=BF),
                k_cache=torch.zeros(6, 2, 16, 64, dtype=BF), v_cache=torch.zeros(6, 2, 16, 64, dtype=BF), table=i32(rows, 2),
                lengths=i32(rows, fill=5), starts=i32(rows + 1), mask=torch.zeros(tokens, dtype=torch.int64),
                ids=torch.zeros(tokens, dtype=torch.int64), refs=i32(6), none=i32(0))


@pytest.mark.parametrize("rows,tokens", [(3, 0), (0, 0), (0, 2)])  # (0, 2): padding tokens alone
@pytest.mark.parametrize("masked", [False, True])
def test_no_new_tokens(calls, rows, tokens, masked):
    a = args(tokens, rows)
    mask = a["mask"] if masked else None
    w4.kv_append(a["k"], a["v"], a["k_cache"], a["v_cache"], a["table"], a["lengths"], a["starts"])
    out = w4.tree_attention(a["q"], a["k_cache"], a["v_cache"], a["table"], a["lengths"], a["starts"], mask, 4)
    assert out.shape == (tokens, 8, 64) and out.dtype == BF
    given = torch.ones(tokens, 8, 64, dtype=BF)
    assert w4.tree_attention(a["q"], a["k_cache"], a["v_cache"], a["table"], a["lengths"], a["starts"], mask, 4, out=given) is given
    assert (given == 1).all()
    path, count, token = w4.tree_accept(a["ids"], a["ids"], mask, a["starts"], 4)
    assert path.tolist() == [[-1] * 4] * rows and count.tolist() == [0] * rows and token.tolist() == [-1] * rows
    assert path.shape == (rows, 4) and (path.dtype, count.dtype, token.dtype) == (torch.int32, torch.int32, torch.int64)
    assert calls == []


def test_compaction_of_no_rows(calls):
    a = args(rows=0)
    out = w4.kv_compact(a["k_cache"], a["v_cache"], a["table"], a["lengths"], i32(0, 4), a["none"])
    assert out.shape == (0,) and out.dtype == torch.int32 and calls == []


def test_no_rows_named(calls):
    a = args()
    before = [a[n].clone() for n in ("table", "lengths", "refs")]
    w4.kv_free(a["table"], a["lengths"], a["refs"], a["none"])
    ok = w4.kv_fork(a["k_cache"], a["v_cache"], a["table"], a["lengths"], a["refs"], a["none"], a["none"])
    assert ok.tolist() == [1]
    given = i32(1)
    assert w4.kv_reserve(a["table"], a["refs"], a["none"], a["none"], 16, ok=given) is given and given.tolist() == [1]
    assert calls == [] and all(torch.equal(x, a[n]) for x, n in zip(before, ("table", "lengths", "refs")))


def test_arguments_are_checked_all_the_same(calls):
    a = args()
    with pytest.raises(ValueError, match="starts"):
        w4.kv_append(a["k"], a["v"], a["k_cache"], a["v_cache"], a["table"], a["lengths"], i32(3))
    with pytest.raises(ValueError, match="mask"):
        w4.tree_attention(a["q"], a["k_cache"], a["v_cache"], a["table"], a["lengths"], a["starts"], torch.zeros(2, dtype=torch.int64), 4)
    with pytest.raises(w4.W4A16Error):
        w4.tree_attention(a["q"], a["k_cache"], a["v_cache"], a["table"], a["lengths"], a["starts"], None, 65)
    with pytest.raises(w4.W4A16Error):
        w4.tree_accept(a["ids"], a["ids"], None, a["starts"], 65)
    with pytest.raises(w4.W4A16Error):
        w4.kv_reserve(a["table"], a["refs"], a["none"], a["none"], 24)
    with pytest.raises(TypeError, match="rows"):
        w4.kv_free(a["table"], a["lengths"], a["refs"], torch.zeros(0))
    assert calls == []
