"""What the paged-cache calls refuse before anything is launched, on CPU: the
C entry points' argument checks, and the binding's checks of what a plain
pointer cannot carry (the compute entry points replaced by a recorder)."""
import ctypes
import struct

import pytest
import torch

import gemm_w4a16_group_gb300 as w4

OK, INVALID, MISALIGNED = 0, -1, -2
FAKE = 1 << 20  # an aligned non-null address; never dereferenced on these paths
BF, E4 = torch.bfloat16, torch.float8_e4m3fn
FIELDS = ("k", "v", "k_scale", "v_scale", "k_layer", "k_page", "k_head", "k_row", "v_layer", "v_page", "v_head", "v_row",
          "layers", "pages", "kv_heads", "page_rows", "dim", "type")


@pytest.fixture(scope="module")
def L():
    return w4.lib()


def cache(**changes):
    d = dict(zip(FIELDS, (FAKE, FAKE, 0, 0, 0, 4096, 2048, 128, 0, 4096, 2048, 128, 1, 4, 2, 16, 128, 0)))
    d.update(changes)
    return struct.pack("=4Q8q6i", *(d[f] for f in FIELDS))


def append(L, c=None, k=FAKE, v=FAKE, strides=(256, 128, 256, 128), table=FAKE, width=4, lengths=FAKE, starts=FAKE, rows=2,
           tokens=3):
    return L.w4a16_kv_append(k, v, *strides, cache() if c is None else c, table, width, lengths, starts, rows, tokens, None)


def attention(L, c=None, q=FAKE, strides=(512, 128), table=FAKE, width=4, lengths=FAKE, starts=FAKE, mask=FAKE, rows=2,
              tokens=3, heads=4, max_tree=8, scale=0.1, out=FAKE, ws=FAKE):
    return L.w4a16_tree_attention(q, *strides, cache() if c is None else c, table, width, lengths, starts, mask, rows, tokens,
                                  heads, max_tree, scale, out, ws, None)


@pytest.mark.parametrize("changes", [
    dict(k=0), dict(v=0), dict(type=2), dict(type=-1), dict(layers=0), dict(pages=0), dict(kv_heads=0), dict(kv_heads=1025),
    dict(dim=96), dict(dim=0), dict(dim=512), dict(page_rows=8), dict(page_rows=24), dict(page_rows=512), dict(k_row=64),
    dict(k_page=-4096), dict(k_page=0), dict(v_head=128), dict(k_page=2048), dict(v_page=4000), dict(k_scale=FAKE),
    dict(type=1), dict(type=1, k_scale=FAKE), dict(layers=2, k_layer=0, v_layer=0)])
def test_caches_that_cannot_be(L, changes):
    """Null bases, unknown types, sizes out of range, strides that fold one element onto another, scales without
    8 bits and 8 bits without scales, more than one layer where values are computed."""
    assert append(L, cache(**changes)) == INVALID
    assert attention(L, cache(**changes)) == INVALID


def test_caches_that_may_be_moved(L):
    """Calls that only move rows take layers, and 8-bit caches without scales; never overlapping ones."""
    def compact(c, out=FAKE + 64):
        return L.w4a16_kv_compact(c, FAKE, 4, FAKE, FAKE, FAKE, 2, 8, out, None)

    for bad in (dict(layers=2, k_layer=8192, v_layer=16384), dict(layers=2, k_layer=16384, v_layer=0), dict(page_rows=12)):
        assert compact(cache(**bad)) == INVALID
    assert compact(cache(k=FAKE + 8)) == MISALIGNED
    assert compact(cache(type=1, k_row=136, k_head=4096, k_page=8192)) == MISALIGNED  # rows of 136 bytes
    assert compact(cache(), out=FAKE) == INVALID        # lengths_out is lengths
    assert compact(cache(), out=FAKE + 4) == INVALID    # ... or overlaps them
    assert compact(None) == INVALID


def test_strides_and_alignment(L):
    assert append(L, cache(k_row=132, k_head=4096, k_page=8192)) == MISALIGNED
    assert append(L, cache(v=FAKE + 2)) == MISALIGNED
    assert append(L, k=FAKE + 8) == MISALIGNED
    assert append(L, strides=(252, 128, 256, 128)) == MISALIGNED
    assert append(L, strides=(256, 128, -256, 128)) == INVALID
    assert append(L, table=FAKE + 2) == MISALIGNED
    assert attention(L, q=FAKE + 4) == MISALIGNED
    assert attention(L, strides=(512, 129)) == MISALIGNED
    assert attention(L, strides=(-512, 128)) == INVALID
    assert attention(L, mask=FAKE + 4) == MISALIGNED
    assert attention(L, out=FAKE + 8) == MISALIGNED
    assert attention(L, ws=FAKE + 128) == MISALIGNED


def test_null_and_sizes(L):
    for name in ("k", "v", "table", "lengths", "starts"):
        assert append(L, **{name: None}) == INVALID
    for name in ("q", "table", "lengths", "starts", "out", "ws"):
        assert attention(L, **{name: None}) == INVALID
    for bad in (dict(rows=0), dict(rows=65536), dict(tokens=0), dict(tokens=-1), dict(width=0), dict(tokens=1 << 27)):
        assert append(L, **bad) == INVALID and attention(L, **bad) == INVALID
    for bad in (dict(heads=3), dict(heads=0), dict(heads=65536), dict(max_tree=0), dict(max_tree=65), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(tokens=1 << 26, heads=64)):
        assert attention(L, **bad) == INVALID
    accept = lambda *a: L.w4a16_tree_accept(*a, None)  # noqa: E731
    good = [FAKE, FAKE, None, FAKE, 2, 3, 8, FAKE, FAKE, FAKE]
    for i, bad in ((0, None), (1, None), (3, None), (4, 0), (4, 65536), (5, 0), (6, 0), (6, 65), (7, None), (8, None), (9, None)):
        assert accept(*good[:i], bad, *good[i + 1:]) == INVALID
    assert accept(*good[:9], FAKE + 4) == MISALIGNED
    free = [FAKE, 4, 2, FAKE, FAKE, 8, FAKE, 2]
    for i, bad in ((0, None), (1, 0), (2, 0), (3, None), (4, None), (5, 0), (6, None), (7, 0), (7, 4097)):
        assert L.w4a16_kv_free(*free[:i], bad, *free[i + 1:], None) == INVALID
    fork = [cache(), FAKE, 4, 2, FAKE, FAKE, FAKE, FAKE, 1, FAKE]
    for i, bad in ((0, None), (1, None), (2, 0), (3, 0), (4, None), (5, None), (6, None), (7, None), (8, 0), (8, 4097), (9, None)):
        assert L.w4a16_kv_fork(*fork[:i], bad, *fork[i + 1:], None) == INVALID
    reserve = [FAKE, 4, 2, FAKE, 8, 16, FAKE, FAKE, 1, FAKE]
    for i, bad in ((0, None), (1, 0), (2, 0), (3, None), (4, 0), (5, 20), (5, 0), (6, None), (7, None), (8, 0), (8, 4097), (9, None)):
        assert L.w4a16_kv_reserve(*reserve[:i], bad, *reserve[i + 1:], None) == INVALID
    assert L.w4a16_kv_reserve(*reserve[:9], FAKE + 2, None) == MISALIGNED


def test_workspace_sizes(L):
    assert w4.tree_attention_workspace_bytes(8, 2, 128, 1) % 256 == 0
    assert w4.tree_attention_workspace_bytes(8, 2, 128, 64) >= w4.tree_attention_workspace_bytes(8, 2, 128, 1) > 0
    for bad in ((8, 3, 128, 1), (8, 2, 100, 1), (8, 2, 128, 0), (8, 2, 128, 65), (0, 1, 64, 1), (2, 4, 64, 1)):
        assert w4.tree_attention_workspace_bytes(*bad) == 0
    assert "index" in w4.strerror(-6)


class FakeLib:
    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name.endswith("_bytes") or name in ("w4a16_strerror", "w4a16_last_cuda_error"):
            return getattr(self.real, name)

        def record(*args):
            self.calls.append((name, args))
            return 0

        return record


@pytest.fixture
def fake(monkeypatch):
    f = FakeLib(w4.lib())
    monkeypatch.setattr(w4, "lib", lambda auto_build=True: f)
    monkeypatch.setattr(w4, "_is_device_tensor", lambda t: True)
    monkeypatch.setattr(w4, "_stream", lambda stream, device=None: ctypes.c_void_p(0))
    monkeypatch.setattr(w4, "_workspace", lambda need, like, dev, stream, handle: torch.empty(need, dtype=torch.uint8))
    monkeypatch.setattr(w4, "_small_out", lambda shape, dtype, like, dev, stream, handle: torch.empty(shape, dtype=dtype))
    return f


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


@pytest.fixture
def step():
    """Good arguments of every call, by name."""
    d = dict(q=torch.zeros(5, 8, 64, dtype=BF), k=torch.zeros(5, 2, 64, dtype=BF), v=torch.zeros(5, 2, 64, dtype=BF),
             k_cache=torch.zeros(6, 2, 16, 64, dtype=BF), v_cache=torch.zeros(6, 2, 16, 64, dtype=BF), page_table=i32(3, 2),
             lengths=i32(3), starts=i32(4), mask=torch.zeros(5, dtype=torch.int64), refs=i32(6), rows=i32(2), want=i32(2),
             src=i32(2), dst=i32(2), target=torch.zeros(5, dtype=torch.int64), draft=torch.zeros(5, dtype=torch.int64),
             path=i32(3, 4), count=i32(3))
    return d


CALLS = {
    "kv_append": ("k", "v", "k_cache", "v_cache", "page_table", "lengths", "starts"),
    "tree_attention": ("q", "k_cache", "v_cache", "page_table", "lengths", "starts", "mask", 4),
    "tree_accept": ("target", "draft", "mask", "starts", 4),
    "kv_compact": ("k_cache", "v_cache", "page_table", "lengths", "path", "count"),
    "kv_free": ("page_table", "lengths", "refs", "rows"),
    "kv_fork": ("k_cache", "v_cache", "page_table", "lengths", "refs", "src", "dst"),
    "kv_reserve": ("page_table", "refs", "rows", "want", 16),
}


def call(name, step, **kw):
    return getattr(w4, name)(*(step[a] if isinstance(a, str) else a for a in CALLS[name]), **kw)


@pytest.mark.parametrize("name", CALLS)
def test_good_arguments_reach_the_entry_point(fake, step, name):
    call(name, step)
    assert [c[0] for c in fake.calls] == ["w4a16_" + name]


@pytest.mark.parametrize("name", CALLS)
def test_every_tensor_is_checked(fake, step, name):
    """A wrong type, a wrong size and a gap in the memory of any argument are refused, and nothing is called."""
    for arg in CALLS[name]:
        if not isinstance(arg, str):
            continue
        t = step[arg]
        wrong = t.to(torch.float32) if t.dtype != torch.float32 else t.to(torch.float64)
        with pytest.raises((TypeError, ValueError)):
            call(name, {**step, arg: wrong})
        # (the others set the call's sizes, or are checked against one another below)
        if arg in ("mask", "lengths", "draft", "count") or (arg == "starts" and name != "tree_accept"):
            with pytest.raises(ValueError):
                call(name, {**step, arg: torch.cat([t, t])})
        gap = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)[..., ::2]
        with pytest.raises(ValueError):
            call(name, {**step, arg: gap})
    assert not fake.calls


def test_shapes_that_do_not_fit(fake, step):
    for name, changes in (
            ("kv_append", dict(k=torch.zeros(5, 3, 64, dtype=BF))), ("kv_append", dict(v=torch.zeros(4, 2, 64, dtype=BF))),
            ("kv_append", dict(k=torch.zeros(5, 128, dtype=BF))), ("kv_append", dict(k=torch.zeros(5, 2, 32, dtype=BF))),
            ("kv_append", dict(k_cache=torch.zeros(1, 6, 2, 16, 64, dtype=BF))),
            ("kv_append", dict(v_cache=torch.zeros(6, 2, 32, 64, dtype=BF))),
            ("tree_attention", dict(q=torch.zeros(5, 8, 128, dtype=BF))), ("tree_attention", dict(lengths=i32(2))),
            ("tree_attention", dict(page_table=i32(6))), ("kv_compact", dict(path=i32(12))),
            ("kv_compact", dict(path=i32(2, 4))), ("kv_fork", dict(dst=i32(3))), ("kv_fork", dict(refs=i32(5))),
            ("kv_reserve", dict(want=i32(1)))):
        with pytest.raises(ValueError):
            call(name, {**step, **changes})
    with pytest.raises(w4.W4A16Error, match="heads=7"):
        call("tree_attention", {**step, "q": torch.zeros(5, 7, 64, dtype=BF)})
    with pytest.raises(ValueError, match="workspace"):
        call("tree_attention", step, workspace=torch.zeros(1000, dtype=torch.uint8))
    with pytest.raises(ValueError, match="out"):
        call("tree_attention", step, out=torch.zeros(5, 8, 32, dtype=BF))
    assert not fake.calls


def test_eight_bit_caches_need_their_scales(fake, step):
    e = {**step, "k_cache": torch.zeros(6, 2, 16, 64).to(E4), "v_cache": torch.zeros(6, 2, 16, 64).to(E4)}
    one = torch.ones(2)
    for name in ("kv_append", "tree_attention"):
        with pytest.raises(ValueError, match="scale"):
            call(name, e)
        with pytest.raises(ValueError, match="v_scale"):
            call(name, e, k_scale=one, v_scale=torch.ones(3))
        with pytest.raises(ValueError, match="belong"):
            call(name, step, k_scale=one, v_scale=one)
        call(name, e, k_scale=one, v_scale=one)
    with pytest.raises(TypeError):
        call("kv_append", {**step, "v_cache": e["v_cache"]}, k_scale=one, v_scale=one)
    call("kv_compact", e)
    call("kv_fork", e)
    assert [c[0] for c in fake.calls] == ["w4a16_kv_append", "w4a16_tree_attention", "w4a16_kv_compact", "w4a16_kv_fork"]


def test_strides_reach_the_entry_point(fake, step):
    """Views of a fused product and of a cache whose memory runs [pages, rows, heads, dim]."""
    fused = torch.zeros(5, 12, 64, dtype=BF)
    nhd = torch.zeros(6, 16, 2, 64, dtype=BF).transpose(1, 2)
    call("tree_attention", {**step, "q": fused[:, :8], "k_cache": nhd})
    a = fake.calls[-1][1]
    assert a[0] == fused.data_ptr() and a[1:3] == (12 * 64, 64)
    got = dict(zip(FIELDS, struct.unpack("=4Q8q6i", a[3])))
    assert (got["k_page"], got["k_head"], got["k_row"]) == (2048, 64, 128)
    assert (got["v_page"], got["v_head"], got["v_row"]) == (2048, 1024, 64)
    assert (got["layers"], got["pages"], got["kv_heads"], got["page_rows"], got["dim"], got["type"]) == (1, 6, 2, 16, 64, 0)
    layers = torch.zeros(4, 6, 2, 16, 64, dtype=BF)
    call("kv_compact", {**step, "k_cache": layers, "v_cache": layers})
    got = dict(zip(FIELDS, struct.unpack("=4Q8q6i", fake.calls[-1][1][0])))
    assert got["layers"] == 4 and got["k_layer"] == 6 * 2048


def test_cpu_tensors_are_refused(step):
    for name in CALLS:
        with pytest.raises(ValueError, match="CUDA"):
            call(name, step)
