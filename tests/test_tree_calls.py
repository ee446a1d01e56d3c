"""Host side of the tree-speculation calls, on the CPU: strides of single
tokens, sizes of workspaces and who uses one, operands that overlap, and streams
of another device."""

import contextlib
import ctypes
import threading
import types

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from paged_kv_cache_254_gb300 import _build, _lib, ops
from tests.test_abi import FAKE, NULL, shape


def strided_views(T, H, d, device="cpu"):
    """[T, H, d] views whose heads are not contiguous within a token."""
    qkv = torch.zeros(T, H, 3, d, dtype=torch.bfloat16, device=device)
    wide = torch.zeros(T, H, 2 * d, dtype=torch.bfloat16, device=device)
    return {"interleaved": qkv[:, :, 1], "expanded": qkv[:, :1, 0].expand(T, H, d), "sliced": wide[:, :, ::2],
            "half": wide[:, :, :d], "transposed": torch.zeros(T, d, H, dtype=torch.bfloat16, device=device).transpose(1, 2)}


@pytest.mark.parametrize("T", [1, 2, 5])
@pytest.mark.parametrize("view", ["interleaved", "expanded", "sliced", "half", "transposed"])
def test_heads_must_be_contiguous_whatever_the_token_count(T, view):
    t = strided_views(T, 4, 16)[view]
    with pytest.raises(ValueError, match="contiguous"):
        ops._token_rows("q", t, torch.bfloat16, (T, 4, 16), -1)


def test_token_strides_that_are_fine():
    rows = torch.zeros(5, 7 * 16, dtype=torch.bfloat16)
    q = rows[:, :64].unflatten(1, (4, 16))
    assert ops._token_rows("q", q, torch.bfloat16, (5, 4, 16), -1) == 112
    assert ops._token_rows("q", q[:1], torch.bfloat16, (1, 4, 16), -1) == 64
    assert ops._token_rows("q", q[:1].as_strided((1, 4, 16), (1, 16, 1)), torch.bfloat16, (1, 4, 16), -1) == 64
    assert ops._token_rows("q", q[:0], torch.bfloat16, (0, 4, 16), -1) == 64
    one_head = rows.unflatten(1, (7, 16))[:, 3:4]
    assert ops._token_rows("k", one_head, torch.bfloat16, (5, 1, 16), -1) == 112


# ---------------------------------------------------------------- workspaces
def test_a_refused_shape_leaves_no_size_behind(monkeypatch):
    # the library answers 0 for a shape that it refuses; a valid one that differs from it in a field
    # that the size does not depend on still gets its own
    fake = types.SimpleNamespace(pa_decode_tree_workspace_bytes=lambda s, p: 4096 if s.max_blocks_per_seq > 0 else 0)
    monkeypatch.setattr(_lib, "load", lambda: fake)
    monkeypatch.setattr(ops, "_call", lambda fn, dev, *a: fn(*a))
    monkeypatch.setattr(ops, "_tree_bytes", {})
    for mb, want in ((0, 0), (9, 4096), (0, 4096), (9, 4096)):
        assert ops._tree_workspace_bytes(0, _lib.PaShape(2, 8, 2, 128, 16, 64, mb, _lib.PA_BF16), 8) == want


class FakeLibrary:
    """Stands for libpa: sizes are 1000 bytes, and a call waits until another is inside as well.  ``used`` are the
    workspaces that the calls were given."""

    def __init__(self, buffers):
        self.buffers, self.used, self.inside = buffers, [], threading.Barrier(2)

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *a: 1000
        return self.call

    def call(self, *args):
        values = {getattr(a, "value", a) for a in args if isinstance(a, (int, ctypes.c_void_p, ctypes.c_size_t))}
        self.used.append(next(b for b in self.buffers if b.data_ptr() in values))
        assert all(w is not self.used[-1] for w in ops._sp_cache.values())   # not to be found by a third call
        self.inside.wait(timeout=30)
        return 0


@pytest.fixture
def fake_library(monkeypatch):
    buffers, empty, zeros = [], torch.empty, torch.zeros

    def on_the_host(make):
        def f(*size, dtype=None, device=None):
            t = make(*size, dtype=dtype)
            if dtype == torch.uint8:
                buffers.append(t)
            return t
        return f

    lib = FakeLibrary(buffers)
    monkeypatch.setattr(_lib, "load", lambda: lib)
    monkeypatch.setattr(torch, "empty", on_the_host(empty))
    monkeypatch.setattr(torch, "zeros", on_the_host(zeros))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=7))
    monkeypatch.setattr(torch.cuda, "device", type("Here", (contextlib.nullcontext,), {}))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    for name, value in (("_need_cuda", lambda *a: None), ("_arg", lambda *a: None), ("_index", lambda *a: 0),
                        ("_raw_stream", lambda d: 7), ("_call", lambda fn, dev, *a: fn(*a)), ("_sp_cache", {}),
                        ("_fast", types.SimpleNamespace(decode_tree=lambda *a: NotImplemented))):
        monkeypatch.setattr(ops, name, value)
    return lib


def host_call(name):
    """A call of one of the attention entry points with tensors of the right shapes."""
    N, Hq, Hkv, d, B = 2, 4, 2, 128, 16
    half = lambda *s: torch.ones(*s, dtype=torch.float16)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)
    q, k, v, table, ctx = half(N, Hq, d), half(4, Hkv, B, d), half(4, Hkv, B, d), i32([0, 1], [2, 3]), i32(5, 6)
    start, u8 = i32(0, 1, 2), lambda *s: torch.ones(s, dtype=torch.uint8)
    return {"decode": lambda: ops.pa_decode(q, k, v, table, ctx, 0.1),
            "multi": lambda: ops.pa_decode_multi(q, k, v, table, ctx, start, 0.1, max_q_len=1),
            "shared_prefix": lambda: ops.pa_decode_shared_prefix(q, k, v, table, ctx, start[:2], i32(0), 0.1),
            "fp8": lambda: ops.pa_decode_fp8(q, u8(4, Hkv, 2, B, d), table, ctx, 0.1, 1.0, 1.0),
            "int4": lambda: ops.pa_decode_int4(q, u8(4, Hkv, B, d + 8), table, ctx, 0.1),
            "tree": lambda: ops.pa_decode_tree(q, k, v, table, ctx, start, torch.ones(2, dtype=torch.int64), 0.1, 1)}[name]


@pytest.mark.parametrize("one", ["decode", "multi", "shared_prefix", "fp8", "int4", "tree"])
@pytest.mark.parametrize("other", ["tree", "multi"])
def test_two_threads_on_one_stream_do_not_share_a_workspace(fake_library, one, other):
    # a call is several launches: another thread's may come between them, on the same stream
    for round_ in range(2):                               # the second time one is kept already
        fake_library.used.clear()
        failed = []

        def run(call):
            try:
                call()
            except Exception as e:                        # a broken barrier: the other call failed
                failed.append(e)

        threads = [threading.Thread(target=run, args=(host_call(n),)) for n in (one, other)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not failed, failed
        a, b = fake_library.used
        assert a is not b
        assert len(ops._sp_cache) in (1, 2) and all(w is a or w is b for w in ops._sp_cache.values())   # one a key


@pytest.mark.parametrize("capturing", [False, True])
def test_a_workspace_belongs_to_the_stream_of_the_call(monkeypatch, capturing):
    # freed memory is used again in the order of the stream that it was allocated on: a captured call's, which is freed
    # at once, and one that a larger one replaces
    current, made = [None], []

    @contextlib.contextmanager
    def on(stream):
        before, current[0] = current[0], stream or current[0]
        yield
        current[0] = before

    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: made.append(current[0]) or empty(*a))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing and current[0] == "side")
    monkeypatch.setattr(ops, "_sp_cache", {})
    for need in (10, 1 << 21):
        ops._lend(None, 0, 5, need, lambda ws: ws, "side")
    assert made == ["side", "side"] and len(ops._sp_cache) == (0 if capturing else 1)
    ops._lend(None, 0, 0, 10, lambda ws: ws)
    assert made[2:] == [None]


# ---------------------------------------------------------------- overlapping operands
@pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is not refused would start a kernel")
@pytest.mark.parametrize("tokens", [1 << 20, 1 << 29, 1 << 30, (1 << 31) - 1])
def test_rotated_queries_over_other_operands_at_any_token_count(tokens):
    _build.build()
    at = lambda rows: ctypes.c_void_p(FAKE.value + 32 * rows)          # a token's row is 32 bytes

    def status(q, k, v, out):
        rope = _lib.PaRope(None, 0, 0, 1.0, 1e-6, None, None)
        return _lib.load().pa_rope_append_kv(shape(num_q_heads=1, num_kv_heads=1, head_dim=16), rope, tokens, q, 16, k, 16,
                                             v, 16, FAKE, FAKE, out, FAKE, at(1), NULL, NULL)

    n = tokens
    assert status(at(0), at(2 * n), at(3 * n), at(n)) == 3              # side by side: fine (no GPU here)
    assert status(at(0), at(2 * n), at(3 * n), at(n - 1)) == 1          # into q's last row
    assert status(at(n), at(2 * n), at(3 * n), at(1)) == 1              # q_out's last row into q's first
    assert status(at(0), at(2 * n - 1), at(3 * n), at(n)) == 1          # into the keys
    assert status(at(0), at(3 * n), at(2 * n - 1), at(n)) == 1          # into the values


# ---------------------------------------------------------------- streams
def test_a_stream_of_another_device_is_refused(monkeypatch):
    # with it current the call would go to the stream that is current on the tensors' device
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    with FakeTensorMode():
        here = [torch.empty(2, device="cuda:0"), None, torch.empty(3, dtype=torch.int32, device="cuda:0"), 0.5]
    made = []
    with pytest.raises(ValueError, match="stream"):
        ops._on_stream(types.SimpleNamespace(device=torch.device("cuda", 1)), lambda *a: made.append(a), *here)
    assert not made
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: made.append(t))
    ops._on_stream(types.SimpleNamespace(device=torch.device("cuda", 0)), lambda *a: made.append(a), *here)
    assert len(made) == 3
