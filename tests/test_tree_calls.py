"""Host side of the tree-speculation calls, on the CPU: strides of single
tokens, and sizes of workspaces."""

import types

import pytest
import torch

from paged_kv_cache_254_gb300 import _lib, ops


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
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    sizes = []
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: sizes.append(a[0]) or empty(*a))
    for mb, want in ((0, 0), (9, 4096), (0, 4096), (9, 4096)):
        ops._tree_workspace(0, _lib.PaShape(2, 8, 2, 128, 16, 64, mb, _lib.PA_BF16), 8)
        assert sizes[-1] == want
