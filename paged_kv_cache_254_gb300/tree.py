"""Ancestor masks of drafted trees, as ``pa_decode_tree`` and
``pa_tree_verify`` take them."""

from __future__ import annotations

import torch

MAX_NODES = 64


def tree_masks(parents: torch.Tensor, q_start: torch.Tensor) -> torch.Tensor:
    """int64 [T]: bit j of entry q_start[b] + i is set when node j of tree b is
    node i or one of its ancestors.

    ``parents`` [T] (any integer type) holds each node's parent as an index
    within its own tree, lower than the node's, or -1 for a root; ``q_start``
    [N + 1] each tree's first entry.  Works where its inputs live; the checks
    read one value back."""
    if parents.dim() != 1 or q_start.dim() != 1 or q_start.numel() < 1:
        raise ValueError("parents [T], q_start [N + 1]")
    T, dev = parents.shape[0], parents.device
    starts = q_start.to(device=dev, dtype=torch.int64)
    sizes = starts.diff()
    if bool((starts[0] != 0) | (starts[-1] != T) | (sizes < 0).any() | (sizes > MAX_NODES).any()):
        raise ValueError(f"q_start must rise from 0 to {T} in steps of at most {MAX_NODES}")
    first = torch.repeat_interleave(starts[:-1], sizes)
    node = torch.arange(T, device=dev) - first
    up = parents.to(torch.int64)
    if bool(((up >= node) | (up < -1)).any()):
        raise ValueError("a node's parent must be a lower node of its tree, or -1")
    mask = torch.ones_like(node) << node
    # a round adds the ways of the ancestors reached so far: 1, 2, 4, ... steps up
    up = torch.where(up >= 0, up + first, -1)
    for _ in range(6):
        has = up >= 0
        at = up.clamp(min=0)
        if T:
            mask = torch.where(has, mask | mask[at], mask)
            up = torch.where(has, up[at], -1)
    return mask
