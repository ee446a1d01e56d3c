"""fp64 attention of drafted trees, the accepted path, and keeping its tokens.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

A sequence's last n cached tokens are the nodes of a drafted tree.  A node sees
every token cached before the tree and the nodes that its mask names.  The
accepted path follows, from node 0 on, the child whose token is the one the
target model chose; its tokens then move to consecutive positions.  All three
are written as walks over single tokens."""

from __future__ import annotations

import numpy as np

from .attention import _i64, f64, gather_sequence


def decode_tree_ref(q, k_pool, v_pool, block_tables, context_lens, q_start, masks, scale: float) -> np.ndarray:
    """[T, Hq, d] fp64; a node that sees nothing gives a zero row.  masks:
    Python ints (or int64), bit j = node j.  Only visible keys and values enter
    the sums."""
    tables, lens, starts = _i64(block_tables), _i64(context_lens), _i64(q_start)
    bits = [int(m) & ((1 << 64) - 1) for m in (masks.tolist() if hasattr(masks, "tolist") else masks)]
    q64 = f64(q)
    T, Hq, d = q64.shape
    Hkv, B = k_pool.shape[1], k_pool.shape[2]
    g = Hq // Hkv
    out = np.zeros((T, Hq, d))
    for b in range(len(lens)):
        ctx, r0 = int(lens[b]), int(starts[b])
        n = int(starts[b + 1]) - r0
        base = ctx - n
        if n == 0:
            continue
        for kh in range(Hkv):
            K, V = gather_sequence(k_pool, v_pool, tables[b], ctx, kh, B)
            for i in range(n):
                seen = list(range(base)) + [base + j for j in range(n) if (bits[r0 + i] >> j) & 1]
                if not seen:
                    continue
                for h in range(kh * g, (kh + 1) * g):
                    s = scale * (K[seen] @ q64[r0 + i, h])
                    e = np.exp(s - s.max())
                    out[r0 + i, h] = (e / e.sum()) @ V[seen]
    return out


def masks_ref(parents):
    """Ancestor masks of one tree, by walking up from each node."""
    out = []
    for i in range(len(parents)):
        m, j = 0, i
        while j >= 0:
            m |= 1 << j
            j = int(parents[j])
        out.append(m)
    return out


def verify_ref(parents, draft, target):
    """(accepted nodes, next token) of one tree by walking down: from the
    current node to its lowest child whose token is the target's choice."""
    if len(parents) == 0:
        return [], -1
    path, at = [0], 0
    while True:
        for c in range(at + 1, len(parents)):
            if parents[c] == at and draft[c] == target[at]:
                at = c
                path.append(c)
                break
        else:
            return path, int(target[at])


def keep_ref(k_bits, v_bits, path, q_start, block_tables, context_lens, block_size: int):
    """New (k, v) pools (bit patterns [NB, Hkv, B, d]) with the path's tokens
    moved to consecutive positions; every row is read from before the call."""
    k, v = np.array(k_bits, copy=True), np.array(v_bits, copy=True)
    for b, row in enumerate(np.asarray(path)):
        n = int(q_start[b + 1]) - int(q_start[b])
        base = int(context_lens[b]) - n
        for d, node in enumerate(row):
            if node < 0:
                break
            s, t = base + int(node), base + d
            sb, tb = int(block_tables[b][s // block_size]), int(block_tables[b][t // block_size])
            k[tb, :, t % block_size] = k_bits[sb, :, s % block_size]
            v[tb, :, t % block_size] = v_bits[sb, :, s % block_size]
    return k, v
