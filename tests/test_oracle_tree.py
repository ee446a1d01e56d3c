"""Pins of the tree and rotary oracles to something other than themselves."""

import itertools

import numpy as np
import pytest
import torch

from oracle.attention import decode_multi_ref, decode_ref
from oracle.kv_ops import bits
from oracle.rope import norm_ref, rotate_ref
from oracle.tree import decode_tree_ref, keep_ref, masks_ref, verify_ref


def small(ctx, d=8, Hq=4, Hkv=2, B=4, seed=0):
    r = np.random.default_rng(seed)
    need = [-(-c // B) for c in ctx]
    NB = sum(need) + 2
    ids = r.permutation(NB)
    tables = np.full((len(ctx), max(max(need), 1)), -1)
    at = 0
    for b, k in enumerate(need):
        tables[b, :k] = ids[at:at + k]
        at += k
    return r.normal(size=(NB, Hkv, B, d)), r.normal(size=(NB, Hkv, B, d)), tables, np.array(ctx), r


def test_chain_is_the_causal_chunk():
    kp, vp, tables, ctx, r = small([9, 5, 3])
    n = [4, 5, 1]
    qs = np.cumsum([0] + n)
    q = r.normal(size=(sum(n), 4, 8))
    masks = [m for k in n for m in masks_ref(list(range(-1, k - 1)))]
    np.testing.assert_allclose(decode_tree_ref(q, kp, vp, tables, ctx, qs, masks, 0.3),
                               decode_multi_ref(q, kp, vp, tables, ctx, qs, 0.3), rtol=1e-12, atol=1e-12)


def test_each_branch_is_a_plain_sequence():
    # a node's row equals single-token decode over a cache that holds its way alone
    kp, vp, tables, ctx, r = small([11])
    parents = [-1, 0, 0, 1, 2, 2]
    q = r.normal(size=(6, 4, 8))
    got = decode_tree_ref(q, kp, vp, tables, ctx, [0, 6], masks_ref(parents), 0.4)
    flat_k = [kp[tables[0, t // 4], :, t % 4] for t in range(11)]
    flat_v = [vp[tables[0, t // 4], :, t % 4] for t in range(11)]
    for i in range(6):
        way, j = [], i
        while j >= 0:
            way.append(j)
            j = parents[j]
        keep = list(range(5)) + [5 + j for j in sorted(way)]
        k1 = np.stack([flat_k[t] for t in keep], 1)[None]           # one block as long as the way
        v1 = np.stack([flat_v[t] for t in keep], 1)[None]
        want = decode_ref(q[i:i + 1], k1, v1, [[0]], [len(keep)], 0.4)
        np.testing.assert_allclose(got[i], want[0], rtol=1e-12, atol=1e-12)


def test_empty_row_is_zero_and_unseen_nodes_do_not_matter():
    kp, vp, tables, ctx, r = small([3])
    q = r.normal(size=(3, 4, 8))
    a = decode_tree_ref(q, kp, vp, tables, ctx, [0, 3], [0b001, 0b000, 0b101], 1.0)
    assert (a[1] == 0).all()
    kp[tables[0, 0], :, 1] = np.nan
    vp[tables[0, 0], :, 1] = np.inf
    assert np.array_equal(a, decode_tree_ref(q, kp, vp, tables, ctx, [0, 3], [0b001, 0b000, 0b101], 1.0))


def test_verify_against_every_path():
    # the longest root path whose every step is the lowest matching child
    r = np.random.default_rng(4)
    for _ in range(200):
        n = int(r.integers(1, 8))
        parents = [-1] + [int(r.integers(0, i)) for i in range(1, n)]
        draft, target = r.integers(0, 2, n).tolist(), r.integers(0, 2, n).tolist()
        path, nxt = verify_ref(parents, draft, target)
        best = [0]
        for k in range(1, n + 1):
            for way in itertools.combinations(range(n), k):
                if way[0] == 0 and all(
                        parents[b] == a and draft[b] == target[a] and
                        not any(parents[c] == a and draft[c] == target[a] for c in range(b))
                        for a, b in zip(way, way[1:])):
                    best = max(best, list(way), key=len)
        assert path == best and nxt == target[best[-1]]


def test_keep_moves_rows_of_the_state_before_the_call():
    kp, vp, tables, ctx, r = small([10])
    kb, vb = bits(torch.from_numpy(kp).half()), bits(torch.from_numpy(vp).half())
    k, v = keep_ref(kb, vb, [[0, 1, 3, 4, -1, -1]], [0, 6], tables, ctx, 4)

    def at(x, t):
        return x[tables[0, t // 4], :, t % 4]
    for d, node in enumerate([0, 1, 3, 4]):
        assert np.array_equal(at(k, 4 + d), at(kb, 4 + node))
        assert np.array_equal(at(v, 4 + d), at(vb, 4 + node))
    for t in (0, 1, 2, 3, 8, 9):
        assert np.array_equal(at(k, t), at(kb, t))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_relative_and_keeps_lengths(interleaved):
    r = np.random.default_rng(1)
    f = 10.0 ** -np.arange(4)
    x, y = r.normal(size=(1, 1, 10)), r.normal(size=(1, 1, 10))
    a = rotate_ref(x, [7], f, interleaved)
    assert np.allclose((a ** 2).sum(), (x ** 2).sum())
    assert np.array_equal(a[..., 8:], x[..., 8:])
    one = (rotate_ref(x, [107], f, interleaved) * rotate_ref(y, [100], f, interleaved)).sum()
    two = (a * y).sum()                                # scores depend on the distance alone
    assert np.isclose(one, two)
    # a quarter turn, by hand: (a, b) -> (-b, a)
    q = rotate_ref(np.array([[[1.0, 2.0]]]), [1], [np.pi / 2], interleaved)
    assert np.allclose(q, [[[-2.0, 1.0]]])


def test_norm_by_hand():
    assert np.allclose(norm_ref(np.array([3.0, 4.0]), np.array([1.0, 2.0]), 0.0), [3 / 12.5 ** 0.5, 8 / 12.5 ** 0.5])
