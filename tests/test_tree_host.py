"""Host side of the tree-speculation operators: refusals that answer without
touching a GPU, ancestor masks, rotary frequencies, and cutting sequences back."""

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle.tree import masks_ref
from paged_kv_cache_254_gb300 import BlockManager, _build, _lib, ops, rope_inv_freq, tree_masks
from tests.test_abi import BUF_BYTES, FAKE, NULL, shape


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _lib.load()


def off(k):
    return ctypes.c_void_p(FAKE.value + k)


@pytest.mark.parametrize("kw,status", [
    (dict(max_nodes=0), 1), (dict(max_nodes=65), 1), (dict(total=-1), 1), (dict(scale=float("inf")), 1),
    (dict(q=NULL), 1), (dict(masks=NULL), 1), (dict(q_start=NULL), 1), (dict(q=off(2)), 1), (dict(masks=off(4)), 1),
    (dict(sh=dict(head_dim=96)), 2), (dict(sh=dict(block_size=8)), 2), (dict(sh=dict(num_q_heads=6)), 2),
    (dict(sh=dict(dtype=2)), 1), (dict(sh=dict(num_seqs=-1)), 1), (dict(sh=dict(num_seqs=0)), 0),
    (dict(out=FAKE), 1), (dict(out=ctypes.c_void_p(FAKE.value + 2048)), 1),      # over q
])
def test_decode_tree_checks(lib, kw, status):
    sh = shape(**{**dict(head_dim=128, num_q_heads=8, num_kv_heads=2), **kw.pop("sh", {})})
    a = {**dict(max_nodes=4, total=8, q=FAKE, q_start=FAKE, masks=FAKE, scale=0.1), **kw}
    assert lib.pa_decode_tree(sh, a["max_nodes"], a["total"], a["q"], a["q_start"], a["masks"], FAKE, FAKE, FAKE,
                              FAKE, a["scale"], a.get("out", off(1 << 16)), FAKE, BUF_BYTES, NULL, NULL) == status


def test_tree_workspace_of_bad_shapes_is_zero(lib):
    assert lib.pa_decode_tree_workspace_bytes(shape(head_dim=80), 4) == 0
    assert lib.pa_decode_tree_workspace_bytes(shape(), 65) == 0
    assert lib.pa_decode_tree_workspace_bytes(None, 4) == 0


def test_verify_checks(lib):
    def v(n=2, p=8, t=4, qs=FAKE, masks=FAKE, draft=FAKE, path=FAKE, nxt=FAKE):
        return lib.pa_tree_verify(n, p, t, qs, masks, draft, FAKE, FAKE, path, FAKE, nxt, FAKE, NULL, NULL)
    assert v(n=-1) == 1 and v(p=0) == 1 and v(p=65) == 1 and v(t=-1) == 1
    assert v(n=0) == 0
    assert v(qs=NULL) == 1 and v(path=NULL) == 1 and v(masks=NULL) == 1 and v(draft=NULL) == 1
    assert v(masks=off(4)) == 1 and v(nxt=off(4)) == 1


def test_keep_checks(lib):
    def k(p=8, path=FAKE, k_pool=FAKE, v_pool=off(1 << 16), table=FAKE, **sh):
        return lib.pa_keep_kv(shape(**sh), p, path, FAKE, table, FAKE, k_pool, v_pool, NULL, NULL)
    assert k(v_pool=FAKE) == 1                            # one pool for both
    assert k(p=0) == 1 and k(p=65) == 1 and k(path=NULL) == 1 and k(table=NULL) == 1 and k(k_pool=off(8)) == 1
    assert k(dtype=2) == 1 and k(num_seqs=-1) == 1 and k(max_blocks_per_seq=0) == 1
    assert k(num_blocks=1 << 27) == 2
    assert k(num_seqs=0) == 0
    assert lib.pa_keep_kv(None, 8, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, NULL, NULL) == 1


def test_rope_append_checks(lib):
    def r(n=4, q=FAKE, k=off(1 << 17), v=off(3 << 16), qs=512, ks=512, vs=512, out=off(1 << 16), v_pool=off(1 << 19), rot=64, freq=FAKE, scale=1.0, eps=1e-6, qw=None,
          rope=True, pos=FAKE, **sh):
        rp = _lib.PaRope(freq.value, rot, 0, scale, eps, qw, None) if rope else None
        return lib.pa_rope_append_kv(shape(**sh), rp, n, q, qs, k, ks, v, vs, pos, FAKE, out, FAKE, v_pool, NULL, NULL)
    assert r(n=0) == 0
    assert r(rope=False) == 1 and r(n=-1) == 1 and r(q=NULL) == 1 and r(out=NULL) == 1 and r(pos=NULL) == 1
    assert r(freq=NULL) == 1 and r(rot=80) == 1 and r(rot=-16) == 1
    assert r(rot=24) == 2 and r(head_dim=72, qs=576, ks=576, vs=576) == 2 and r(head_dim=272, qs=4096) == 2
    assert r(qs=504) == 1 and r(ks=504) == 1 and r(vs=516) == 1          # shorter than a row; not 16 bytes
    assert r(scale=float("nan")) == 1 and r(eps=-1.0) == 1 and r(eps=float("inf")) == 1
    assert r(qw=FAKE.value + 8) == 1 and r(q=off(8)) == 1 and r(dtype=3) == 1 and r(num_q_heads=0) == 1
    assert r(v_pool=FAKE) == 1                            # one pool for both
    assert r(k=off((1 << 16) + 512)) == 1 and r(v=off((1 << 16) - 512)) == 1   # q_out over the keys, the values
    # q_out over a shifted or strided q
    assert r(out=off(16)) == 1 and r(out=FAKE, qs=520) == 1 and r(q=off(1024), out=off(512)) == 1


def test_python_calls_refuse_host_tensors():
    x = torch.zeros(2, 2, 64, dtype=torch.float16)
    pool = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ops.pa_decode_tree(x, pool, pool, i[None], i, i, i.long(), 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        ops.pa_tree_verify(i.long(), i.long(), i.long(), i, i)
    with pytest.raises(ValueError, match="CUDA"):
        ops.pa_keep_kv(i[None], i, i, i[None], pool, pool)
    with pytest.raises(ValueError, match="CUDA"):
        ops.pa_rope_append_kv(x, x, x, i, i.long(), pool, pool, None)


# ---------------------------------------------------------------- ancestor masks
@pytest.mark.parametrize("sizes", [[1], [64, 0, 5], [7, 64, 1, 33], []])
def test_tree_masks_match_the_walk(sizes):
    r = np.random.default_rng(sum(sizes))
    trees = [[-1] + [int(r.integers(-1, i)) for i in range(1, n)] if n else [] for n in sizes]
    want = [m - (1 << 64) if m >> 63 else m for t in trees for m in masks_ref(t)]
    flat = torch.tensor([p for t in trees for p in t], dtype=torch.int32)
    got = tree_masks(flat, torch.tensor(np.cumsum([0] + sizes), dtype=torch.int32))
    assert got.dtype == torch.int64 and got.tolist() == want


def test_tree_masks_of_a_64_node_chain():
    got = tree_masks(torch.arange(-1, 63), torch.tensor([0, 64]))
    assert got.tolist() == [(1 << (i + 1)) - 1 for i in range(63)] + [-1]


@pytest.mark.parametrize("parents,starts", [
    ([0], [0, 1]), ([-1, 1], [0, 2]), ([-2], [0, 1]), ([-1, 0], [0, 1]), ([-1, 0], [1, 2]), ([-1, 0], [0, 3, 2]),
    ([-1] * 65, [0, 65]),
])
def test_tree_masks_refusals(parents, starts):
    with pytest.raises(ValueError):
        tree_masks(torch.tensor(parents), torch.tensor(starts))


# ---------------------------------------------------------------- frequencies
def test_plain_and_linear_frequencies():
    f, s = rope_inv_freq(8, base=10000.0, device="cpu")
    assert s == 1.0 and f.dtype == torch.float32
    np.testing.assert_allclose(f.numpy(), [1.0, 0.1, 0.01, 0.001], rtol=1e-7)
    g, _ = rope_inv_freq(8, scaling="linear", factor=4.0, device="cpu")
    np.testing.assert_allclose(g.numpy(), f.numpy() / 4, rtol=1e-7)


def test_ntk_keeps_the_fastest_and_stretches_the_slowest():
    f, _ = rope_inv_freq(64, device="cpu")
    g, s = rope_inv_freq(64, scaling="ntk", factor=8.0, device="cpu")
    assert s == 1.0 and g[0] == f[0]
    assert math.isclose(float(f[-1] / g[-1]), 8.0, rel_tol=1e-5)


def test_yarn_blends_by_the_number_of_turns():
    f, _ = rope_inv_freq(64, device="cpu")
    g, s = rope_inv_freq(64, scaling="yarn", factor=16.0, original_len=4096, device="cpu")
    assert math.isclose(s, 0.1 * math.log(16.0) + 1)
    turns = 4096 * f.double() / (2 * math.pi)
    assert torch.equal(g[turns >= 32], f[turns >= 32]) and (turns >= 32).any()
    np.testing.assert_allclose(g[turns <= 1].numpy(), f[turns <= 1].numpy() / 16, rtol=1e-6)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and ((g < f) & (g > f / 16))[mid].all()


@pytest.mark.parametrize("kw", [dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, base=0.0),
                                dict(rotary_dim=8, factor=0.5), dict(rotary_dim=8, scaling="other"),
                                dict(rotary_dim=8, scaling="yarn", factor=2.0)])
def test_frequency_refusals(kw):
    with pytest.raises(ValueError):
        rope_inv_freq(**kw, device="cpu")


# ---------------------------------------------------------------- cutting sequences back
def test_truncate_returns_whole_blocks():
    bm = BlockManager(8, 4)
    bm.add_sequence("a", 6)
    bm.append_slots([("a", 9)])                       # 15 tokens, 4 blocks
    table = bm.table("a")
    bm.truncate("a", 8)
    assert bm.table("a") == table[:2] and bm.length("a") == 8 and bm.num_free == 6
    assert bm.append_slots([("a", 1)]).tolist() == [table[3] * 4]   # the block freed last comes first
    bm.truncate("a", 0)
    assert bm.table("a") == [] and bm.num_free == 8


def test_truncate_leaves_shared_blocks_to_their_other_owner():
    bm = BlockManager(8, 4)
    bm.add_sequence("a", 8)
    bm.fork("a", "b")
    blocks = bm.table("a")
    bm.truncate("b", 3)
    assert bm.table("a") == blocks and bm.refcount(blocks[1]) == 1 and bm.refcount(blocks[0]) == 2
    assert bm.num_free == 6
    bm.append_slots([("b", 1)])                       # writes into the shared block: copied first
    assert bm.take_copies().tolist() == [[blocks[0], bm.table("b")[0]]]


def test_truncate_refusals():
    bm = BlockManager(8, 4)
    bm.add_sequence("a", 6)
    for n in (-1, 7):
        with pytest.raises(ValueError):
            bm.truncate("a", n)
    with pytest.raises(KeyError):
        bm.truncate("z", 0)
    bm.fork("a", "b")
    bm.append_slots([("b", 1)])                       # queues a copy into b's second block
    with pytest.raises(RuntimeError):
        bm.truncate("b", 2)
    bm.take_copies()
    bm.truncate("b", 2)
    assert bm.length("b") == 2
