"""A whole run of tree speculation, as a program makes it: the block manager
reserves the tree's slots, the fused call norms, rotates and appends, the tree
is attended to and verified, its accepted tokens are kept, the sequences are cut
back, and the next step decodes over what is left.

The final cache and output are compared with the fp64 oracle on a sequence that
never speculated: the accepted tokens alone, one after the other."""

import numpy as np
import pytest
import torch

from oracle.attention import decode_ref
from oracle.rope import norm_ref, rotate_ref
from oracle.tree import decode_tree_ref, masks_ref, verify_ref
from tests.gpu_util import assert_close, need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def dev(a, t):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", t)


@pytest.mark.parametrize("Hq,Hkv,d,nodes,captured", [(8, 2, 128, 9, False), (16, 2, 64, 40, False), (8, 1, 128, 33, True)])
def test_three_steps_of_speculation(Hq, Hkv, d, nodes, captured):
    import paged_kv_cache_254_gb300 as pa
    r = np.random.default_rng(Hq + nodes)
    B, N = 16, 5
    prompts = [0, 3, 40, 16, 100]
    bm = pa.BlockManager(200, B, seed=1)
    dt = torch.bfloat16
    kp = torch.zeros(200, Hkv, B, d, dtype=dt, device="cuda")
    vp = torch.zeros_like(kp)
    freq, scale = pa.rope_inv_freq(d, scaling="yarn", factor=4.0, original_len=64)
    gen = torch.Generator(device="cuda").manual_seed(3)
    qw, kw = (torch.randn(d, device="cuda", generator=gen).to(dt) for _ in range(2))
    kept = [[] for _ in range(N)]                 # (k, v, position) of every token that stays, in order

    def append(qkv, pos, slots):
        T = len(pos)
        q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], 1))
        out = pa.pa_rope_append_kv(q, k, v, dev(pos, torch.int32), dev(slots, torch.int64), kp, vp, freq,
                                   rope_scale=scale, q_weight=qw, k_weight=kw)
        return out, k, v, T

    def draw(T):
        return torch.randn(T, (Hq + 2 * Hkv) * d, device="cuda", generator=gen).to(dt)

    for b, n in enumerate(prompts):
        slots = bm.add_sequence(b, n)
        if n:
            _, k, v, _ = append(draw(n), np.arange(n), slots)
            kept[b] += [(k[i], v[i], i) for i in range(n)]
    for step in range(3):
        sizes = [int(x) for x in r.integers(1, nodes + 1, size=N)]
        sizes[step] = nodes
        parents = [[-1] + [int(r.integers(max(0, i - 4), i)) for i in range(1, n)] for n in sizes]
        depth = []
        for p in parents:
            level = [0] * len(p)
            for i in range(1, len(p)):
                level[i] = level[p[i]] + 1
            depth.append(level)
        before = [bm.length(b) for b in range(N)]
        slots = bm.append_slots([(b, n) for b, n in enumerate(sizes)])
        assert slots is not None and len(bm.take_copies()) == 0
        pos = np.concatenate([before[b] + np.array(depth[b]) for b in range(N)])
        qkv = draw(len(pos))
        q, k, v, T = append(qkv, pos, slots)
        qs = np.concatenate([[0], np.cumsum(sizes)])
        q_start = dev(qs, torch.int32)
        table = dev(bm.block_tables(range(N), 16), torch.int32)
        lens = dev(bm.context_lens(range(N)), torch.int32)
        masks = pa.tree_masks(dev(np.concatenate(parents), torch.int32), q_start)
        draft, target = r.integers(0, 2, size=T), r.integers(0, 2, size=T)
        td, tt = dev(draft, torch.int64), dev(target, torch.int64)

        def attend_verify_keep():
            out = pa.pa_decode_tree(q, kp, vp, table, lens, q_start, masks, d ** -0.5, max_nodes=nodes)
            path, count, nxt, new_lens = pa.pa_tree_verify(masks, td, tt, q_start, lens, max_nodes=nodes)
            pa.pa_keep_kv(path, q_start, lens, table, kp, vp)
            return out, path, count, nxt, new_lens

        want = decode_tree_ref(q, kp, vp, table, lens, qs, masks, d ** -0.5)
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out, path, count, nxt, new_lens = attend_verify_keep()
            graph.replay()
        else:
            out, path, count, nxt, new_lens = attend_verify_keep()
        assert_close(out, want, what=f"tree attention, step {step}")
        for b in range(N):
            way, following = verify_ref(parents[b], draft[qs[b]:qs[b + 1]].tolist(), target[qs[b]:qs[b + 1]].tolist())
            assert path[b, :len(way)].tolist() == way and int(count[b]) == len(way) and int(nxt[b]) == following
            kept[b] += [(k[qs[b] + i], v[qs[b] + i], before[b] + d_) for d_, i in enumerate(way)]
            bm.truncate(b, int(new_lens[b]))
            assert bm.length(b) == len(kept[b])
    # a last single-token decode over the kept tokens, against a cache built without speculation
    q1 = torch.randn(N, Hq, d, device="cuda", generator=gen).to(dt)
    got = pa.pa_decode(q1, kp, vp, dev(bm.block_tables(range(N), 16), torch.int32),
                       dev(bm.context_lens(range(N)), torch.int32), d ** -0.5)
    f = freq.double().cpu().numpy()
    for b in range(N):
        ks = torch.stack([x[0] for x in kept[b]])
        vs = torch.stack([x[1] for x in kept[b]])
        kr = rotate_ref(norm_ref(ks, kw, 1e-6), [x[2] for x in kept[b]], f, False, scale)
        n = len(kept[b])
        kr16 = torch.from_numpy(kr).to(dt)         # the cache holds 16-bit keys
        dense = decode_ref(q1[b:b + 1], kr16.transpose(0, 1)[None], vs.transpose(0, 1)[None], [[0]], [n], d ** -0.5)
        assert_close(got[b:b + 1], dense, what=f"decode after three steps, sequence {b}")
