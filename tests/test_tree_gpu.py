"""pa_decode_tree, pa_tree_verify and pa_keep_kv against the fp64 oracle.

Tolerance of the attention, per element: half a step of the 16-bit output plus
2^-12 of the largest |v| it may weigh.  The latter holds: softmax weights kept
as a pair of 16-bit values (2^-14 relative); their sum over up to 4096 keys, 16
adds in 4 chains a stage and one a stage (84 * 2^-24 < 2^-17); the products'
fp32 accumulation, at most 512 steps (2^-15); scores, whose fp32 dot products
are off by at most 2^-16 of a weight here, and ex2.approx (2^-22).  Their sum is
below 2^-13; a factor of 2 is left for the tensor core's own alignment of
addends.  Longer contexts (up to 33000 keys) take 2^-11: eight times the
accumulation steps."""

import numpy as np
import pytest
import torch

from oracle.kv_ops import bits
from oracle.tree import decode_tree_ref, keep_ref, masks_ref, verify_ref
from tests.gpu_util import dev_case, need_gpu, plant_key, sharpen
from workloads import DecodeConfig, make_decode_case, make_values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def pa():
    import paged_kv_cache_254_gb300 as m
    return m


def signed(masks):
    return torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64, device="cuda")


def random_tree(n, r):
    return [-1] + [int(r.integers(max(0, i - 6), i)) for i in range(1, n)] if n else []


def tree_case(ctx, sizes, Hq=8, Hkv=2, d=128, B=16, dtype="bf16", seed=3, poison=False):
    cfg = DecodeConfig(name="tree", num_seqs=len(ctx), num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, block_size=B,
                       dtype=dtype, seed=seed, ctx_fixed=tuple(ctx), pool_factor=1.5)
    case = make_decode_case(cfg, device="cuda", poison_unused=poison)
    qs = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    q = make_values((int(qs[-1]), Hq, d), dtype, torch.Generator(device="cuda").manual_seed(seed + 5), "cuda")
    r = np.random.default_rng(seed)
    masks = [m for n in sizes for m in masks_ref(random_tree(n, r))]
    return case, q, qs, masks


def run(case, q, qs, masks, nodes=None, **kw):
    bt, cl = dev_case(case)
    return pa().pa_decode_tree(q, case.k_pool, case.v_pool, bt, cl, torch.from_numpy(qs).cuda(), signed(masks),
                               case.scale, max_nodes=nodes, **kw)


def oracle(case, q, qs, masks):
    return decode_tree_ref(q, case.k_pool, case.v_pool, case.block_tables, case.context_lens, qs, masks, case.scale)


def close(got, ref, case, what="", slack=2.0 ** -12):
    v = case.v_pool[torch.isfinite(case.v_pool)]
    top = float(v.abs().max()) if v.numel() else 1.0
    g = got.detach().double().cpu().numpy()
    assert np.isfinite(ref).all() and np.isfinite(g).all(), f"{what}: non-finite"
    err = np.abs(g - ref)
    bound = torch.finfo(got.dtype).eps / 2 * np.abs(ref) + slack * top
    assert (err <= bound).all(), f"{what}: worst {np.max(err - bound):.3e} over the bound, max err {err.max():.3e}"


EDGE = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 100, 129, 517]


def sizes_for(ctx, nodes, r):
    s = [int(r.integers(0, min(nodes, c) + 1)) for c in ctx]
    s[-1] = min(nodes, ctx[-1])                       # one tree of the full size
    s[3], s[4] = min(nodes, ctx[3]), 0                # (nearly) no context before the tree; no tree
    return s


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B", [16, 32])
@pytest.mark.parametrize("g,nodes", [(1, 1), (1, 16), (4, 4), (16, 1),            # one 16-row tile
                                     (1, 17), (1, 64), (4, 13), (8, 9), (16, 8),  # one 128-row tile
                                     (2, 64), (4, 33), (4, 64), (8, 31), (8, 64), (16, 23), (16, 64)])
def test_shapes_and_trees(dtype, d, B, g, nodes):
    r = np.random.default_rng(g * 100 + nodes + d + B)
    sizes = sizes_for(EDGE, nodes, r)
    case, q, qs, masks = tree_case(EDGE, sizes, Hq=g, Hkv=1, d=d, B=B, dtype=dtype, seed=7 + g + nodes + d + B,
                                   poison=True)
    close(run(case, q, qs, masks, nodes), oracle(case, q, qs, masks), case, f"{dtype} d{d} B{B} g{g} nodes {nodes}")


@pytest.mark.parametrize("g,nodes", [(4, 3), (4, 20), (8, 64)])
def test_heads_of_several_groups(g, nodes):
    r = np.random.default_rng(nodes)
    ctx = [70, 300, 1000, 64, 64, 90]
    case, q, qs, masks = tree_case(ctx, sizes_for(ctx, nodes, r), Hq=3 * g, Hkv=3, seed=31 + nodes)
    close(run(case, q, qs, masks, nodes), oracle(case, q, qs, masks), case)


@pytest.mark.parametrize("g,nodes", [(2, 8), (4, 24), (8, 48)])
def test_any_mask_and_rows_that_see_nothing(g, nodes):
    # masks that are no trees: random sets, empty ones, bits past the tree; with and without keys before it
    r = np.random.default_rng(nodes)
    ctx = [nodes, nodes + 1, 200, nodes, 77, nodes + 16]
    sizes = [nodes, nodes, nodes, nodes - 3, 5, nodes]
    case, q, qs, _ = tree_case(ctx, sizes, Hq=2 * g, Hkv=2, seed=41 + nodes, poison=True)
    masks = [int(m) for m in r.integers(0, 1 << 63, size=int(qs[-1]))]
    for i in range(0, len(masks), 3):
        masks[i] = 0
    masks[1] = ((1 << 64) - 1) ^ ((1 << nodes) - 1)         # only bits past the tree
    got = run(case, q, qs, masks, nodes)
    close(got, oracle(case, q, qs, masks), case)
    assert (got[[0, 1, 3]] == 0).all()                      # sequence 0 has no keys before its tree


@pytest.mark.parametrize("g,nodes", [(4, 4), (4, 16), (8, 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_unseen_nodes_may_hold_anything(g, nodes, bad):
    ctx, sizes = [nodes + 13, 200, nodes], [nodes, nodes, nodes]
    case, q, qs, masks = tree_case(ctx, sizes, Hq=2 * g, Hkv=2, seed=51 + nodes, poison=True)
    want = oracle(case, q, qs, masks)
    B = 16
    hit = [1, nodes - 1]                                    # nodes spoilt in every tree
    for b in range(3):
        for j in hit:
            t = ctx[b] - nodes + j
            blk = int(case.block_tables[b, t // B])
            case.v_pool[blk, :, t % B, (5 * j) % 128] = bad
            case.k_pool[blk, :, t % B, 7] = bad
    got = run(case, q, qs, masks, nodes)
    sees = np.array([any((masks[i] >> j) & 1 for j in hit) for i in range(int(qs[-1]))])
    assert sees.any() and not sees.all()
    clean = torch.from_numpy(~sees)
    close(got[clean.cuda()], want[~sees], case, "rows that do not see the spoilt nodes")
    # a row that sees one is NaN, except that a key of -inf score simply gets no weight:
    # V is spoilt as well here, so NaN it is
    assert torch.isnan(got[torch.from_numpy(sees).cuda()].float()).all()


def test_long_contexts_split_across_ctas():
    ctx = [20000, 17, 9000, 33000]
    for g, nodes in ((4, 4), (4, 30), (8, 40)):
        sizes = [nodes, min(nodes, 17), nodes // 2, nodes]
        case, q, qs, masks = tree_case(ctx, sizes, Hq=g, Hkv=1, seed=61 + nodes, poison=True)
        rows = [0, int(qs[1]) - 1, int(qs[1]), int(qs[2]), int(qs[3]), int(qs[4]) - 1]
        got = run(case, q, qs, masks, nodes)
        # the oracle on a few rows (a full one walks 2M keys a head): trees cut to those rows' visibility
        ref = np.concatenate([decode_rows(case, q, qs, masks, i) for i in rows])
        close(got[torch.tensor(rows).cuda()], ref, case, f"long, {nodes} nodes", slack=2.0 ** -11)
        assert torch.isfinite(got.float()).all()


def decode_rows(case, q, qs, masks, i):
    """The oracle's row i alone, as a tree of which only that node asks."""
    b = int(np.searchsorted(qs, i, side="right")) - 1
    n = int(qs[b + 1] - qs[b])
    one = decode_tree_ref(q[i:i + 1].expand(n, -1, -1)[:n], case.k_pool, case.v_pool, case.block_tables[b:b + 1],
                          case.context_lens[b:b + 1], [0, n], [masks[i]] + [0] * (n - 1), case.scale)
    return one[:1]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("q_mult,k_growth", [(8.0, 0.0), (2.0, 6.0)])
@pytest.mark.parametrize("g,nodes", [(8, 2), (4, 16), (8, 40)])
def test_peaked_scores(dtype, q_mult, k_growth, g, nodes):
    ctx = [3000, 70, 2000, 64, 64, 777, 65, 1500]
    r = np.random.default_rng(nodes)
    case, q, qs, masks = tree_case(ctx, sizes_for(ctx, nodes, r), Hq=g, Hkv=1, dtype=dtype, seed=71 + nodes)
    q.mul_(q_mult)
    sharpen(case, 1.0, k_growth)
    # scores up to ~300 in magnitude: their fp32 dot products are off by up to 2^-12 of a weight
    close(run(case, q, qs, masks, nodes), oracle(case, q, qs, masks), case, slack=2.0 ** -11)


def test_dominant_keys_on_one_branch():
    ctx, nodes = [2500], 40
    case, q, qs, masks = tree_case(ctx, [nodes], Hq=8, Hkv=2, seed=81)
    plant_key(case, 0, 1000, target=20.0, q=q[0])
    plant_key(case, 0, ctx[0] - nodes + 11, target=35.0, q=q[nodes - 1])
    close(run(case, q, qs, masks, nodes), oracle(case, q, qs, masks), case, slack=2.0 ** -11)


def test_chain_equals_the_chunk_call():
    ctx, sizes = [40, 300, 17], [5, 12, 16]
    case, q, qs, _ = tree_case(ctx, sizes, Hq=8, Hkv=2, seed=91)
    masks = [m for n in sizes for m in masks_ref(list(range(-1, n - 1)))]
    bt, cl = dev_case(case)
    chunk = pa().pa_decode_multi(q, case.k_pool, case.v_pool, bt, cl, torch.from_numpy(qs).cuda(), case.scale,
                                 max_q_len=16)
    want = oracle(case, q, qs, masks)
    close(run(case, q, qs, masks, 16), want, case)
    close(chunk, want, case)


@pytest.mark.parametrize("g,nodes", [(4, 4), (4, 20), (8, 64)])
def test_deterministic_and_placement_invariant(g, nodes):
    ctx = [700, 3000, 65, 1200]
    case, q, qs, masks = tree_case(ctx, [nodes, nodes, nodes // 2, nodes], Hq=2 * g, Hkv=2, seed=101)
    a = run(case, q, qs, masks, nodes)
    assert torch.equal(a, run(case, q, qs, masks, nodes))
    nb = case.num_blocks
    perm = np.random.default_rng(1).permutation(nb)
    pt = torch.from_numpy(perm).cuda()
    k2, v2 = torch.empty_like(case.k_pool), torch.empty_like(case.v_pool)
    k2[pt], v2[pt] = case.k_pool, case.v_pool
    case.k_pool, case.v_pool = k2, v2
    case.block_tables = np.where(case.block_tables >= 0, perm[np.clip(case.block_tables, 0, nb - 1)], -1).astype(np.int32)
    assert torch.equal(a, run(case, q, qs, masks, nodes))


@pytest.mark.parametrize("g,nodes", [(2, 6), (8, 6), (8, 30)])
def test_malformed_trees_and_blocks_poison_their_rows_only(g, nodes):
    ctx = [100, 400, 3, 70, 90]
    sizes = [nodes, nodes + 3, 5, 1, 4]             # 1: larger than max_nodes; 2: more than its context
    case, q, qs, masks = tree_case(ctx, sizes, Hq=2 * g, Hkv=2, seed=111)
    case.block_tables[4, 2] = case.num_blocks + 3   # a bad block id
    err = pa().new_error_word("cuda")
    got = run(case, q, qs, masks, nodes, err=err).float()
    assert pa().pa_read_error(err) == 4 and int(err.item()) == (2 | 1)
    for b in (1, 2, 4):
        assert torch.isnan(got[qs[b]:qs[b + 1]]).all()
    keep = list(range(qs[0], qs[1])) + list(range(qs[3], qs[4]))
    case2 = type(case)(**{**case.__dict__, "block_tables": case.block_tables[[0, 3]],
                          "context_lens": case.context_lens[[0, 3]]})
    ref = oracle(case2, q[keep], np.array([0, nodes, nodes + 1], dtype=np.int32), [masks[i] for i in keep])
    close(got[keep].to(q.dtype), ref, case)
    # rows outside every sequence stay as they were
    out = torch.full_like(q, 3.0)
    short = qs.copy()
    short[-2:] = short[-3]
    bt, cl = dev_case(case)
    pa().pa_decode_tree(q, case.k_pool, case.v_pool, bt, cl, torch.from_numpy(short).cuda(), signed(masks), case.scale,
                        max_nodes=nodes, out=out)
    assert (out[short[-1]:] == 3.0).all()


def test_refusals_on_the_device():
    case, q, qs, masks = tree_case([40], [4], Hq=8, Hkv=2)
    bt, cl = dev_case(case)
    good = dict(q=q, k_pool=case.k_pool, v_pool=case.v_pool, block_tables=bt, context_lens=cl,
                q_start=torch.from_numpy(qs).cuda(), tree_masks=signed(masks), scale=case.scale, max_nodes=4)
    E = (ValueError, TypeError, pa().PagedAttentionError)
    for bad in (dict(max_nodes=65), dict(max_nodes=0), dict(tree_masks=signed(masks).int()), dict(q=q[:, :, :64]),
                dict(q=q.float()), dict(tree_masks=signed(masks)[:2]), dict(scale=float("nan")), dict(q=q[:, :3]),
                dict(out=q[:2]), dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda")),
                dict(context_lens=cl.long()), dict(block_tables=bt.cpu()), dict(q_start=good["q_start"][:1])):
        with pytest.raises(E):
            pa().pa_decode_tree(**{**good, **bad})
    # no rows at all: fine
    none = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert pa().pa_decode_tree(**{**good, "q": q[:0], "tree_masks": signed([]), "q_start": none}).shape[0] == 0


@pytest.mark.parametrize("g,nodes,N", [(2, 4, 700), (8, 3, 700), (16, 9, 400)])
def test_many_short_sequences(g, nodes, N):
    # more sequences than threads look for a chunk's beginning, empty trees and contexts among them
    r = np.random.default_rng(N + nodes)
    ctx = [int(x) for x in r.integers(0, 40, size=N)]
    sizes = [int(r.integers(0, min(nodes, c) + 1)) for c in ctx]
    cfg = DecodeConfig(name="many", num_seqs=N, num_q_heads=g, num_kv_heads=1, head_dim=64, block_size=16, dtype="fp16",
                       seed=N, ctx_fixed=tuple(ctx), pool_factor=1.2)
    case = make_decode_case(cfg, device="cuda", poison_unused=True)
    qs = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    q = make_values((int(qs[-1]), g, 64), "fp16", torch.Generator(device="cuda").manual_seed(N), "cuda")
    masks = [m for n in sizes for m in masks_ref(random_tree(n, r))]
    close(run(case, q, qs, masks, nodes), oracle(case, q, qs, masks), case)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g,nodes", [(4, 4), (2, 20), (4, 64)])
def test_one_long_sequence_in_many_pieces(d, g, nodes):
    case, q, qs, masks = tree_case([4000], [nodes], Hq=2 * g, Hkv=2, d=d, seed=161 + nodes)
    close(run(case, q, qs, masks, nodes), oracle(case, q, qs, masks), case)


def test_negative_and_zero_scales():
    case, q, qs, masks = tree_case([70, 300, 40], [20, 33, 40], Hq=8, Hkv=2, seed=171)
    for case.scale in (-0.09, 0.0):
        close(run(case, q, qs, masks, 40), oracle(case, q, qs, masks), case, f"scale {case.scale}")
    small, sq, sqs, sm = tree_case([70, 30], [4, 3], Hq=8, Hkv=2, seed=181)
    mid, mq, mqs, mm = tree_case([70, 90], [12, 9], Hq=8, Hkv=2, seed=191)
    for s in (-0.09, 0.0):
        small.scale = mid.scale = s
        close(run(small, sq, sqs, sm, 4), oracle(small, sq, sqs, sm), small, f"scale {s}")
        close(run(mid, mq, mqs, mm, 12), oracle(mid, mq, mqs, mm), mid, f"scale {s}")


def test_compiled_and_checked_host_sides_agree():
    # the compiled calls and the Python ones behind them give the same results
    from paged_kv_cache_254_gb300 import ops
    case, q, qs, masks = tree_case([300, 70], [20, 9], Hq=8, Hkv=2, seed=201)
    bt, cl = dev_case(case)
    args = (q, case.k_pool, case.v_pool, bt, cl, torch.from_numpy(qs).cuda(), signed(masks), case.scale, 20, None, None,
            None)
    want = ops._decode_tree(*args)
    fast = ops._load_fast()
    got = fast.decode_tree(ops._sp_cache, *args)
    assert got is not NotImplemented and torch.equal(got, want)
    assert fast.decode_tree({}, *args) is NotImplemented                     # no workspace yet
    trees, draft, target, vqs = verify_inputs([6, 13, 0, 64], seed=9)
    v = (signed([m for t in trees for m in masks_ref(t)]), cat(draft), cat(target), torch.from_numpy(vqs).cuda(),
         torch.tensor([10, 13, 4, 99], dtype=torch.int32, device="cuda"), 64, None, None)
    for a, b in zip(fast.tree_verify(*v), ops._tree_verify(*v)):
        assert a.dtype == b.dtype and a.shape == b.shape and a.is_contiguous() and torch.equal(a, b)
    given = torch.empty(4, 64, dtype=torch.int32, device="cuda")
    assert fast.tree_verify(*v[:6], given, None)[0] is given
    # whatever is not plainly right is declined, and nothing is launched
    for bad in ((q.float(),) + args[1:], args[:8] + (0,) + args[9:], args[:8] + (65,) + args[9:], args[:7] + (1,) + args[8:],
                args[:4] + (cl.long(),) + args[5:], args[:9] + (q,) + args[10:], (q.cpu(),) + args[1:]):
        assert fast.decode_tree(ops._sp_cache, *bad) is NotImplemented
    for bad in (1 << 70, -(1 << 70)):
        with pytest.raises(ValueError):
            pa().pa_decode_tree(*args[:8], max_nodes=bad)
        with pytest.raises(ValueError):
            pa().pa_tree_verify(*v[:5], bad)
    assert fast.tree_verify(*v[:5]) is NotImplemented and fast.keep_kv() is NotImplemented


def test_captured_graphs_share_nothing():
    # two captured calls replayed side by side on two streams, after eager calls that regrow the shared workspace
    a = tree_case([3000, 900], [20, 20], Hq=8, Hkv=2, seed=121)
    b = tree_case([2000, 1100, 50], [4, 4, 4], Hq=8, Hkv=2, seed=131)
    want = [run(*a, 20), run(*b, 4)]
    args = []
    for case, q, qs, masks in (a, b):
        bt, cl = dev_case(case)
        args.append((q, case.k_pool, case.v_pool, bt, cl, torch.from_numpy(qs).cuda(), signed(masks), case.scale))
    graphs, outs = [], []
    for x, nodes in zip(args, (20, 4)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(pa().pa_decode_tree(*x, max_nodes=nodes))
        graphs.append(g)
    big = tree_case([70] * 40, [64] * 40, Hq=16, Hkv=1, seed=141)
    run(*big, 64)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_calls_on_two_streams_at_once():
    a = tree_case([3000, 900], [20, 20], Hq=8, Hkv=2, seed=151)
    want = run(*a, 20)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = [run(*a, 20, stream=s) for _ in range(10) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


# ---------------------------------------------------------------- verification
def verify_inputs(sizes, seed, tokens=3):
    r = np.random.default_rng(seed)
    trees = [random_tree(n, r) for n in sizes]
    draft = [r.integers(0, tokens, n) for n in sizes]
    target = [r.integers(0, tokens, n) for n in sizes]
    qs = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    return trees, draft, target, qs


def cat(x):
    return torch.from_numpy(np.concatenate(x).astype(np.int64)).cuda()


@pytest.mark.parametrize("sizes", [[1], [8], [0, 5, 64], [64] * 40, list(range(65))])
@pytest.mark.parametrize("tokens", [1, 2, 5, 50000])
def test_verify(sizes, tokens):
    trees, draft, target, qs = verify_inputs(sizes, seed=len(sizes) + tokens, tokens=tokens)
    ctx = np.array([n + 7 * i for i, n in enumerate(sizes)], dtype=np.int32)
    P = max(sizes)
    path, count, nxt, lens = pa().pa_tree_verify(
        signed([m for t in trees for m in masks_ref(t)]), cat(draft), cat(target), torch.from_numpy(qs).cuda(),
        torch.from_numpy(ctx).cuda(), max_nodes=P)
    for b, n in enumerate(sizes):
        want, wn = verify_ref(trees[b], draft[b].tolist(), target[b].tolist())
        assert path[b].tolist() == want + [-1] * (P - len(want))
        assert int(count[b]) == len(want) and int(nxt[b]) == wn and int(lens[b]) == ctx[b] - n + len(want)


def test_verify_malformed_and_refusals():
    trees, draft, target, qs = verify_inputs([6, 3, 4], seed=2)
    m = signed([x for t in trees for x in masks_ref(t)])
    ctx = torch.tensor([10, 2, 9], dtype=torch.int32, device="cuda")     # 1: more nodes than context
    start = torch.from_numpy(qs).cuda()
    err = pa().new_error_word("cuda")
    path, count, nxt, lens = pa().pa_tree_verify(m, cat(draft), cat(target), start, ctx, max_nodes=5, err=err)
    assert int(err.item()) == 2                                           # 0: more nodes than max_nodes
    for b in (0, 1):
        assert path[b].tolist() == [-1] * 5 and int(count[b]) == 0 and int(nxt[b]) == -1 and int(lens[b]) == int(ctx[b])
    assert path[2, 0] == 0 and int(count[2]) >= 1
    E = (ValueError, TypeError, pa().PagedAttentionError)
    good = dict(tree_masks=m, draft_tokens=cat(draft), target_tokens=cat(target), q_start=start, context_lens=ctx)
    for bad in (dict(max_nodes=0), dict(max_nodes=65), dict(draft_tokens=cat(draft).int()), dict(context_lens=ctx[:2]),
                dict(target_tokens=cat(target)[:4]), dict(path=path, max_nodes=6)):
        with pytest.raises(E):
            pa().pa_tree_verify(**{**good, **bad})


# ---------------------------------------------------------------- keeping the accepted tokens
@pytest.mark.parametrize("dtype,d,B,Hkv", [("bf16", 128, 16, 8), ("fp16", 64, 32, 3), ("bf16", 64, 16, 1),
                                           ("bf16", 80, 16, 2), ("fp16", 256, 32, 5)])
@pytest.mark.parametrize("nodes", [1, 9, 64])
def test_keep(dtype, d, B, Hkv, nodes):
    r = np.random.default_rng(nodes + d)
    sizes = [nodes, 0, max(1, nodes // 2), nodes, nodes, nodes]
    ctx = np.array([nodes + int(x) for x in r.integers(0, 70, size=6)], dtype=np.int32)
    case = make_decode_case(DecodeConfig(name="keep", num_seqs=6, num_q_heads=Hkv, num_kv_heads=Hkv, head_dim=d,
                                         block_size=B, dtype=dtype, seed=5, ctx_fixed=tuple(ctx), pool_factor=1.5),
                            device="cuda", poison_unused=True)
    qs = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    path = np.full((6, nodes), -1, dtype=np.int32)
    for b, n in enumerate(sizes):
        k = [n, 0, min(n, 1), n // 2, max(1, n - 1), min(3, n)][b]    # every node; none; the root; some; all but one
        path[b, :k] = np.sort(r.permutation(n)[:k])
    want = keep_ref(bits(case.k_pool), bits(case.v_pool), path, qs, case.block_tables, ctx, B)
    bt, cl = dev_case(case)
    pa().pa_keep_kv(torch.from_numpy(path).cuda(), torch.from_numpy(qs).cuda(), cl, bt, case.k_pool, case.v_pool)
    torch.cuda.synchronize()
    assert np.array_equal(bits(case.k_pool), want[0]) and np.array_equal(bits(case.v_pool), want[1])


def test_keep_bad_paths_move_nothing():
    ctx = [30, 30, 30, 30, 30, 5]
    case, _, _, _ = tree_case(ctx, [4] * 6, Hq=2, Hkv=2, d=64, seed=7)
    case.block_tables[4, 1] = -5
    path = np.array([[0, 2, 2, -1], [0, 3, 1, -1], [0, 4, -1, -1], [-7, 1, 2, 3], [1, 3, -1, -1], [1, 2, 3, -1]], dtype=np.int32)
    sizes = [4, 4, 4, 4, 4, 6]
    sizes[5] = 4
    qs = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    k0, v0 = bits(case.k_pool), bits(case.v_pool)
    only = np.full_like(path, -1)
    only[5] = path[5]
    want = keep_ref(k0, v0, only, qs, case.block_tables, ctx, 16)
    err = pa().new_error_word("cuda")
    bt, cl = dev_case(case)
    pa().pa_keep_kv(torch.from_numpy(path).cuda(), torch.from_numpy(qs).cuda(), cl, bt, case.k_pool, case.v_pool, err=err)
    assert pa().pa_read_error(err) == 4 and int(err.item()) == (128 | 1)
    assert np.array_equal(bits(case.k_pool), want[0]) and np.array_equal(bits(case.v_pool), want[1])
    # sizes that cannot be: more nodes than context, a context past the table
    err = pa().new_error_word("cuda")
    cl2 = torch.tensor([3, 10 ** 6, -1, 4, 4, 4], dtype=torch.int32, device="cuda")
    pa().pa_keep_kv(torch.from_numpy(only).cuda(), torch.from_numpy(qs).cuda(), cl2, bt, case.k_pool, case.v_pool, err=err)
    assert int(err.item()) & 2
    E = (ValueError, TypeError, pa().PagedAttentionError)
    for bad in (dict(path=bt.long()), dict(k_pool=case.k_pool.float()), dict(path=torch.zeros(6, 65, dtype=torch.int32, device="cuda")),
                dict(q_start=cl), dict(v_pool=case.v_pool[:2])):
        with pytest.raises(E):
            pa().pa_keep_kv(**{**dict(path=torch.from_numpy(only).cuda(), q_start=torch.from_numpy(qs).cuda(),
                                      context_lens=cl, block_tables=bt, k_pool=case.k_pool, v_pool=case.v_pool), **bad})
