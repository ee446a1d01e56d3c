"""Calls on the block-scaled 8-bit cache as programs make them: both host sides, views of a
projection, other streams, threads, graphs, empty calls, refusals, and a whole run of them
together."""

import threading

import numpy as np
import pytest
import torch

from oracle.attention import decode_multi_ref
from oracle.bs8 import append_bs8_ref, dequantized_pools, pack_bs8_ref
from tests.bs8_util import DTYPES, attention, check, dev, pa, place, random_pool
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def i32(x):
    return dev(np.asarray(x, np.int32))


def f32(t):
    return t.detach().float().cpu().numpy()


class Call:
    """A cache, new tokens and queries, and each attention over it."""

    def __init__(self, seed, ctx, n, Hq=8, Hkv=2, B=16, d=128, dtype="bf16", fmt="e4m3"):
        r = np.random.default_rng(seed)
        self.table_np, NB = place(r, ctx, B)
        self.pool_np = random_pool(r, NB, Hkv, B, d, fmt, powers=True)
        self.q_start_np = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        T, t = int(self.q_start_np[-1]), DTYPES[dtype]
        self.qkv = torch.from_numpy(r.standard_normal((T, (Hq + 2 * Hkv) * d))).to(t).cuda()
        q, k, v = self.qkv.split([Hq * d, Hkv * d, Hkv * d], 1)
        self.k, self.v = k.unflatten(1, (Hkv, d)), v.unflatten(1, (Hkv, d))
        self.q = q.unflatten(1, (Hq, d)).contiguous()
        self.one = torch.from_numpy(r.standard_normal((len(ctx), Hq, d))).to(t).cuda()
        self.ctx, self.n, self.fmt, self.B, self.scale = list(ctx), max(1, max(n)), fmt, B, float(1 / np.sqrt(d))
        self.pool, self.table, self.lens, self.q_start = dev(self.pool_np), dev(self.table_np), i32(ctx), dev(self.q_start_np)

    def append(self, **kw):
        pa().pa_append_kv_bs8(self.k, self.v, self.table, self.lens, self.q_start, self.pool, self.fmt, self.n, **kw)

    def chunk(self, **kw):
        return pa().pa_decode_multi_bs8(self.q, self.pool, self.table, self.lens, self.q_start, self.scale, self.fmt, self.n, **kw)

    def decode(self, **kw):
        return pa().pa_decode_bs8(self.one, self.pool, self.table, self.lens, self.scale, self.fmt, **kw)

    def appended(self):
        return append_bs8_ref(self.pool_np, f32(self.k), f32(self.v), self.table_np, self.ctx, self.q_start_np, self.B, self.fmt)


CTX, NEW = [700, 33, 1, 16, 260], [5, 33, 1, 1, 20]


# ---------------------------------------------------------------- the two host sides
def test_both_host_sides_make_the_same_calls(monkeypatch):
    from paged_kv_cache_254_gb300 import _lib, ops
    outs, fast = [], ops._load_fast()
    assert not isinstance(fast, _lib._Declining)
    for module in (fast, _lib._Declining()):
        monkeypatch.setattr(ops, "_fast", module)
        c = Call(1, CTX, NEW)
        c.append()
        wide = [torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        pairs = i32([[2, 1], [0, 3]])
        pa().pa_unpack_blocks_bs8(pairs, c.pool, *wide)
        outs.append([c.pool.clone(), c.chunk(), c.decode(), *wide])
        pa().pa_pack_blocks_bs8(i32([[1, 0]]), *wide, c.pool)
        outs[-1].append(c.pool)
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_the_compiled_side_takes_ordinary_calls(monkeypatch):
    # (a call that it declines is made all the same, only later: the Python side is not reached here)
    from paged_kv_cache_254_gb300 import ops
    c = Call(2, CTX, NEW)
    c.append(), c.chunk(), c.decode()                          # workspaces are there from here on
    for name in ("_append_kv_bs8", "_decode_bs8", "_decode_multi_bs8", "_convert_bs8"):
        monkeypatch.setattr(ops, name, lambda *a: pytest.fail("declined"))
    err = pa().new_error_word("cuda")
    c.append(err=err)
    out = torch.empty_like(c.q)
    assert c.chunk(out=out, err=err) is out
    c.decode()
    wide = [torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pa().pa_unpack_blocks_bs8(i32([[2, 1]]), c.pool, *wide, err=err)
    pa().pa_pack_blocks_bs8(i32([[1, 0]]), *wide, c.pool, err=err)
    assert int(err.item()) == 0


# ---------------------------------------------------------------- operands
def test_append_takes_views_of_a_projection():
    c = Call(3, CTX, NEW)
    assert c.k.stride(0) == 12 * 128 and not c.k.is_contiguous()
    c.append()
    assert np.array_equal(c.pool.cpu().numpy(), c.appended())
    one = Call(4, [40], [1])
    one.k = one.k.as_strided((1, 2, 128), (8, 128, 1))         # a single token's own stride is never used
    one.append()
    assert np.array_equal(one.pool.cpu().numpy(), one.appended())


def test_given_outputs_and_workspaces():
    c = Call(5, CTX, NEW)
    c.append()
    want = c.chunk(), c.decode()
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    for f, w in zip((c.chunk, c.decode), want):
        out = torch.full_like(w, 7)
        assert f(out=out, workspace=ws) is out and torch.equal(out, w)
        with pytest.raises(Exception, match="[Ww]orkspace"):
            f(workspace=ws[:512])
    for f, q in ((c.chunk, c.q), (c.decode, c.one)):
        with pytest.raises(Exception):
            f(out=q)                                           # over the queries


def test_refusals():
    c = Call(6, CTX, NEW)
    before = c.pool.clone()
    bad = [lambda: pa().pa_append_kv_bs8(c.k.float(), c.v, c.table, c.lens, c.q_start, c.pool),
           lambda: pa().pa_append_kv_bs8(c.k, c.v.half(), c.table, c.lens, c.q_start, c.pool),
           lambda: pa().pa_append_kv_bs8(c.k[:, :1], c.v[:, :1], c.table, c.lens, c.q_start, c.pool),
           lambda: pa().pa_append_kv_bs8(c.k, c.v, c.table.long(), c.lens, c.q_start, c.pool),
           lambda: pa().pa_append_kv_bs8(c.k, c.v, c.table, c.lens[:-1], c.q_start, c.pool),
           lambda: pa().pa_append_kv_bs8(c.k, c.v, c.table, c.lens, c.q_start[:-1], c.pool),
           lambda: pa().pa_append_kv_bs8(c.k, c.v, c.table, c.lens, c.q_start, c.pool[..., :-32]),
           lambda: pa().pa_append_kv_bs8(c.k, c.v, c.table, c.lens, c.q_start, c.pool, max_new=0),
           lambda: pa().pa_append_kv_bs8(c.k, c.v, c.table, c.lens, c.q_start, c.pool, "fp8"),
           lambda: pa().pa_append_kv_bs8(c.k.transpose(1, 2), c.v, c.table, c.lens, c.q_start, c.pool),
           lambda: pa().pa_decode_bs8(c.one.float(), c.pool, c.table, c.lens, 0.1),
           lambda: pa().pa_decode_bs8(c.one[:-1], c.pool, c.table, c.lens, 0.1),
           lambda: pa().pa_decode_bs8(c.one[:, :3].contiguous(), c.pool, c.table, c.lens, 0.1),
           lambda: pa().pa_decode_bs8(c.one, c.pool.view(torch.int8), c.table, c.lens, 0.1),
           lambda: pa().pa_decode_bs8(c.one, c.pool, c.table, c.lens, float("nan")),
           lambda: pa().pa_decode_bs8(c.one[..., :64].contiguous(), c.pool[..., :-1], c.table, c.lens, 0.1),
           lambda: pa().pa_decode_multi_bs8(c.q, c.pool, c.table, c.lens, c.q_start, 0.1, max_q_len=0),
           lambda: pa().pa_decode_multi_bs8(c.q, c.pool, c.table, c.lens, c.q_start.long(), 0.1),
           lambda: pa().pa_decode_multi_bs8(c.q, c.pool, c.table, c.lens, None, 0.1),
           lambda: pa().pa_decode_multi_bs8(c.q, c.pool, c.table, c.lens, c.q_start[1:], 0.1),
           lambda: pa().pa_decode_multi_bs8(c.q, c.pool, c.table, c.lens, c.q_start, 0.1, out=c.q[:-1]),
           lambda: pa().pa_copy_blocks_bs8(i32([1, 2]), c.pool),
           lambda: pa().pa_copy_blocks_bs8(i32([[1, 2]]), c.pool[..., :-16])]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError, pa().PagedAttentionError)):
            call()
            pytest.fail(f"call {i} was not refused")
    torch.cuda.synchronize()
    assert torch.equal(c.pool, before)


def test_calls_without_work():
    c = Call(7, [16, 40], [0, 0])
    before = c.pool.clone()
    c.append()
    assert c.chunk().shape == (0, 8, 128) and torch.equal(c.pool, before)
    none = Call(8, [0, 0], [0, 0])
    none.append()
    assert (none.decode() == 0).all()                          # as pa_decode: nothing cached, zeros
    empty, zero = torch.zeros(0, 3, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    assert pa().pa_decode_bs8(c.one[:0], c.pool, empty, zero, 0.1).shape == (0, 8, 128)
    assert pa().pa_decode_multi_bs8(c.q, c.pool, empty, zero, i32([0]), 0.1).shape == (0, 8, 128)
    pa().pa_append_kv_bs8(c.k, c.v, empty, zero, i32([0]), c.pool)
    pairs = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    wide = [torch.zeros(2, 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pa().pa_copy_blocks_bs8(pairs, c.pool)
    pa().pa_pack_blocks_bs8(pairs, *wide, c.pool)
    pa().pa_unpack_blocks_bs8(pairs, c.pool, *wide)
    assert torch.equal(c.pool, before) and not wide[0].any()


def test_largest_chunks_are_found_on_the_host():
    c = Call(9, CTX, NEW)
    c.append()
    again = Call(9, CTX, NEW)
    pa().pa_append_kv_bs8(again.k, again.v, again.table, again.lens, again.q_start, again.pool)
    assert torch.equal(c.pool, again.pool)
    assert torch.equal(c.chunk(), pa().pa_decode_multi_bs8(c.q, c.pool, c.table, c.lens, c.q_start, c.scale))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n", [4, 40])
def test_infinite_queries_are_nan_whatever_their_scores(dtype, n):
    # every key is negative in dimension 5: an infinity there gives no score but -inf
    c = Call(30, [100, 300], [n, n], dtype=dtype)
    c.k[..., 5] = -c.k[..., 5].abs() - 1
    pa().bs8_scales(c.pool)[...] = 1.0
    c.pool[..., 32:] = 0xB8                                    # -1 in every place
    c.append()
    c.one[0, 1, 5], c.one[1, 3, 5] = float("inf"), float("nan")
    c.q[2, 1, 5], c.q[n, 7, 5], c.q[n + 1, 2, 5] = float("inf"), float("-inf"), float("nan")
    one, q = c.decode(), c.chunk()
    torch.cuda.synchronize()
    assert one.isnan().all(-1).nonzero().tolist() == [[0, 1], [1, 3]] == one.isnan().any(-1).nonzero().tolist()
    want = [[2, 1], [n, 7], [n + 1, 2]]
    assert q.isnan().all(-1).nonzero().tolist() == want == q.isnan().any(-1).nonzero().tolist()


def test_the_timeout_path():
    # every worker's first stage waits, for 100 us at most, on a barrier that nothing completes
    c = Call(31, [700, 2000, 33], [1, 1, 1], Hq=16)
    c.append()
    want = c.decode()
    pa().pa_set_decode_stall_ns(100_000)
    try:
        err = pa().new_error_word("cuda")
        out = c.decode(err=err)
        assert pa().pa_read_error(err) == 5                    # PA_ERR_TIMEOUT
        assert out.isnan().all()                               # cut rows too, through the merge
    finally:
        pa().pa_set_decode_stall_ns(0)
    err = pa().new_error_word("cuda")
    assert torch.equal(c.decode(err=err), want) and pa().pa_read_error(err) == 0


# ---------------------------------------------------------------- streams, threads, graphs
def test_calls_on_another_stream():
    c = Call(10, CTX, NEW)
    c.append()
    want = c.chunk(), c.decode()
    other = Call(10, CTX, NEW)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    other.append(stream=s)
    outs = [other.chunk(stream=s), other.decode(stream=s)]
    with torch.cuda.stream(s):
        outs += [other.chunk(), other.decode()]
    s.synchronize()
    assert torch.equal(other.pool, c.pool) and all(torch.equal(o, want[i % 2]) for i, o in enumerate(outs))


def test_threads_on_one_stream():
    from paged_kv_cache_254_gb300 import ops
    made = [Call(11, CTX, NEW), Call(12, [2000, 5], [3, 5], Hkv=8), Call(13, [900], [200])]
    calls = []
    for c in made:
        c.append()
        calls += [c.chunk, c.decode,
                  lambda c=c: ops._decode_bs8(c.one, c.pool, c.table, c.lens, c.scale, ops.KV_FORMATS[c.fmt], None, None, None)]
    want = [f() for f in calls]
    torch.cuda.synchronize()
    outs = [[None] * 50 for _ in calls]

    def run(i):
        for k in range(50):
            outs[i][k] = calls[i]()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, x) for x in o)


def test_a_captured_step_replayed_over_new_inputs():
    """A decode step (append, then attention over what was appended) as a graph: tokens,
    tables and lengths are read when it is replayed."""
    N, Hq, Hkv, d, B = 3, 8, 2, 128, 16
    r = np.random.default_rng(14)
    lens = np.array([15, 0, 40])
    table_np = r.permutation(12).reshape(N, 4).astype(np.int32)
    pool_np = np.zeros((12, Hkv, 32 + 2 * B * d), np.uint8)
    old = [torch.from_numpy(r.standard_normal((int(lens.sum()), Hkv, d))).bfloat16() for _ in range(2)]
    starts = np.concatenate([[0], np.cumsum(lens)])
    pool_np = append_bs8_ref(pool_np, f32(old[0]), f32(old[1]), table_np, lens, starts, B, "e4m3")
    pool, table, ctx, q_start = dev(pool_np), dev(table_np), i32(lens), i32(range(N + 1))
    q, k, v = (torch.zeros(N, h, d, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv))
    warm = pool.clone()
    def step(pool):
        pa().pa_append_kv_bs8(k, v, table, ctx, q_start, pool, max_new=1)
        return (pa().pa_decode_bs8(q, pool, table, ctx, 0.1),
                pa().pa_decode_multi_bs8(q, pool, table, ctx, q_start, 0.1, max_q_len=1))
    ctx += 1
    step(warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(pool)
    assert np.array_equal(pool.cpu().numpy(), pool_np)
    for _ in range(3):
        lens = lens + 1
        ctx.copy_(i32(lens))
        new = [torch.from_numpy(r.standard_normal(x.shape) * 3).bfloat16() for x in (q, k, v)]
        for x, y in zip((q, k, v), new):
            x.copy_(y)
        graph.replay()
        pool_np = append_bs8_ref(pool_np, f32(new[1]), f32(new[2]), table_np, lens, np.arange(N + 1), B, "e4m3")
        assert np.array_equal(pool.cpu().numpy(), pool_np)
        want, bound = attention(new[0], pool_np, table_np, lens, np.arange(N + 1), 0.1, B, "e4m3")
        for o in outs:
            check(o, want, bound)


@pytest.mark.parametrize("kind", ["decode", "chunk"])
def test_captured_calls_share_nothing(kind):
    # two graphs replayed side by side, after eager calls that replaced the stream's workspace
    made = [Call(15, [800, 30, 900], [3, 2, 4]), Call(16, [3000], [7])]
    for c in made:
        c.append()
    calls = [getattr(c, kind) for c in made]
    want = [f() for f in calls]
    graphs, outs = [], []
    for f in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f())
        graphs.append(g)
    big = Call(17, [100] * 64, [8] * 64, Hkv=8)
    big.chunk(), big.decode()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_a_captured_branch_on_another_stream():
    made = [Call(18, [800, 30, 900], [3, 2, 4]), Call(19, [3000], [7])]
    for c in made:
        c.append()
    want = [(c.chunk(), c.decode()) for c in made]
    torch.cuda.synchronize()
    side, graph, outs = torch.cuda.Stream(), torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        for _ in range(3):
            outs.append((0, made[0].chunk(stream=side), made[0].decode(stream=side)))
            outs.append((1, made[1].chunk(), made[1].decode()))
        here.wait_stream(side)
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, want[i][0]) and torch.equal(b, want[i][1]) for i, a, b in outs)


def test_calls_of_different_sizes_queued_on_one_workspace():
    made = [Call(20 + i, [50 + 700 * i] * (4 - i), [1 + 3 * i] * (4 - i), Hkv=1 << i) for i in range(4)]
    ws = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    for c in made:
        c.append()
    want = [(c.chunk(), c.decode()) for c in made]
    got = [[(c.chunk(workspace=ws), c.decode(workspace=ws)) for c in made] for _ in range(5)]
    for g in got:
        assert all(torch.equal(a, b) for x, y in zip(g, want) for a, b in zip(x, y))


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("Hq,Hkv,d,B,fmt,dtype", [(8, 2, 128, 16, "e4m3", "bf16"), (4, 4, 64, 32, "e5m2", "fp16")])
def test_a_run_of_serving(Hq, Hkv, d, B, fmt, dtype):
    """Prompts in chunks, a fork whose last block is copied before it is written, decode
    steps, drafted tokens, and a cold sequence that leaves for a 16-bit cache and comes
    back: the pool is the oracle's to the byte throughout, outputs are within their bounds."""
    r = np.random.default_rng(Hq + B)
    bm = pa().BlockManager(64, B, seed=2)
    pool_np = np.zeros((64, Hkv, 32 + 2 * B * d), np.uint8)
    pool = pa().bs8_pool(64, Hkv, B, d)
    t, scale = DTYPES[dtype], float(1 / np.sqrt(d))
    err = pa().new_error_word("cuda")

    def step(seqs, sizes):
        nonlocal pool_np
        copies = bm.take_copies()
        if len(copies):
            pa().pa_copy_blocks_bs8(i32(copies), pool, err=err)
            pool_np = pool_np.copy()
            for a, b in copies:
                pool_np[b] = pool_np[a]
        T, qs = sum(sizes), np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        q, k, v = torch.from_numpy(r.standard_normal((T, (Hq + 2 * Hkv) * d)) * 2).to(t).split([Hq * d, Hkv * d, Hkv * d], 1)
        q, k, v = q.unflatten(1, (Hq, d)), k.unflatten(1, (Hkv, d)), v.unflatten(1, (Hkv, d))
        table, ctx = bm.block_tables(seqs, 8), bm.context_lens(seqs)
        gt, gc, gs = i32(table), i32(ctx), dev(qs)
        pa().pa_append_kv_bs8(k.cuda(), v.cuda(), gt, gc, gs, pool, fmt, max(sizes), err=err)
        pool_np = append_bs8_ref(pool_np, f32(k), f32(v), table, ctx, qs, B, fmt)
        assert np.array_equal(pool.cpu().numpy(), pool_np)
        q = q.contiguous()
        want, bound = attention(q, pool_np, table, ctx, qs, scale, B, fmt)
        check(pa().pa_decode_multi_bs8(q.cuda(), pool, gt, gc, gs, scale, fmt, max(sizes), err=err), want, bound, "chunk")
        if max(sizes) == 1:
            check(pa().pa_decode_bs8(q.cuda(), pool, gt, gc, scale, fmt, err=err), want, bound, "decode")
        assert int(err.item()) == 0

    prompts = {"a": [70, 33], "b": [1, 40], "c": [50]}
    for name, parts in prompts.items():
        assert bm.add_sequence(name, parts[0]) is not None
    step(list("abc"), [p[0] for p in prompts.values()])
    for name in "ab":
        bm.append_slots([(name, prompts[name][1])])
    step(list("ab"), [prompts[n][1] for n in "ab"])
    bm.fork("a", "d")
    for _ in range(3):                                         # one token each
        bm.append_slots([(n, 1) for n in "abcd"])
        step(list("abcd"), [1] * 4)
    bm.append_slots([(n, 5) for n in "db"])                    # drafted tokens; two are accepted
    step(list("db"), [5, 5])
    for n in "db":
        bm.truncate(n, bm.length(n) - 3)
    bm.append_slots([(n, 1) for n in "bd"])                    # over the slots of rejected ones
    step(list("bd"), [1, 1])

    # sequence a goes to a 16-bit cache, is decoded there, and comes back
    ids = bm.table("a")
    wide = [torch.zeros(len(ids), Hkv, B, d, dtype=t, device="cuda") for _ in range(2)]
    out_pairs = np.array([[b, i] for i, b in enumerate(ids)], np.int32)
    pa().pa_unpack_blocks_bs8(dev(out_pairs), pool, *wide, kv_format=fmt, err=err)
    for got, val in zip(wide, dequantized_pools(pool_np, B, d, fmt)):
        assert torch.equal(got.cpu(), torch.from_numpy(val[ids]).float().to(t))
    n = bm.length("a")
    pa().pa_pack_blocks_bs8(dev(out_pairs[:, ::-1].copy()), *wide, pool, kv_format=fmt, err=err)
    before = dequantized_pools(pool_np, B, d, fmt)
    pool_np = pack_bs8_ref(pool_np, *(f32(w) for w in wide), out_pairs[:, ::-1], fmt)
    assert np.array_equal(pool.cpu().numpy(), pool_np) and int(err.item()) == 0
    if fmt == "e4m3":                                          # values are e4m3's, so packed again they are the same
        for x, y in zip(before, dequantized_pools(pool_np, B, d, fmt)):
            assert np.array_equal(x[ids], y[ids])
    q = torch.from_numpy(r.standard_normal((1, Hq, d))).to(t)
    table = bm.block_tables(["a"], 8)
    want, bound = attention(q, pool_np, table, [n], [0, 1], scale, B, fmt)
    check(pa().pa_decode_bs8(q.cuda(), pool, i32(table), i32([n]), scale, fmt), want, bound, "back")
