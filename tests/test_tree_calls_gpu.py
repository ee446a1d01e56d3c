"""The tree-speculation calls on the device: strides of single tokens through
both host sides, calls after a refused one, errors that other calls left, threads
and graphs."""

import contextlib
import ctypes
import threading

import numpy as np
import pytest
import torch

from oracle.kv_ops import bits
from oracle.tree import keep_ref
from tests.gpu_util import need_gpu
from tests.test_tree_calls import strided_views

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def pa():
    import paged_kv_cache_254_gb300 as m
    return m


# ---------------------------------------------------------------- one token's strides
@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("view", ["interleaved", "expanded", "sliced", "half", "transposed"])
@pytest.mark.parametrize("arg", ["q", "k_new", "v_new"])
def test_scattered_heads_are_refused(T, view, arg):
    from paged_kv_cache_254_gb300 import ops
    H, d = 4, 64
    freq, _ = pa().rope_inv_freq(d)
    dense = torch.ones(T, H, d, dtype=torch.bfloat16, device="cuda")
    pools = [torch.zeros(4, H, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    a = dict(q=dense, k_new=dense, v_new=dense, positions=torch.zeros(T, dtype=torch.int32, device="cuda"),
             slot_mapping=torch.arange(T, device="cuda"), k_pool=pools[0], v_pool=pools[1], inv_freq=freq)
    a[arg] = strided_views(T, H, d, "cuda")[view]
    with pytest.raises(ValueError, match="contiguous"):
        pa().pa_rope_append_kv(**a)
    rest = (False, 1.0, None, None, 1e-6, None, None)
    assert ops._load_fast().rope_append_kv(*a.values(), *rest) is NotImplemented
    torch.cuda.synchronize()
    assert not bits(pools[0]).any() and not bits(pools[1]).any()


def test_one_token_of_a_fused_projection():
    # one row of [q | k | v], whose parts are dense within the token: as before
    H, d = 4, 64
    freq, _ = pa().rope_inv_freq(d)
    row = torch.randn(1, 3 * H * d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    q, k, v = (x.unflatten(1, (H, d)) for x in row.split(H * d, 1))
    pools = [torch.zeros(4, H, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    pos, slot = torch.full((1,), 9, dtype=torch.int32, device="cuda"), torch.full((1,), 21, device="cuda")
    a = pa().pa_rope_append_kv(q, k, v, pos, slot, pools[0], pools[1], freq)
    b = pa().pa_rope_append_kv(*(x.contiguous() for x in (q, k, v)), pos, slot, pools[2], pools[3], freq)
    assert torch.equal(a, b) and np.array_equal(bits(pools[0]), bits(pools[2]))
    assert torch.equal(pools[1][1, :, 5], v[0])


# ---------------------------------------------------------------- workspaces
def small_tree(N=2, nodes=5, Hq=8, Hkv=2, d=64, B=16, MB=4, seed=7):
    """Arguments of a pa_decode_tree call: contexts of 3 blocks and a bit, chains of ``nodes``."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    values = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()
    table = torch.randperm(N * MB, device="cuda", generator=g).int().view(N, MB)
    masks = torch.tensor([(2 << i) - 1 for i in range(nodes)] * N, device="cuda")
    return dict(q=values(N * nodes, Hq, d), k_pool=values(N * MB, Hkv, B, d), v_pool=values(N * MB, Hkv, B, d),
                block_tables=table, context_lens=torch.full((N,), 3 * B + 2, dtype=torch.int32, device="cuda"),
                q_start=torch.arange(0, N * nodes + 1, nodes, dtype=torch.int32, device="cuda"), tree_masks=masks,
                scale=d ** -0.5, max_nodes=nodes)


def test_a_valid_call_after_a_refused_one():
    a = small_tree(N=3, nodes=7)                       # sizes that no other test has
    with pytest.raises(pa().PagedAttentionError):
        pa().pa_decode_tree(**{**a, "block_tables": a["block_tables"][:, :0].contiguous()})
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        captured = pa().pa_decode_tree(**a)
    graph.replay()
    torch.cuda.synchronize()
    eager = pa().pa_decode_tree(**a, stream=torch.cuda.Stream())     # no workspace kept for this one
    torch.cuda.synchronize()
    assert torch.isfinite(eager.float()).all() and torch.equal(captured, eager)


# ---------------------------------------------------------------- errors of other calls
def cudart():
    """The runtime that torch has loaded."""
    with open("/proc/self/maps") as f:
        path = next(line.split()[-1] for line in f if "libcudart" in line)
    return ctypes.CDLL(path)


@contextlib.contextmanager
def broken_capture():
    """A stream whose capture a synchronising call has invalidated: more work on it is refused until the block ends."""
    rt, s = cudart(), torch.cuda.Stream()
    handle = ctypes.c_void_p(s.cuda_stream)
    err = pa().new_error_word("cuda")
    torch.cuda.synchronize()
    assert rt.cudaStreamBeginCapture(handle, 2) == 0              # 2: relaxed, other streams are free
    try:
        assert pa().pa_read_error(err, s) == 3                    # PA_ERR_CUDA: a capturing stream does not synchronise
        yield s
    finally:
        ended = rt.cudaStreamEndCapture(handle, ctypes.byref(ctypes.c_void_p()))
        rt.cudaGetLastError()                                     # torch's own runtime forgets about it
        assert ended != 0


def leave_an_error():
    """The library's last call in this thread failed, and nothing is the matter any more."""
    with broken_capture():
        pass


def path_to_keep():
    """A tree, pa_keep_kv arguments and the pools after it; a second run would move other rows."""
    a = small_tree(N=1, nodes=6, seed=11)
    path = torch.tensor([[0, 2, 3, 5, -1, -1]], dtype=torch.int32, device="cuda")
    rest = (path.cpu().numpy(), [0, 6], a["block_tables"].cpu().numpy(), a["context_lens"].tolist(), 16)
    want = keep_ref(bits(a["k_pool"]), bits(a["v_pool"]), *rest)
    assert not np.array_equal(want[0], keep_ref(*want, *rest)[0])
    return a, (path, a["q_start"], a["context_lens"], a["block_tables"], a["k_pool"], a["v_pool"]), want


def test_an_old_error_is_not_taken_for_the_calls_own():
    a, keep, want = path_to_keep()
    clean = pa().pa_decode_tree(**a)
    leave_an_error()
    assert torch.equal(pa().pa_decode_tree(**a), clean)
    leave_an_error()
    pa().pa_keep_kv(*keep)
    torch.cuda.synchronize()
    assert np.array_equal(bits(a["k_pool"]), want[0]) and np.array_equal(bits(a["v_pool"]), want[1])
    # queries in place: rotated once
    freq, _ = pa().rope_inv_freq(64)
    q, kv = a["q"], a["q"][:, :2].contiguous()
    rope = (kv, kv, torch.arange(6, dtype=torch.int32, device="cuda") + 3, torch.arange(6, device="cuda"), a["k_pool"],
            a["v_pool"], freq)
    want_q = pa().pa_rope_append_kv(q, *rope)
    leave_an_error()
    assert torch.equal(pa().pa_rope_append_kv(q, *rope, out=q), want_q)
    # the calls that do not run twice, but failed for nothing
    leave_an_error()
    pa().pa_append_kv(kv, kv, rope[3], a["k_pool"], a["v_pool"])
    leave_an_error()
    one = pa().pa_decode(q[:1], a["k_pool"], a["v_pool"], a["block_tables"], a["context_lens"], 0.1)
    assert torch.isfinite(one.float()).all()


def test_a_failed_call_is_not_made_again(monkeypatch):
    # a launch that the runtime refuses is raised at once: a second try could run what the first left half done
    from paged_kv_cache_254_gb300 import ops
    tries = []
    for name in ("_keep_kv", "_rope_append_kv"):
        monkeypatch.setattr(ops, name, lambda *a, name=name: tries.append(name))
    a, keep, _ = path_to_keep()
    freq, _ = pa().rope_inv_freq(64)
    q, kv = a["q"], a["q"][:, :2].contiguous()
    rope = (kv, kv, torch.arange(6, dtype=torch.int32, device="cuda"), torch.arange(6, device="cuda"), a["k_pool"],
            a["v_pool"], freq)
    before = bits(a["k_pool"])
    with broken_capture() as s:
        for call in (lambda: pa().pa_keep_kv(*keep, stream=s), lambda: pa().pa_rope_append_kv(q, *rope, out=q, stream=s)):
            with pytest.raises(pa().PagedAttentionError) as e:
                call()
            assert e.value.status == 3
    torch.cuda.synchronize()
    assert not tries and np.array_equal(bits(a["k_pool"]), before)


# ---------------------------------------------------------------- several threads, several graphs
def chunk_args(a):
    """pa_decode_multi arguments over the same cache (chains are what a chunk sees)."""
    return {k: a[k] for k in ("q", "k_pool", "v_pool", "block_tables", "context_lens", "q_start", "scale")}


def test_threads_on_one_stream():
    # trees of several sizes (the cut pairs' states differ), through both host sides, and chunks
    from paged_kv_cache_254_gb300 import ops
    trees = [small_tree(N=n, nodes=p, Hq=8, Hkv=1, MB=40, seed=n + p) for n, p in ((3, 5), (9, 3), (2, 20))]
    for t in trees:
        t["context_lens"] += 500
    args = [tuple(t.values()) + (None, None, None) for t in trees]
    calls = [lambda a=a: ops._decode_tree(*a) for a in args]
    calls += [lambda t=t: pa().pa_decode_tree(**t) for t in trees]
    calls += [lambda t=t, p=p: pa().pa_decode_multi(**chunk_args(t), max_q_len=p) for t, p in zip(trees[:2], (5, 3))]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    outs = [[None] * 100 for _ in calls]

    def run(i):
        for k in range(100):
            outs[i][k] = calls[i]()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, x) for x in o)


@pytest.mark.parametrize("kind", ["decode", "multi"])
def test_captured_decodes_share_nothing(kind):
    # two captured calls replayed side by side, after eager calls that replaced the stream's workspace
    made = [small_tree(N=n, nodes=5, MB=60, seed=n) for n in (3, 6)]
    calls = []
    for t in made:
        t["context_lens"] += 800
        if kind == "multi":
            calls.append(lambda t=t: pa().pa_decode_multi(**chunk_args(t), max_q_len=5))
        else:
            one = t["q"][:t["block_tables"].shape[0]].contiguous()
            calls.append(lambda t=t, one=one: pa().pa_decode(one, t["k_pool"], t["v_pool"], t["block_tables"],
                                                             t["context_lens"], t["scale"]))
    want = [c() for c in calls]
    graphs, outs = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c())
        graphs.append(g)
    big = small_tree(N=64, nodes=12, Hq=32, Hkv=2, d=128, seed=5)
    pa().pa_decode_tree(**big)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


@pytest.mark.parametrize("kind", ["decode", "multi", "tree"])
def test_a_captured_branch_on_another_stream(kind):
    # a graph with two branches that run at once, each with calls that pick their own workspaces
    made = [small_tree(N=n, nodes=5, MB=60, seed=n) for n in (3, 6)]
    calls = []
    for t in made:
        t["context_lens"] += 800
        one = t["q"][:t["block_tables"].shape[0]].contiguous()
        calls.append({"tree": lambda s, t=t: pa().pa_decode_tree(**t, stream=s),
                      "multi": lambda s, t=t: pa().pa_decode_multi(**chunk_args(t), max_q_len=5, stream=s),
                      "decode": lambda s, t=t, one=one: pa().pa_decode(one, t["k_pool"], t["v_pool"], t["block_tables"],
                                                                       t["context_lens"], t["scale"], stream=s)}[kind])
    want = [c(None) for c in calls]
    torch.cuda.synchronize()
    side, graph, outs = torch.cuda.Stream(), torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        for _ in range(4):
            outs.append((0, calls[0](side)))
            outs.append((1, calls[1](None)))
        here.wait_stream(side)
    for _ in range(10):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i, o in outs)


# ---------------------------------------------------------------- rotary positions
@pytest.mark.parametrize("interleaved", [False, True])
def test_frequencies_that_are_not_finite(interleaved):
    H, d, T = 2, 64, 5
    freq, _ = pa().rope_inv_freq(d)
    bad = {3: float("inf"), 17: float("-inf"), 30: float("nan")}
    spoilt = freq.clone()
    for j, f in bad.items():
        spoilt[j] = f
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(T, H, d, device="cuda", generator=g).bfloat16() for _ in range(3))
    pos, slots = torch.tensor([0, 1, -5, 4096, 77], dtype=torch.int32, device="cuda"), torch.arange(T, device="cuda")
    pools = [torch.zeros(1, H, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    want = pa().pa_rope_append_kv(q, k, v, pos, slots, pools[0], pools[1], freq, interleaved=interleaved)
    got = pa().pa_rope_append_kv(q, k, v, pos, slots, pools[2], pools[3], spoilt, interleaved=interleaved)
    nan = torch.zeros(d, dtype=torch.bool, device="cuda")
    for j in bad:
        nan[[2 * j, 2 * j + 1] if interleaved else [j, j + d // 2]] = True
    for a, b in ((got, want), (pools[2][0, :, :T], pools[0][0, :, :T])):
        assert torch.isnan(a[..., nan]).all() and torch.equal(a[..., ~nan], b[..., ~nan])


# ---------------------------------------------------------------- large pools
@pytest.mark.parametrize("nodes", [2, 12, 40])
def test_blocks_past_32_bits_of_elements(nodes):
    # the same step over a small pool and over one whose blocks lie past element 2^32 (and byte 2^33)
    N, Hq, Hkv, d, B, MB = 2, 32, 8, 128, 16, 6
    a = small_tree(N=N, nodes=nodes, Hq=Hq, Hkv=Hkv, d=d, B=B, MB=MB, seed=nodes)
    a["context_lens"] += nodes                         # 50 tokens before each tree
    NB = (1 << 32) // (Hkv * B * d) + 40
    first = NB - N * MB
    assert first * Hkv * B * d > 1 << 32
    large = dict(a, block_tables=a["block_tables"] + first)
    for name in ("k_pool", "v_pool"):
        large[name] = torch.empty(NB, Hkv, B, d, dtype=torch.bfloat16, device="cuda")
        large[name][first:] = a[name]
    freq, _ = pa().rope_inv_freq(d)
    g = torch.Generator(device="cuda").manual_seed(1)
    T = N * nodes
    k, v = (torch.randn(T, Hkv, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    at = torch.cat([torch.arange(int(c) - nodes, int(c), device="cuda") for c in a["context_lens"]])
    tokens = torch.arange(T, device="cuda")
    path = torch.full((N, nodes), -1, dtype=torch.int32, device="cuda")
    path[:, 0] = nodes - 1

    def step(x):
        slots = x["block_tables"][tokens // nodes, at // B].long() * B + at % B
        q = pa().pa_rope_append_kv(x["q"], k, v, at.int(), slots, x["k_pool"], x["v_pool"], freq)
        out = pa().pa_decode_tree(**dict(x, q=q))
        pa().pa_keep_kv(path, x["q_start"], x["context_lens"], x["block_tables"], x["k_pool"], x["v_pool"])
        return q, out

    for x, y in zip(step(a), step(large)):
        assert torch.isfinite(x.float()).all() and torch.equal(x, y)
    for name in ("k_pool", "v_pool"):
        assert torch.equal(a[name], large[name][first:])
