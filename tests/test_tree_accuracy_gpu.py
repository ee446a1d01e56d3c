"""Accuracy of tree attention that one element's tolerance cannot show: a bias
common to all rows, and whole stages of a long context."""

import numpy as np
import pytest
import torch

from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def pa():
    import paged_kv_cache_254_gb300 as m
    return m


def scattered_table(N, blocks, seed):
    perm = np.random.default_rng(seed).permutation(N * blocks).astype(np.int32).reshape(N, blocks)
    return torch.from_numpy(perm).cuda()


def to_pool(x, table, B):
    """Tokens [N, ctx, Hkv, d] -> pool [NB, Hkv, B, d] by the table (ctx a multiple of B)."""
    N, ctx, H, d = x.shape
    pool = torch.empty(table.numel(), H, B, d, dtype=x.dtype, device="cuda")
    pool[table.long().flatten()] = x.cuda().view(N, ctx // B, B, H, d).transpose(2, 3).flatten(0, 1)
    return pool


@pytest.mark.parametrize("g,nodes", [(8, 2), (4, 16), (8, 16), (8, 64)])
@pytest.mark.parametrize("d", [64, 128])
def test_weights_are_not_biased(g, nodes, d):
    # Even keys are zero: score 0, the largest, weight exactly 1.  Odd keys score -a_r b_i, weights w in (0.5, 1).
    # V is c_j on even keys and -1 on odd ones, c_j near the mean weight: the sums cancel, so an error that all weights
    # share shows against outputs near 0, while the products' partial sums stay small.  Compared are means over N = 16
    # sequences of (got - the exact value rounded), which leaves the output's own rounding out.
    #
    # Weights as hi + lo: off by at most half a step of lo, 2^-17 for w < 1 (hi's step is 2^-8, lo below it has steps
    # of 2^-16 at most), symmetric and independent over n = 512 odd keys and 16 sequences (rows of one sequence are
    # taken as equal): 6 sigma of the mean over the weights' total L > 1.5 n is
    # 6 * 2^-17 / sqrt(3) / (1.5 sqrt(512) sqrt(16)) = 1.9e-7.  ex2.approx, 2^-22 of a weight at most, as if always to
    # one side: 2^-22 * n / L < 1.7e-7.  Partial sums below 16, 128 steps of 2^-24 of it over L > 768: 1.6e-7.  The
    # outputs, 16-bit steps u = 2^-13 (|out| < 2^-5) apart, that a mean error e moves over a step: e u / M variance
    # over M >= 16 * 16 * 64 elements, 6 sigma = 4.9e-7 at e = 1e-6 and M = 16384 (2.5e-7 at 65536).  1.0e-6 in all.
    # (Remainders cut instead of rounded are off by 2^-17.6 on average: 2.9e-6 here.)
    n, B, N = 512, 16, 16
    r = np.random.default_rng(100 * g + nodes + d)
    ctx = 2 * n
    bf = lambda x: torch.tensor(x, dtype=torch.float32).to(torch.bfloat16)
    b = bf(r.uniform(0.05, 0.7, (N, n)))
    a = bf(r.uniform(0.7, 0.9, (N, nodes, g)))
    w = np.exp(-a.double().numpy()[..., None] * b.double().numpy()[:, None, None])       # [N, nodes, g, n]
    assert (w > 0.5).all() and (w < 1).all()
    c = bf(w.mean() + r.uniform(-0.01, 0.01, d))
    pad = 64
    k = torch.zeros(N, ctx + pad, 1, d, dtype=torch.bfloat16)
    v = torch.zeros_like(k)
    k[:, 1:ctx:2, 0, 0] = -b
    v[:, 0:ctx:2, 0] = c
    v[:, 1:ctx:2, 0] = -1.0
    q = torch.zeros(N * nodes, g, d, dtype=torch.bfloat16)
    q[..., 0] = a.view(N * nodes, g)
    table = scattered_table(N, (ctx + pad) // B, 3)
    total = n + w.sum(-1)[..., None]
    exact = (n * c.double().numpy() - w.sum(-1)[..., None]) / total                      # [N, nodes, g, d]
    assert np.abs(exact).max() < 2.0 ** -5
    got = pa().pa_decode_tree(q.cuda(), to_pool(k, table, B), to_pool(v, table, B), table,
                              torch.full((N,), ctx + nodes, dtype=torch.int32, device="cuda"),
                              torch.arange(0, N * nodes + 1, nodes, dtype=torch.int32, device="cuda"),
                              torch.zeros(N * nodes, dtype=torch.int64, device="cuda"), 1.0, max_nodes=nodes)
    rounded = torch.from_numpy(exact).to(torch.bfloat16).double().numpy()
    bias = (got.double().cpu().numpy().reshape(exact.shape) - rounded).mean()
    assert abs(bias) < 1.0e-6, f"outputs are off by {bias:.2e} on average"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g,nodes", [(4, 4), (4, 30), (8, 40)])
def test_every_key_of_a_long_context_counts_once(g, nodes, d, dtype):
    # Keys are zero, so all weights are 1 and every sum is a whole number below 2^24: exact in fp32, whatever the order
    # and the splits.  Each 16 tokens have a 1 in one dim, in turn; a dim has at most 33 such groups, so one that is
    # lost or taken twice moves its output by 3 % or more.  What is left: 1 / L and the product with it (2 steps of 2^-24)
    # and the output's own rounding.
    B, ctxs = 16, [20000, 17 + nodes, 9000, 33000]
    N, longest = len(ctxs), 33008
    r = np.random.default_rng(g * nodes + d)
    group = np.arange(longest) // 16
    v = torch.zeros(N, longest, 1, d, dtype=dtype)
    v[:, torch.arange(longest), 0, torch.from_numpy(group % d)] = 1.0
    table = scattered_table(N, longest // B, nodes)
    sizes = [nodes, nodes, max(1, nodes // 2), nodes]
    starts = np.concatenate([[0], np.cumsum(sizes)])
    masks, exact = [], []
    for n, ctx in zip(sizes, ctxs):
        before = np.bincount(group[:ctx - n] % d, minlength=d)
        for i in range(n):
            m = int(r.integers(0, 1 << 62)) & ((1 << (i + 1)) - 1)
            seen = [ctx - n + j for j in range(n) if (m >> j) & 1]
            masks.append(m)
            exact.append((before + np.bincount(group[seen] % d, minlength=d)) / (ctx - n + len(seen)))
    q = torch.randn(int(starts[-1]), g, d, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    got = pa().pa_decode_tree(q, torch.zeros(table.numel(), 1, B, d, dtype=dtype, device="cuda"), to_pool(v, table, B), table,
                              torch.tensor(ctxs, dtype=torch.int32, device="cuda"),
                              torch.from_numpy(starts.astype(np.int32)).cuda(), torch.tensor(masks, device="cuda"), 0.1,
                              max_nodes=nodes)
    exact = np.repeat(np.array(exact)[:, None], g, 1)
    err = np.abs(got.double().cpu().numpy() - exact)
    # fp16 steps are 2^-24 below its normal range (rows of the short sequence are above it)
    bound = (torch.finfo(dtype).eps / 2 + 2.0 ** -22) * exact + (2.0 ** -25 if dtype == torch.float16 else 0)
    assert (err <= bound).all(), f"{np.max(err / np.maximum(exact, 1e-9)):.4f} of a value off"
