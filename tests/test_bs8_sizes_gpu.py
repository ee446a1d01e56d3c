"""Block-scaled calls at the ends of their sizes."""

import numpy as np
import pytest
import torch

from tests.bs8_bounds import rows_of
from tests.bs8_util import check, dev, pa, place, random_pool
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("most", [300, 2 ** 31 - 1])
def test_any_bound_for_many_sequences(most):
    r = np.random.default_rng(1)
    N, B, d = 40, 16, 64
    ctx, n = [int(c) for c in r.integers(30, 300, N)], [int(c) for c in r.integers(0, 25, N)]
    table, NB = place(r, ctx, B)
    pool = random_pool(r, NB, 1, B, d, "e4m3")
    qs = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    q = torch.from_numpy(r.standard_normal((int(qs[-1]), 16, d))).bfloat16()
    err = pa().new_error_word("cuda")
    out = pa().pa_decode_multi_bs8(q.cuda(), dev(pool), dev(table), dev(np.array(ctx, np.int32)), dev(qs), 0.125,
                                   max_q_len=most, err=err)
    assert int(err.item()) == 0
    check(out, *rows_of(q, pool, table, ctx, qs, 0.125, B, "e4m3"))


@pytest.mark.parametrize("call", ["pack", "unpack"])
def test_conversions_of_2_to_the_30_pieces(call):
    """2^20 pairs of 1024 heads, keys and values, are 2^31 warps: all but the last pair are out of range."""
    r = np.random.default_rng(2)
    H, B, d, n = 1024, 16, 64, 1 << 20
    pool = dev(random_pool(r, 1, H, B, d, "e4m3"))
    pairs = torch.full((n, 2), 5, dtype=torch.int32, device="cuda")
    pairs[-1] = 0
    k, v = (torch.randn(1, H, B, d, device="cuda").half() for _ in range(2))
    one = pairs[-1:].contiguous()
    if call == "pack":
        pa().pa_pack_blocks_bs8(pairs, k, v, pool)
        want = pa().bs8_pool(1, H, B, d)
        pa().pa_pack_blocks_bs8(one, k, v, want)
        keep = [*range(8), *range(32, pool.shape[2])]          # without the spare bytes
        assert torch.equal(pool[..., keep], want[..., keep])
    else:
        k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
        pa().pa_unpack_blocks_bs8(pairs, pool, k, v)
        pa().pa_unpack_blocks_bs8(one, pool, k2, v2)
        assert torch.equal(k, k2) and torch.equal(v, v2) and k2.any()


@pytest.mark.parametrize("most", [2 ** 31, 2 ** 32 + 1, 2 ** 63])
def test_bounds_past_32_bits(most):
    r = np.random.default_rng(3)
    ctx, n, B, d = [40, 200], [9, 30], 16, 64
    table, NB = place(r, ctx, B)
    qs = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    q, k, v = (torch.from_numpy(r.standard_normal((39, h, d))).half().cuda() for h in (4, 2, 2))
    args, pools, outs = (dev(table), dev(np.array(ctx, np.int32)), dev(qs)), [], []
    start = random_pool(r, NB, 2, B, d, "e4m3")
    for m in (30, most):
        pools.append(dev(start))
        err = pa().new_error_word("cuda")
        pa().pa_append_kv_bs8(k, v, *args, pools[-1], max_new=m, err=err)
        outs.append(pa().pa_decode_multi_bs8(q, pools[-1], *args, 0.1, max_q_len=m, err=err))
        assert int(err.item()) == 0
    assert torch.equal(*pools) and torch.equal(*outs)
