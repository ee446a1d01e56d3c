"""Bad blocks among the tokens of a chunk itself: the rows that see them are NaN, the others what they were."""

import numpy as np
import pytest
import torch

from oracle.bs8 import scales_of
from tests.bs8_bounds import rows_of
from tests.bs8_util import check, dev, pa, place, random_pool
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("B,d,dtype", [(16, 128, torch.bfloat16), (32, 64, torch.float16)])
@pytest.mark.parametrize("ctx,n,block", [(165, 7, 160), (165, 7, 96), (200, 50, 160), (200, 50, 192), (900, 300, 640),
                                         (900, 300, 880), (3000, 5, 2976)])
def test_rows_before_a_bad_block_are_untouched(B, d, dtype, ctx, n, block):
    """block: its first position.  Rows of one token, of one group and of one tile see it or do not."""
    r = np.random.default_rng(n + block)
    block -= block % B
    table, NB = place(r, [ctx, 40], B)
    pool = random_pool(r, NB, 2, B, d, "e4m3")
    qs = np.array([0, n, n + 3], np.int32)
    q = torch.from_numpy(r.standard_normal((n + 3, 16, d))).to(dtype)
    want, bound = rows_of(q, pool, table, [ctx, 40], qs, 0.1, B, "e4m3")
    sees = np.zeros(want.shape[:2], bool)
    sees[:n] = (np.arange(ctx - n, ctx) >= block)[:, None]

    def run(table, pool, bit, heads):
        err = pa().new_error_word("cuda")
        out = pa().pa_decode_multi_bs8(q.cuda(), dev(pool), dev(table), dev(np.array([ctx, 40], np.int32)), dev(qs), 0.1,
                                       max_q_len=n, err=err)
        bad = np.zeros_like(sees)
        bad[:, heads] = sees[:, heads]
        assert int(err.item()) == bit
        assert out.cpu()[torch.from_numpy(bad)].isnan().all()
        check(out.cpu()[torch.from_numpy(~bad)], want[~bad], bound[~bad])

    run(table, pool, 0, slice(0, 0))
    t = table.copy()
    t[0, block // B] = NB + 1
    run(t, pool, 1, slice(None))
    for s in (np.nan, np.inf, -0.5):
        for i in (0, 1):
            p = pool.copy()
            scales_of(p)[table[0, block // B], 1, i] = s
            run(table, p, 256, slice(8, 16))


@pytest.mark.parametrize("kind", ["decode", "chunk"])
def test_a_bad_id_says_nothing_of_other_blocks_scales(kind):
    """A block that no table names holds no scale: it is not read in place of one that is out of range."""
    r = np.random.default_rng(3)
    table, NB = place(r, [100, 50], 16)
    pool = random_pool(r, NB, 2, 16, 128, "e4m3")
    free = (set(range(NB)) - set(table[table < NB].tolist())).pop()
    table, pool = np.where(table == 0, free, np.where(table == free, 0, table)), pool.copy()   # block 0 is free now
    pool[[0, free]] = pool[[free, 0]]
    pool[0] = 0xFF
    assert not (table == 0).any()
    table[0, 2] = -1
    args = (dev(pool), dev(table.astype(np.int32)), dev(np.array([100, 50], np.int32)))
    q = torch.from_numpy(r.standard_normal((2, 8, 128))).bfloat16().cuda()
    err = pa().new_error_word("cuda")
    if kind == "decode":
        out = pa().pa_decode_bs8(q, *args, 0.1, err=err)
    else:
        out = pa().pa_decode_multi_bs8(q, *args, dev(np.array([0, 1, 2], np.int32)), 0.1, err=err)
    assert int(err.item()) == 1 and out[0].isnan().all() and not out[1].isnan().any()
