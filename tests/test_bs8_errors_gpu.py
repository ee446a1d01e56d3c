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
