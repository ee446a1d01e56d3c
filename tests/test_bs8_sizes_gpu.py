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
