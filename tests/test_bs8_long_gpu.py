"""Long contexts over the block-scaled 8-bit cache, cut into many pieces: within each row's own bounds, under which no
lost block goes unseen (test_bs8_bounds.py)."""

import numpy as np
import pytest

from tests.bs8_bounds import LONG, long_case, rows_of
from tests.bs8_util import check, dev, pa
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("i", range(len(LONG)))
@pytest.mark.parametrize("values", ["random", "block by block"])
def test_no_piece_is_lost(i, values):
    q, pool, table, ctx, q_start, scale, B = long_case(i, values)
    args = (dev(pool), dev(table), dev(np.array(ctx, np.int32)))
    err = pa().new_error_word("cuda")
    if LONG[i][1] is None:
        out = pa().pa_decode_bs8(q.cuda(), *args, scale, err=err)
    else:
        out = pa().pa_decode_multi_bs8(q.cuda(), *args, dev(q_start), scale, err=err)
    assert int(err.item()) == 0
    check(out, *rows_of(q, pool, table, ctx, q_start, scale, B, "e4m3"), values)
