"""The bounds of the block-scaled attention tests see a lost piece, and agree with the oracle otherwise."""

import numpy as np
import pytest

from oracle.attention import decode_multi_ref
from oracle.bs8 import dequantized_pools
from tests.bs8_bounds import LONG, long_case, rows_of


@pytest.mark.parametrize("i", range(len(LONG)))
@pytest.mark.parametrize("values", ["random", "block by block"])
def test_outputs_are_the_oracles(i, values):
    q, pool, table, ctx, q_start, scale, B = long_case(i, values)
    want, bound = rows_of(q, pool, table, ctx, q_start, scale, B, "e4m3")
    ref = decode_multi_ref(q, *dequantized_pools(pool, B, q.shape[2], "e4m3"), table, ctx, q_start, scale)
    assert np.allclose(want, ref, rtol=1e-9, atol=1e-12 * np.abs(ref).max())
    assert (bound > 0).all() and (bound < np.abs(want).max(-1, keepdims=True)).all()


@pytest.mark.parametrize("i", range(len(LONG)))
def test_any_lost_block_is_beyond_the_bound(i):
    q, pool, table, ctx, q_start, scale, B = long_case(i, "block by block")
    want, bound = rows_of(q, pool, table, ctx, q_start, scale, B, "e4m3")
    r = np.random.default_rng(i)
    for b, c in enumerate(ctx):
        last = int(q_start[b + 1]) - 1                        # (a row is enough here)
        nb = -(-c // B)
        for lb in {0, nb - 1, *r.integers(0, nb, 3).tolist()}:
            got, _ = rows_of(q[last:last + 1], pool, table[b:b + 1], [c], [0, 1], scale, B, "e4m3", lost=[(0, lb)])
            over = np.abs(got[0] - want[last]) > 2 * bound[last]
            assert over.any(-1).all(), f"block {lb} of sequence {b}"   # in every head
