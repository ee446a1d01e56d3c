"""Attention over the block-scaled 8-bit cache where value scales are far apart, within bounds of each row's own."""

import numpy as np
import pytest
import torch

from oracle.bs8 import positions, scales_of
from tests.bs8_bounds import rows_of
from tests.bs8_util import check, dev, pa, place, random_pool
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def outputs(q, pool, table, ctx, q_start, scale, fmt, kind):
    args = (dev(pool), dev(table), dev(np.asarray(ctx, np.int32)))
    err = pa().new_error_word("cuda")
    if kind == "decode":
        out = pa().pa_decode_bs8(q.cuda(), *args, scale, kv_format=fmt, err=err)
    else:
        out = pa().pa_decode_multi_bs8(q.cuda(), *args, dev(q_start), scale, kv_format=fmt, err=err)
    assert int(err.item()) == 0
    return out


KINDS = [("decode", 1), ("chunk", 5), ("chunk", 40)]           # 40 tokens of 8 heads: groups of 256 rows


@pytest.mark.parametrize("kind,n", KINDS)
@pytest.mark.parametrize("fmt,B,d", [("e4m3", 16, 128), ("e5m2", 32, 64)])
@pytest.mark.parametrize("far", [30, 50, 90])
@pytest.mark.parametrize("loud", ["first", "last", "all over"])
def test_small_values_beside_large_ones_that_a_row_does_not_look_at(kind, n, fmt, B, d, far, loud):
    """Blocks whose value scale is 2^far times the others' and whose keys all but no weight falls on: what they add
    to the output is 2^-40 of the others' part, and must not cost that part its bits."""
    r = np.random.default_rng(far + n)
    ctx = [400, 64 + n]
    table, NB = place(r, ctx, B)
    pool = random_pool(r, NB, 2, B, d, fmt, spread=1.0)
    s = scales_of(pool)
    first = positions(B, d)[0][:, 0]
    one = 0x38 if fmt == "e4m3" else 0x3C
    s[..., 0] = 0.001 * 4 / (448 if fmt == "e4m3" else 57344)   # the other dimensions' part of a score: next to nothing
    pool[:, :, first] = one
    small = s[..., 1].copy()
    s[..., 1] = small * 2.0 ** (-far if far > 50 else -far // 2)
    for row, c in zip(table, ctx):
        nb = -(-c // B)
        at = {"first": [0], "last": [(c - n) // B - 1], "all over": range(0, (c - n) // B, 3)}[loud]
        for i in at:
            pool[row[i]][:, first] = one | 0x80
            s[row[i], :, 1] *= 2.0 ** far
        assert nb > len(at)
    q = torch.from_numpy(r.standard_normal((n * 2, 16, d))).bfloat16()
    # scores of +-e to the base 2 apart from the rest, 2 e = far + 40
    q[..., 0] = (far + 40) / 2 * np.log(2.0) / (0.001 * 4 / (448 if fmt == "e4m3" else 57344))
    q_start = np.array([0, n, 2 * n], np.int32)
    out = outputs(q, pool, table, ctx, q_start, 1.0, fmt, kind)
    want, bound = rows_of(q, pool, table, ctx, q_start, 1.0, B, fmt)
    assert (bound < np.abs(want).max(-1, keepdims=True) / 8).all()
    check(out, want, bound, f"{kind} {far} {loud}")


@pytest.mark.parametrize("kind,n", KINDS)
def test_blocks_of_zeros_before_large_values(kind, n):
    """The smallest scale (zeros as an append leaves them) in the first blocks, values of 2^25 behind them: the
    zeros' keys have their share of the softmax."""
    r = np.random.default_rng(n)
    ctx, B, d = [300, 200], 16, 128
    table, NB = place(r, ctx, B)
    pool = random_pool(r, NB, 2, B, d, "e4m3")
    s = scales_of(pool)
    s[..., 0] /= 16
    s[..., 1] *= 2.0 ** 25 / s[..., 1].max()
    for row in table:
        pool[row[:5], :, 32 + B * d:] = 0
        s[row[:5], :, 1] = 2.0 ** -126
    q = torch.from_numpy(r.standard_normal((n * 2, 16, d))).bfloat16()
    q_start = np.array([0, n, 2 * n], np.int32)
    out = outputs(q, pool, table, ctx, q_start, 0.1, "e4m3", kind)
    check(out, *rows_of(q, pool, table, ctx, q_start, 0.1, B, "e4m3"))
