"""What rounding its softmax weights to 16 bits costs a chunk's rows over the block-scaled 8-bit cache."""

import numpy as np
import pytest
import torch

from oracle.bs8 import positions, scales_of
from tests.bs8_bounds import rows_of
from tests.bs8_util import check, dev, pa, place
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def one_key(g, n, e):
    """Rows of 2 sequences, n tokens each, whose key 0 has score 0, key 70 score e(rows) and the others -e / 4 * 3,
    to the base 2."""
    r = np.random.default_rng(g + n)
    B, d, Hkv, fmt = 16, 128, 2, "e4m3"
    ctx = [128 + n, 140 + n]
    table, NB = place(r, ctx, B)
    pool = np.zeros((NB, Hkv, 32 + 2 * B * d), np.uint8)
    t = torch.from_numpy(r.standard_normal((NB, Hkv, B * d)).astype(np.float32) * 60).to(torch.float8_e4m3fn)
    pool[..., 32 + B * d:] = t.view(torch.uint8).numpy()
    scales_of(pool)[..., 0], scales_of(pool)[..., 1] = 1.0, 0.0123
    first = positions(B, d)[0][:, 0]                          # dimension 0 of the key rows
    pool[:, :, first] = 0xB4                                  # -0.75
    for row in table:
        pool[row[0]][:, first[0]] = 0x00
        pool[row[70 // B]][:, first[70 % B]] = 0x38           # 1
    q = torch.zeros(2 * n, g * Hkv, d, dtype=torch.float64)
    q[..., 0] = torch.from_numpy(e(r, q.shape[:2]) * np.log(2.0))
    q = q.half()
    q_start = np.array([0, n, 2 * n], np.int32)
    out = pa().pa_decode_multi_bs8(q.cuda(), dev(pool), dev(table), dev(np.array(ctx, np.int32)), dev(q_start), 1.0,
                                   kv_format=fmt)
    return out, *rows_of(q, pool, table, ctx, q_start, 1.0, B, fmt)


@pytest.mark.parametrize("g,n", [(4, 5), (8, 16), (8, 40)])
def test_a_row_of_one_key_does_not_depend_on_how_its_weight_is_rounded(g, n):
    """Key 0 (score 0) sets a row's reference, key 70 (score e to the base 2, 8 to 11.9) follows in the second half of
    the stage, where a weight of up to 2^12 leaves the reference where it is, and has over 0.98 of the softmax (the
    other keys' scores are -e / 4 * 3).  Numerator and denominator that hold the same weight give its value
    whatever the rounding; a weight rounded in one of them alone moves the whole row by up to 2^-11, in the mean square by
    2^-12.4 or so.

    Per row: c, the factor by which the output is off along the true one.  What remains in it is the
    outputs' own rounding, at most 2^-11 each way and uniform, so 2^-11 / 3^0.5 in the mean square for each of 128
    dimensions and 2^-11 / (3 * 128)^0.5 = 2.5e-5 for c, or a little more as the dimensions count by their squares
    (normal values: 3^0.5 of it, 4.3e-5, were all of the rounding's steps the widest); and of the key's own rounding
    what the other keys' share of 0.02 lets through, 0.02 * 2^-12 = 5e-6.  Over 40 rows and more 6e-5 is
    not reached (the rows' mean square varies by a sixth); a weight rounded in the numerator alone gives 1.5e-4."""
    out, want, _ = one_key(g, n, lambda r, size: r.uniform(8.0, 11.9, size))
    c = (out.double().cpu().numpy() * want).sum(-1) / (want * want).sum(-1) - 1
    assert c.size >= 40 and np.sqrt((c * c).mean()) < 6e-5


@pytest.mark.parametrize("g,n", [(4, 5), (8, 40)])
@pytest.mark.parametrize("lo,hi", [(11.5, 12.5), (12, 100), (100, 114), (113, 116), (115, 128), (126, 130), (140, 900)])
def test_scores_that_leave_the_reference_far_behind(g, n, lo, hi):
    """The weight of key 70 by the reference that key 0 has set is 2^lo to 2^hi: beyond 2^12, beyond the 2^115 where
    it can no longer be multiplied by 2^13, and beyond 2^128."""
    check(*one_key(g, n, lambda r, size: r.uniform(lo, hi, size)))
