"""Pins of the block-scaled 8-bit cache's oracle: the layout, the scales' rule by
hand, appends in any cut, and round trips."""

import numpy as np
import pytest

from oracle.bs8 import (append_bs8_ref, dequantized_pools, needed_scale, pack_bs8_ref, positions, scales_of)
from oracle.fp8 import max_finite


@pytest.mark.parametrize("B", [16, 32])
@pytest.mark.parametrize("d", [64, 128])
def test_every_byte_of_a_piece_has_one_place(B, d):
    key, val = positions(B, d)
    assert sorted(np.concatenate([key.ravel(), val.ravel()])) == list(range(32, 32 + 2 * B * d))
    assert ((key - 32) // (B * d) == 0).all() and ((val - 32) // (B * d) == 1).all()
    for at in (key, val):                                    # 16 dimensions stay together and aligned
        parts = at.reshape(B, d // 16, 16)
        assert (parts == parts[..., :1] + np.arange(16)).all() and (parts[..., 0] % 16 == 0).all()


def test_places_by_hand():
    key, val = positions(16, 128)
    assert key[3, 0] == 32 + 3 * 128 + 3 * 16 and key[9, 17] == 32 + 9 * 128 + 0 * 16 + 1
    assert val[3, 5] == 32 + 16 * 128 + 3 * 128 + 5 and val[9, 16] == 32 + 16 * 128 + 9 * 128 + 3 * 16
    key, val = positions(32, 64)
    assert key[5, 33] == 32 + 5 * 64 + 33 and val[17, 0] == 32 + 32 * 64 + 16 * 64 and val[8, 0] == 32 + 32 * 64 + 8 * 64 + 32


@pytest.mark.parametrize("top,fmt,want", [
    (448.0, "e4m3", 1.0), (448.5, "e4m3", 2.0), (1.0, "e4m3", 2.0 ** -8), (0.875, "e4m3", 2.0 ** -9),
    (57344.0, "e5m2", 1.0), (3.0, "e5m2", 2.0 ** -14), (0.0, "e4m3", 2.0 ** -126), (1e-40, "e5m2", 2.0 ** -126),
    (3e38, "e4m3", 2.0 ** 120),
])
def test_scales_by_hand(top, fmt, want):
    assert needed_scale([0.0, -top, np.inf, np.nan], fmt) == np.float32(want)
    assert top <= max_finite(fmt) * want


def _append(parts, B=16, d=64, fmt="e4m3", start=0):
    """A sequence's rows appended part by part; the pool's values."""
    pool = np.zeros((8, 2, 2 * B * d + 32), dtype=np.uint8)
    table, ctx = np.array([[5, 1, 6, 0]]), start
    for k, v in parts:
        ctx += len(k)
        pool = append_bs8_ref(pool, k, v, table, [ctx], [0, len(k)], B, fmt)
    ks, vs = dequantized_pools(pool, B, d, fmt)
    order = lambda x: x[[5, 1, 6, 0]].transpose(1, 0, 2, 3).reshape(2, -1, d)[:, :ctx]  # noqa: E731
    return order(ks), order(vs), pool


@pytest.mark.parametrize("fmt,half", [("e4m3", 2.0 ** -4), ("e5m2", 2.0 ** -3)])
def test_appended_values_are_within_half_a_step(fmt, half):
    r = np.random.default_rng(1)
    k, v = r.standard_normal((2, 40, 2, 64)).astype(np.float32)
    for cut in ([40], [1] * 40, [7, 20, 13], [16, 16, 8]):
        at = np.cumsum([0] + cut)
        gk, gv, _ = _append([(k[a:b], v[a:b]) for a, b in zip(at, at[1:])], fmt=fmt)
        for got, x in ((gk, k), (gv, v)):
            want = x.transpose(1, 0, 2).astype(np.float64)
            # one rounding in the format's normal range; a few steps of its subnormals (2^-9 or 2^-16 of
            # a scale that is at most 2 max / F) below it
            tiny = 2.0 * np.abs(want).max() / max_finite(fmt) * (2.0 ** -9 if fmt == "e4m3" else 2.0 ** -16)
            assert (np.abs(got - want) <= half * np.abs(want) + 2 * tiny).all()


def test_one_append_equals_many_where_codes_are_normal():
    """Powers of two move codes by whole exponents: the cut of an append does not matter."""
    r = np.random.default_rng(2)
    k, v = np.exp2(r.uniform(-3, 3, (2, 33, 2, 64))).astype(np.float32)
    whole = _append([(k, v)])[2]
    single = _append([(k[i:i + 1], v[i:i + 1]) for i in range(33)])[2]
    assert np.array_equal(whole, single)


def test_a_first_slot_starts_a_block_afresh():
    k = np.full((3, 2, 64), 0.5, dtype=np.float32)
    used = np.full((8, 2, 2 * 16 * 64 + 32), 0x7E, dtype=np.uint8)
    scales_of(used)[...] = np.nan
    got = append_bs8_ref(used, k, k, np.array([[3]]), [3], [0, 3], 16, "e4m3")
    assert (scales_of(got)[3] == 2.0 ** -9).all()
    assert np.isnan(scales_of(got)[2]).all()
    assert (dequantized_pools(got, 16, 64, "e4m3")[0][3, :, :3] == 0.5).all()


def test_older_codes_follow_a_larger_scale():
    one, big = np.full((1, 2, 64), 1.0, np.float32), np.full((1, 2, 64), 100.0, np.float32)
    gk, _, pool = _append([(one, one), (big, one)])
    assert (gk[:, 0] == 1.0).all() and (np.abs(gk[:, 1] - 100) <= 100 * 2.0 ** -4).all()
    assert (scales_of(pool)[5, :, 0] == 0.25).all() and (scales_of(pool)[5, :, 1] == 2.0 ** -8).all()


def test_infinities_and_nan():
    k = np.ones((2, 2, 64), dtype=np.float32)
    k[0, 0, :3] = [np.inf, -np.inf, np.nan]
    gk, gv, _ = _append([(k, np.ones_like(k))])
    assert gk[0, 0, 0] == 448 * 2.0 ** -8 and gk[0, 0, 1] == -448 * 2.0 ** -8 and np.isnan(gk[0, 0, 2])
    assert (gv == 1).all()


@pytest.mark.parametrize("B,d", [(16, 128), (32, 64)])
def test_packing_is_an_append_of_whole_blocks(B, d):
    r = np.random.default_rng(3)
    kp, vp = r.standard_normal((2, 5, 2, B, d)).astype(np.float32)
    zero = np.zeros((6, 2, 2 * B * d + 32), dtype=np.uint8)
    got = pack_bs8_ref(zero, kp, vp, [[4, 1], [0, 3]], "e5m2")
    rows = [np.concatenate([p[4], p[0]], 1).transpose(1, 0, 2) for p in (kp, vp)]
    want = append_bs8_ref(zero, *rows, np.array([[1, 3]]), [2 * B], [0, 2 * B], B, "e5m2")
    assert np.array_equal(got, want)
