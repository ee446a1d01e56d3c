"""The block-scaled 8-bit cache on the GPU: appends, packing and copies are exact to the
byte; decode stays within bounds derived from its roundings."""

import numpy as np
import pytest
import torch

from oracle.bs8 import append_bs8_ref, dequantized_pools, pack_bs8_ref, scales_of
from tests.bs8_util import DTYPES, attention, check, dev, pa, place, random_pool
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

FORMATS = ["e4m3", "e5m2"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def f32(t):
    return t.detach().float().cpu().numpy()


def append_case(r, ctx, n, Hkv, d, B, dtype, fmt):
    table, NB = place(r, ctx, B)
    pool = random_pool(r, NB, Hkv, B, d, fmt, powers=True)
    T = int(np.sum(n))
    kv = torch.from_numpy(r.standard_normal((T, 2 * Hkv, d)) * np.exp2(r.uniform(-4, 4, (T, 2 * Hkv, 1)))).to(DTYPES[dtype])
    q_start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    return table, pool, kv, q_start


def run_append(table, pool, kv, q_start, ctx, fmt, Hkv, **kw):
    p, kv = dev(pool), kv.cuda()
    err = pa().new_error_word("cuda")
    pa().pa_append_kv_bs8(kv[:, :Hkv], kv[:, Hkv:], dev(table), dev(np.asarray(ctx, np.int32)), dev(q_start), p,
                          kv_format=fmt, err=err, **kw)
    return p.cpu().numpy(), int(err.item())


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("B", [16, 32])
@pytest.mark.parametrize("d", [64, 128])
def test_append_is_exact(fmt, dtype, B, d):
    r = np.random.default_rng(B + d)
    ctx = [1, 16, 17, 40, 100, 33, 5, 64, 0, 129]
    n = [1, 16, 1, 8, 70, 33, 2, 1, 0, 3]
    for Hkv in (1, 3):
        table, pool, kv, q_start = append_case(r, ctx, n, Hkv, d, B, dtype, fmt)
        want = append_bs8_ref(pool, f32(kv[:, :Hkv]), f32(kv[:, Hkv:]), table, ctx, q_start, B, fmt)
        got, err = run_append(table, pool, kv, q_start, ctx, fmt, Hkv)
        assert err == 0 and np.array_equal(got, want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_of_extreme_values(fmt):
    """Infinities, NaN, zeros, subnormals, the largest values; rows alone and beside ordinary ones."""
    r = np.random.default_rng(5)
    ctx, n, B, d = [20, 17, 3, 16, 40], [3, 1, 3, 16, 24], 16, 128
    table, pool, kv, q_start = append_case(r, ctx, n, 2, d, B, "bf16", fmt)
    kv[0, 0, :4] = torch.tensor([np.inf, -np.inf, np.nan, 1.0])
    kv[1, 1] = 0
    kv[3] = 0
    kv[4:7] *= 1e-38
    kv[7, :, ::2] = 3.3e38
    kv[9, 2] = np.nan
    kv[24:, 1] = np.inf
    want = append_bs8_ref(pool, f32(kv[:, :2]), f32(kv[:, 2:]), table, ctx, q_start, B, fmt)
    got, err = run_append(table, pool, kv, q_start, ctx, fmt, 2)
    t = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}[fmt]
    nan = [torch.from_numpy(x[..., 32:].copy()).view(t).float().isnan().numpy() for x in (got, want)]
    assert err == 0 and np.array_equal(*nan)
    assert np.array_equal(got[..., 32:][~nan[1]], want[..., 32:][~nan[1]])
    assert np.array_equal(got[..., :32], want[..., :32])


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_to_blocks_with_any_scale(fmt):
    """Scales that are no power of two, zero, subnormal and the largest."""
    r = np.random.default_rng(6)
    ctx, n, B, d = [20] * 8, [2] * 8, 16, 64
    table, pool, kv, q_start = append_case(r, ctx, n, 1, d, B, "fp16", fmt)
    for b, s in enumerate([0.3, 1.7, 0.0, 1e-40, 2.0 ** 127, 3.0e38, 2.0 ** -126, 0.0123]):
        scales_of(pool)[table[b, 1]] = s
    want = append_bs8_ref(pool, f32(kv[:, :1]), f32(kv[:, 1:]), table, ctx, q_start, B, fmt)
    got, err = run_append(table, pool, kv, q_start, ctx, fmt, 1)
    assert err == 0 and np.array_equal(got, want)


def test_append_by_any_cut_gives_the_same_normal_codes():
    r = np.random.default_rng(7)
    B, d, T = 16, 128, 75
    kv = torch.from_numpy(np.exp2(r.uniform(-3, 3, (T, 4, d)))).bfloat16()
    table, NB = place(r, [T], B)
    pools = []
    for cut in ([T], [1] * T, [30, 1, 44]):
        p, at = pa().bs8_pool(NB, 2, B, d), np.cumsum([0] + cut)
        for a, b in zip(at, at[1:]):
            x = kv[a:b].cuda()
            pa().pa_append_kv_bs8(x[:, :2], x[:, 2:], dev(table), dev(np.array([b], np.int32)),
                                  dev(np.array([0, b - a], np.int32)), p, max_new=int(b - a))
        pools.append(p.cpu().numpy())
    assert np.array_equal(pools[0], pools[1]) and np.array_equal(pools[0], pools[2])


def test_append_of_malformed_sequences():
    """Each bad sequence sets its bit and changes nothing; its neighbours are appended."""
    r = np.random.default_rng(8)
    B, d = 16, 64
    ctx, n = [20, 20, 20, 20], [4, 4, 4, 4]
    table, pool, kv, q_start = append_case(r, ctx, n, 2, d, B, "bf16", "e4m3")
    good = lambda skip: append_bs8_ref(  # noqa: E731
        pool, f32(kv[:, :2]), f32(kv[:, 2:]), table, [c if i not in skip else 0 for i, c in enumerate(ctx)],
        q_start, B, "e4m3") if not skip else _only(pool, kv, table, ctx, q_start, B, skip)
    for bad_ctx in (3, -1, 33):
        c = [20, bad_ctx, 20, 20]
        got, err = run_append(table, pool, kv, q_start, c, "e4m3", 2, max_new=4)
        assert err == 2 and np.array_equal(got, good({1}))
    t = table.copy()
    t[2, 1] = -5
    got, err = run_append(t, pool, kv, q_start, ctx, "e4m3", 2, max_new=4)
    assert err == 1 and np.array_equal(got, good({2}))
    got, err = run_append(table, pool, kv, q_start, ctx, "e4m3", 2, max_new=3)
    assert err == 2 and np.array_equal(got, pool)
    for s in (np.nan, np.inf, -1.0):
        p = pool.copy()
        scales_of(p)[table[3, 1]] = s
        # 20 tokens, 4 of them new: the block starts afresh, whatever its scale was
        got, err = run_append(table, p, kv, q_start, ctx, "e4m3", 2, max_new=4)
        assert err == 0 and np.array_equal(got, good(set()))
        # 22 tokens, 4 new: it holds two older ones
        c = [20, 20, 20, 22]
        got, err = run_append(table, p, kv, q_start, c, "e4m3", 2, max_new=4)
        want = good({3})
        want[table[3, 1]] = p[table[3, 1]]
        assert err == 256 and np.array_equal(got, want)
    qs = np.array([0, 4, 2, 12, 99], np.int32)                # a negative chunk, rows past the end
    got, err = run_append(table, pool, kv, qs, ctx, "e4m3", 2, max_new=10)
    assert err == 2


def _only(pool, kv, table, ctx, q_start, B, skip):
    out = pool
    for b in range(len(ctx)):
        if b not in skip:
            a, e = q_start[b], q_start[b + 1]
            out = append_bs8_ref(out, f32(kv[a:e, :2]), f32(kv[a:e, 2:]), table[b:b + 1], ctx[b:b + 1], [0, e - a], B,
                                 "e4m3")
    return out


# ---------------------------------------------------------------- packing, unpacking, copies
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("B,d", [(16, 64), (16, 128), (32, 64), (32, 128)])
def test_pack_and_unpack_are_exact(fmt, dtype, B, d):
    r = np.random.default_rng(B * d)
    for Hkv, n in ((1, 1), (3, 7), (8, 29)):
        kp, vp = (torch.from_numpy(r.standard_normal((n + 4, Hkv, B, d)) * np.exp2(r.uniform(-5, 5, (n + 4, Hkv, 1, 1))))
                  .to(DTYPES[dtype]) for _ in range(2))
        pool = random_pool(r, n + 3, Hkv, B, d, fmt)
        pairs = np.stack([r.permutation(n + 4)[:n], r.permutation(n + 3)[:n]], 1).astype(np.int32)
        want = pack_bs8_ref(pool, f32(kp), f32(vp), pairs, fmt)
        p, err = dev(pool), pa().new_error_word("cuda")
        pa().pa_pack_blocks_bs8(dev(pairs), kp.cuda(), vp.cuda(), p, kv_format=fmt, err=err)
        assert int(err.item()) == 0 and np.array_equal(p.cpu().numpy(), want)
        back = pairs[:, ::-1].copy()
        k2, v2 = kp.cuda(), vp.cuda()
        pa().pa_unpack_blocks_bs8(dev(back), p, k2, v2, kv_format=fmt, err=err)
        for got, was, val in ((k2, kp, dequantized_pools(want, B, d, fmt)[0]), (v2, vp, dequantized_pools(want, B, d, fmt)[1])):
            exp = was.clone()
            exp[back[:, 1].astype(np.int64)] = torch.from_numpy(val[back[:, 0]]).float().to(DTYPES[dtype])
            assert torch.equal(got.cpu(), exp)
        assert int(err.item()) == 0


def test_bad_pairs_and_scales():
    r = np.random.default_rng(9)
    kp, vp = (torch.from_numpy(r.standard_normal((4, 2, 16, 64))).half().cuda() for _ in range(2))
    pool = dev(random_pool(r, 5, 2, 16, 64, "e4m3"))
    before = pool.clone()
    for pair in ([4, 0], [-1, 0], [0, 5], [0, -3]):
        err = pa().new_error_word("cuda")
        pa().pa_pack_blocks_bs8(dev(np.array([pair], np.int32)), kp, vp, pool, err=err)
        assert int(err.item()) == 8 and torch.equal(pool, before)
    for pair in ([5, 0], [0, 4], [-1, 1]):
        err = pa().new_error_word("cuda")
        k0 = kp.clone()
        pa().pa_unpack_blocks_bs8(dev(np.array([pair], np.int32)), pool, kp, vp, err=err)
        assert int(err.item()) == 8 and torch.equal(kp, k0)
    pa().bs8_scales(pool)[1, 1, 0] = -1.0
    err = pa().new_error_word("cuda")
    pa().pa_unpack_blocks_bs8(dev(np.array([[1, 2]], np.int32)), pool, kp, vp, err=err)
    assert int(err.item()) == 256 and kp[2, 1].isnan().all() and not kp[2, 0].isnan().any() and not vp.isnan().any()


@pytest.mark.parametrize("B,d", [(16, 64), (32, 128)])
def test_copies_take_the_scales_along(B, d):
    r = np.random.default_rng(10)
    pool = random_pool(r, 9, 3, B, d, "e5m2")
    want = pool.copy()
    want[[5, 7]] = pool[[1, 1]]
    p = dev(pool)
    pa().pa_copy_blocks_bs8(dev(np.array([[1, 5], [1, 7], [2, 2]], np.int32)), p)
    assert np.array_equal(p.cpu().numpy(), want)


# ---------------------------------------------------------------- decode
EDGE = [1, 2, 15, 16, 17, 0, 33, 100, 513, 1000, 3001]


def decode_case(r, ctx, Hq, Hkv, B, d, dtype, fmt, q_mult=1.0, **kw):
    table, NB = place(r, ctx, B)
    pool = random_pool(r, NB, Hkv, B, d, fmt, **kw)
    q = (torch.from_numpy(r.standard_normal((len(ctx), Hq, d))) * q_mult).to(DTYPES[dtype])
    return table, pool, q


def run_decode(table, pool, q, ctx, scale, fmt, err=None, **kw):
    return pa().pa_decode_bs8(q.cuda(), dev(pool), dev(table), dev(np.asarray(ctx, np.int32)), scale, kv_format=fmt,
                              err=err, **kw)


def decode_matches(table, pool, q, ctx, scale, B, fmt, what=""):
    starts = np.cumsum([0] + [int(c > 0) for c in ctx])       # rows of sequences that hold something
    rows = [i for i, c in enumerate(ctx) if c > 0]
    want, bound = attention(q[rows], pool, table, ctx, starts, scale, B, fmt)
    err = pa().new_error_word("cuda")
    out = run_decode(table, pool, q, ctx, scale, fmt, err=err)
    assert int(err.item()) == 0
    check(out[rows], want, bound, what)
    assert (out[[i for i, c in enumerate(ctx) if c == 0]] == 0).all()
    return out


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("B", [16, 32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [1, 4, 8, 16])
def test_decode_matches_oracle(fmt, dtype, B, d, g):
    r = np.random.default_rng(g + B + d)
    table, pool, q = decode_case(r, EDGE, 2 * g, 2, B, d, dtype, fmt)
    decode_matches(table, pool, q, EDGE, 1 / np.sqrt(d), B, fmt, f"{fmt} {dtype} B{B} d{d} g{g}")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("case", ["peaked", "negative", "flat", "one", "loud", "quiet", "far", "silent", "zero_k"])
def test_decode_of_unusual_values(fmt, case):
    """Peaked softmaxes, scales and queries of any size, blocks that are all but zero."""
    r = np.random.default_rng(11)
    ctx, B, d = [700, 40, 3], 16, 128
    mult = {"peaked": 16.0, "loud": 2.0 ** 60, "quiet": 2.0 ** -60}.get(case, 1.0)
    scale = {"negative": -0.1, "flat": 0.0, "loud": 2.0 ** -64, "quiet": 2.0 ** 57}.get(case, 1 / np.sqrt(d))
    table, pool, q = decode_case(r, ctx, 8, 2, B, d, "bf16", fmt, q_mult=mult, spread=12.0 if case == "far" else 2.0)
    s = scales_of(pool)
    if case == "one":
        s[...] = 1.0 / (448 if fmt == "e4m3" else 57344)
    if case == "far":
        s[..., 0] = s[..., 0].clip(0, 0.01 if fmt == "e4m3" else 1e-4)   # scores of a size that leaves several keys
    if case == "silent":
        # values of some blocks all zero (least scale), of others tiny: their tokens count in the softmax all the same
        for b in table[0, :44:3]:
            pool[b, :, 32 + B * d:] = 0
            s[b, :, 1] = 2.0 ** -126
        s[table[0, 1:44:3], :, 1] = 2.0 ** -40
        pool[table[1, 0], :, 32 + B * d:] = 0
        s[table[1, 0], :, 1] = 0.0
        pool[table[2, 0], :, 32 + B * d:] = 0
        s[table[2, 0], :, 1] = 2.0 ** -126
    if case == "zero_k":
        s[..., 0] = 0.0
    decode_matches(table, pool, q, ctx, scale, B, fmt, case)


def test_decode_of_long_split_contexts():
    r = np.random.default_rng(12)
    for ctx, Hq, Hkv, B, d in (([20000], 8, 1, 16, 128), ([9000, 11, 12000, 5000], 4, 4, 32, 64)):
        table, pool, q = decode_case(r, ctx, Hq, Hkv, B, d, "bf16", "e4m3", spread=4.0)
        decode_matches(table, pool, q, ctx, 1 / np.sqrt(d), B, "e4m3")


def test_decode_ignores_what_is_not_cached():
    """Slots past the context may hold NaN codes, and the spare bytes anything."""
    r = np.random.default_rng(13)
    ctx, B, d = [5, 17, 250], 16, 128
    table, pool, q = decode_case(r, ctx, 4, 2, B, d, "fp16", "e4m3")
    clean = run_decode(table, pool, q, ctx, 0.09, "e4m3")
    from oracle.bs8 import positions
    key, val = positions(B, d)
    for b, c in enumerate(ctx):
        for at in (key, val):
            pool[table[b, c // B]][:, at[c % B:].ravel()] = 0x7F
    pool[..., 8:32] = 0xFF
    unused = sorted(set(range(len(pool))) - set(table[table < len(pool)]))
    pool[unused] = 0xFF
    assert torch.equal(run_decode(table, pool, q, ctx, 0.09, "e4m3"), clean)


def test_decode_of_cached_nan_is_nan_where_it_is_seen():
    r = np.random.default_rng(14)
    ctx, B, d = [40, 40], 16, 128
    table, pool, q = decode_case(r, ctx, 4, 2, B, d, "bf16", "e4m3")
    from oracle.bs8 import positions
    pool[table[0, 1], 1, positions(B, d)[1][3, 7]] = 0x7F     # a value of head 1
    out = run_decode(table, pool, q, ctx, 0.1, "e4m3")
    assert out[0, 2:, 7].isnan().all() and out.isnan().sum() == 2


def test_decode_errors_poison_their_rows_alone():
    r = np.random.default_rng(15)
    ctx, B, d = [40, 50, 60, 70], 16, 128
    table, pool, q = decode_case(r, ctx, 4, 2, B, d, "bf16", "e4m3")
    clean = run_decode(table, pool, q, ctx, 0.1, "e4m3")

    def only(bad, heads, table=table, pool=pool, ctx=ctx, bit=0):
        err = pa().new_error_word("cuda")
        out = run_decode(table, pool, q, ctx, 0.1, "e4m3", err=err)
        assert int(err.item()) == bit and out[bad, heads].isnan().all()
        rest = torch.ones(out.shape[:2], dtype=torch.bool)
        rest[bad, heads] = False
        assert torch.equal(out[rest], clean[rest])

    t = table.copy()
    t[2, 1] = len(pool)
    only(2, slice(None), table=t, bit=1)
    only(1, slice(None), ctx=[40, -1, 60, 70], bit=2)
    only(1, slice(None), ctx=[40, 81, 60, 70], bit=2)
    for s in (np.nan, np.inf, -0.5):
        for i in (0, 1):
            p = pool.copy()
            scales_of(p)[table[3, 2], 1, i] = s
            only(3, slice(2, 4), pool=p, bit=256)


def test_decode_is_deterministic_and_placement_does_not_matter():
    r = np.random.default_rng(16)
    ctx, B, d = [900, 3000, 10, 1700], 16, 128
    table, pool, q = decode_case(r, ctx, 16, 2, B, d, "bf16", "e4m3")
    a = run_decode(table, pool, q, ctx, 0.09, "e4m3")
    assert torch.equal(a, run_decode(table, pool, q, ctx, 0.09, "e4m3"))
    moved = r.permutation(len(pool))
    t = np.where(table < len(pool), np.argsort(moved)[np.minimum(table, len(pool) - 1)], table).astype(np.int32)
    assert torch.equal(a, run_decode(t, pool[moved], q, ctx, 0.09, "e4m3"))


def test_blocks_past_32_bits_of_bytes():
    """A pool of more than 2^32 bytes: the last blocks are appended to, read, copied and unpacked."""
    B, d, Hkv = 16, 128, 8
    NB = (1 << 32) // (Hkv * (2 * B * d + 32)) + 40
    r = np.random.default_rng(17)
    p = torch.empty((NB, Hkv, 32 + 2 * B * d), dtype=torch.uint8, device="cuda")
    ids = np.array([[NB - 1, NB - 3, 2]], np.int32)
    kv = torch.from_numpy(r.standard_normal((40, 16, d))).bfloat16().cuda()
    ctx, qs = dev(np.array([40], np.int32)), dev(np.array([0, 40], np.int32))
    pa().pa_append_kv_bs8(kv[:, :8], kv[:, 8:], dev(ids), ctx, qs, p)
    small = pa().bs8_pool(4, Hkv, B, d)
    low = dev(np.array([[1, 2, 3]], np.int32))
    pa().pa_append_kv_bs8(kv[:, :8], kv[:, 8:], low, ctx, qs, small)
    keep = [*range(8), *range(32, small.shape[2])]           # without the spare bytes
    assert torch.equal(p[NB - 1][:, keep], small[1][:, keep])
    q = torch.from_numpy(r.standard_normal((1, 64, d))).bfloat16().cuda()
    assert torch.equal(pa().pa_decode_bs8(q, p, dev(ids), ctx, 0.1), pa().pa_decode_bs8(q, small, low, ctx, 0.1))
    pa().pa_copy_blocks_bs8(dev(np.array([[NB - 3, NB - 5]], np.int32)), p)
    assert torch.equal(p[NB - 5], p[NB - 3])
    k16, v16, k2, v2 = (torch.zeros((2, Hkv, B, d), dtype=torch.bfloat16, device="cuda") for _ in range(4))
    pa().pa_unpack_blocks_bs8(dev(np.array([[NB - 5, 1]], np.int32)), p, k16, v16)
    pa().pa_unpack_blocks_bs8(dev(np.array([[2, 1]], np.int32)), small, k2, v2)
    assert torch.equal(k16, k2) and torch.equal(v16, v2)
    # packed again (a smaller power of two may serve the rounded values) it stands for the same values
    pa().pa_pack_blocks_bs8(dev(np.array([[1, NB - 2]], np.int32)), k16, v16, p)
    pa().pa_unpack_blocks_bs8(dev(np.array([[NB - 2, 0]], np.int32)), p, k16, v16)
    assert torch.equal(k16[0], k2[1]) and torch.equal(v16[0], v2[1]) and k2[1].any()
