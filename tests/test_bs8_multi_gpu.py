"""Chunks of new tokens over the block-scaled 8-bit cache: outputs within bounds derived from
their roundings, at every arrangement of rows, split contexts, masks, and malformed chunks."""

import numpy as np
import pytest
import torch

from oracle.bs8 import positions, scales_of
from tests.bs8_util import DTYPES, attention, check, dev, pa, place, random_pool
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def chunk_case(r, ctx, n, Hq, Hkv, B, d, dtype, fmt, q_mult=1.0, **kw):
    table, NB = place(r, ctx, B)
    pool = random_pool(r, NB, Hkv, B, d, fmt, **kw)
    q_start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    q = (torch.from_numpy(r.standard_normal((int(q_start[-1]), Hq, d))) * q_mult).to(DTYPES[dtype])
    return table, pool, q, q_start


def run(table, pool, q, ctx, q_start, scale, fmt, **kw):
    return pa().pa_decode_multi_bs8(q.cuda(), dev(pool), dev(table), dev(np.asarray(ctx, np.int32)), dev(q_start),
                                    scale, kv_format=fmt, **kw)


def matches(table, pool, q, ctx, q_start, scale, B, fmt, what="", **kw):
    err = pa().new_error_word("cuda")
    out = run(table, pool, q, ctx, q_start, scale, fmt, err=err, **kw)
    assert int(err.item()) == 0
    want, bound = attention(q, pool, table, ctx, q_start, scale, B, fmt)
    check(out, want, bound, what)
    return out


# single tokens, empty chunks, whole prompts, chunks behind a context; ends inside blocks and stages
CTX = [1, 40, 128, 129, 0, 300, 17, 260]
NEW = [1, 3, 9, 1, 0, 5, 9, 2]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("B", [16, 32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [1, 8, 16])
def test_short_chunks_match_oracle(fmt, dtype, B, d, g):
    """Rows per pair: 9, 72 (both tiles take every other stage) and 144 (two tiles)."""
    r = np.random.default_rng(B + d + g)
    table, pool, q, q_start = chunk_case(r, CTX, NEW, 2 * g, 2, B, d, dtype, fmt)
    matches(table, pool, q, CTX, q_start, 1 / np.sqrt(d), B, fmt, f"{fmt} {dtype} B{B} d{d} g{g}")


@pytest.mark.parametrize("fmt,dtype,B,d,g", [("e4m3", "bf16", 16, 128, 8), ("e5m2", "fp16", 32, 64, 1),
                                             ("e4m3", "fp16", 32, 128, 4), ("e5m2", "bf16", 16, 64, 16)])
def test_prompts_match_oracle(fmt, dtype, B, d, g):
    """Chunks of hundreds of tokens: several groups of rows, the last one partly filled."""
    r = np.random.default_rng(g)
    ctx, n = [700, 130, 333, 515], [300, 130, 1, 257]
    table, pool, q, q_start = chunk_case(r, ctx, n, 2 * g, 2, B, d, dtype, fmt)
    matches(table, pool, q, ctx, q_start, 1 / np.sqrt(d), B, fmt)


@pytest.mark.parametrize("n", [1, 2, 16, 17, 32, 33, 127, 128, 129, 256, 257])
def test_row_counts_at_the_borders(n):
    """One query head per KV head: rows are tokens; borders of tiles and groups."""
    r = np.random.default_rng(n)
    ctx, new = [n, n + 100, n + 1], [n, n, max(1, n - 1)]
    table, pool, q, q_start = chunk_case(r, ctx, new, 3, 3, 16, 64, "bf16", "e4m3")
    matches(table, pool, q, ctx, q_start, 0.125, 16, "e4m3")


@pytest.mark.parametrize("ctx,n,Hq,Hkv", [([20000], [5], 8, 1), ([9000, 40, 12000], [20, 3, 40], 8, 1),
                                          ([6000, 5000], [300, 17], 4, 4)])
def test_long_split_contexts(ctx, n, Hq, Hkv):
    r = np.random.default_rng(len(ctx))
    table, pool, q, q_start = chunk_case(r, ctx, n, Hq, Hkv, 16, 128, "bf16", "e4m3", spread=4.0)
    matches(table, pool, q, ctx, q_start, 1 / np.sqrt(128), 16, "e4m3")


@pytest.mark.parametrize("case", ["peaked", "negative", "flat", "loud", "quiet", "far", "silent", "zero_k", "growing"])
@pytest.mark.parametrize("n", [[9, 3, 2], [90, 40, 3]])
def test_unusual_values(case, n):
    r = np.random.default_rng(11)
    ctx, B, d, fmt = [700, 40, 3], 16, 128, "e4m3"
    mult = {"peaked": 16.0, "loud": 2.0 ** 60, "quiet": 2.0 ** -60}.get(case, 1.0)
    scale = {"negative": -0.1, "flat": 0.0, "loud": 2.0 ** -64, "quiet": 2.0 ** 57}.get(case, 1 / np.sqrt(d))
    table, pool, q, q_start = chunk_case(r, ctx, n, 8, 2, B, d, "bf16", fmt, q_mult=mult,
                                         spread=12.0 if case == "far" else 2.0)
    s = scales_of(pool)
    if case == "far":
        s[..., 0] = s[..., 0].clip(0, 0.01)
    if case == "growing":                                     # the references rise along the context
        for i, b in enumerate(table[0, :44]):
            s[b, :, 0] *= 1 + i / 4
    if case == "silent":
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
    matches(table, pool, q, ctx, q_start, scale, B, fmt, case)


@pytest.mark.parametrize("n", [[5, 4, 7], [60, 30, 40]])
def test_slots_past_the_context_are_not_seen(n):
    r = np.random.default_rng(13)
    ctx, B, d = [70, 33, 250], 16, 128
    table, pool, q, q_start = chunk_case(r, ctx, n, 8, 2, B, d, "fp16", "e4m3")
    clean = run(table, pool, q, ctx, q_start, 0.09, "e4m3")
    for b, c in enumerate(ctx):
        for at in positions(B, d):
            pool[table[b, c // B]][:, at[c % B:].ravel()] = 0x7F
    pool[..., 8:32] = 0xFF
    pool[sorted(set(range(len(pool))) - set(table[table < len(pool)]))] = 0xFF
    assert torch.equal(run(table, pool, q, ctx, q_start, 0.09, "e4m3"), clean)


@pytest.mark.parametrize("fmt,code", [("e4m3", 0x7F), ("e4m3", 0xFF), ("e5m2", 0x7E), ("e5m2", 0xFC)])
@pytest.mark.parametrize("n", [9, 150])
def test_new_values_that_are_not_finite_spoil_the_rows_that_see_them(fmt, code, n):
    """A value of token 3 of the chunk, and a key of token 5: earlier rows are as they were."""
    r = np.random.default_rng(14)
    ctx, B, d, Hq = [300, 300], 16, 128, 8
    table, pool, q, q_start = chunk_case(r, ctx, [n, n], Hq, 2, B, d, "bf16", fmt)
    clean = run(table, pool, q, ctx, q_start, 0.1, fmt)
    t = 300 - n + 3
    pool[table[0, t // B], 1, positions(B, d)[1][t % B, 7]] = code
    out = run(table, pool, q, ctx, q_start, 0.1, fmt)
    assert torch.equal(out[:3], clean[:3]) and torch.equal(out[n:], clean[n:]) and torch.equal(out[:n, :4], clean[:n, :4])
    assert out[3:n, 4:].isnan().all()
    if fmt == "e4m3":
        t = 300 - n + 5
        pool[table[1, t // B], 0, positions(B, d)[0][t % B, 9]] = code
        out = run(table, pool, q, ctx, q_start, 0.1, fmt)
        assert torch.equal(out[n:n + 5], clean[n:n + 5]) and torch.equal(out[n:, 4:], clean[n:, 4:])
        assert out[n + 5:, :4].isnan().all()


@pytest.mark.parametrize("n", [4, 50])
def test_errors_poison_their_rows_alone(n):
    r = np.random.default_rng(15)
    ctx, B, d = [140, 150, 160, 170], 16, 128
    table, pool, q, q_start = chunk_case(r, ctx, [n] * 4, 4, 2, B, d, "bf16", "e4m3")
    want, bound = attention(q, pool, table, ctx, q_start, 0.1, B, "e4m3")

    def only(b, heads, bit, table=table, pool=pool, ctx=ctx, max_q_len=n):
        err = pa().new_error_word("cuda")
        out = run(table, pool, q, ctx, q_start, 0.1, "e4m3", err=err, max_q_len=max_q_len)
        rows = slice(b * n, (b + 1) * n)
        assert int(err.item()) == bit and out[rows, heads].isnan().all()
        rest = torch.ones(out.shape[:2], dtype=torch.bool)
        rest[rows, heads] = False                             # (where the list is cut depends on every context)
        check(out[rest], want[rest.numpy()], bound[rest.numpy()])

    t = table.copy()
    t[2, 1] = len(pool)
    only(2, slice(None), 1, table=t)
    for bad in (n - 1, -1, 177):
        only(1, slice(None), 2, ctx=[140, bad, 160, 170])
    for s in (np.nan, np.inf, -0.5):
        for i in (0, 1):
            p = pool.copy()
            scales_of(p)[table[3, 2], 1, i] = s
            only(3, slice(2, 4), 256, pool=p)
    err = pa().new_error_word("cuda")
    out = run(table, pool, q, ctx, q_start, 0.1, "e4m3", err=err, max_q_len=n - 1)   # every chunk too long
    assert int(err.item()) == 2 and out.isnan().all()


def test_rows_outside_every_chunk_stay_as_they_are():
    r = np.random.default_rng(16)
    ctx = [50, 60]
    for n in (5, 40):
        table, pool, q, q_start = chunk_case(r, ctx, [n, n], 16, 2, 16, 64, "fp16", "e4m3")
        q = torch.cat([q[:2], q, q[:4]])
        out = torch.full_like(q, 7.0).cuda()
        run(table, pool, q, ctx, q_start + 2, 0.125, "e4m3", out=out, max_q_len=n)
        assert (out[:2] == 7).all() and (out[-4:] == 7).all()
        want, bound = attention(q[2:-4], pool, table, ctx, q_start, 0.125, 16, "e4m3")
        check(out[2:-4], want, bound)


def test_chunks_agree_with_single_tokens():
    """A chunk of one token is a decode, up to the order of sums."""
    r = np.random.default_rng(17)
    ctx, B, d = [900, 33, 1, 2500], 16, 128
    table, pool, q, q_start = chunk_case(r, ctx, [1] * 4, 16, 2, B, d, "bf16", "e4m3")
    one = pa().pa_decode_bs8(q.cuda(), dev(pool), dev(table), dev(np.asarray(ctx, np.int32)), 0.09)
    many = run(table, pool, q, ctx, q_start, 0.09, "e4m3")
    want, bound = attention(q, pool, table, ctx, q_start, 0.09, B, "e4m3")
    check(one, want, bound)
    check(many, want, bound)


def test_deterministic_and_independent_of_placement():
    r = np.random.default_rng(18)
    ctx = [900, 3000, 10, 1700]
    for n in ([9, 16, 2, 1], [300, 20, 10, 77]):
        table, pool, q, q_start = chunk_case(r, ctx, n, 16, 2, 16, 128, "bf16", "e4m3")
        a = run(table, pool, q, ctx, q_start, 0.09, "e4m3")
        assert torch.equal(a, run(table, pool, q, ctx, q_start, 0.09, "e4m3"))
        moved = r.permutation(len(pool))
        t = np.where(table < len(pool), np.argsort(moved)[np.minimum(table, len(pool) - 1)], table).astype(np.int32)
        assert torch.equal(a, run(t, pool[moved], q, ctx, q_start, 0.09, "e4m3"))


def test_bounds_far_above_the_chunks():
    """max_q_len may be any upper bound."""
    r = np.random.default_rng(19)
    ctx, n = [200, 90], [7, 3]
    table, pool, q, q_start = chunk_case(r, ctx, n, 8, 2, 16, 128, "bf16", "e4m3")
    for most in (7, 16, 17, 1000, 2 ** 31 - 1):
        matches(table, pool, q, ctx, q_start, 0.09, 16, "e4m3", max_q_len=most)
