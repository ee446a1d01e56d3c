"""Inputs, oracle answers and bounds shared by the block-scaled 8-bit cache's GPU tests."""

import numpy as np
import torch

from oracle.attention import decode_multi_ref
from oracle.bs8 import dequantized_pools
from oracle.fp8 import max_finite

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def pa():
    import paged_kv_cache_254_gb300 as m
    return m


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def place(r, ctx, B, extra=3, poison=True):
    """Scattered blocks for contexts: a table [N, MB] whose unused entries are out of range, and the pool's size."""
    need = [-(-c // B) for c in ctx]
    NB = sum(need) + extra
    ids = list(r.permutation(NB))
    table = np.full((len(ctx), max(1, max(need, default=1))), NB + 7 if poison else 0, dtype=np.int32)
    for b, n in enumerate(need):
        table[b, :n] = [ids.pop() for _ in range(n)]
    return table, NB


def random_pool(r, NB, Hkv, B, d, fmt, spread=2.0, powers=False):
    """A pool of random finite codes, and scales that differ by up to 2^spread either way."""
    pool = np.zeros((NB, Hkv, 32 + 2 * B * d), dtype=np.uint8)
    n = 2 * B * d
    x = torch.from_numpy(r.standard_normal((NB, Hkv, n)).astype(np.float32) * max_finite(fmt) / 5)
    x = x.clamp(-max_finite(fmt), max_finite(fmt))
    t = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}[fmt]
    pool[..., 32:] = x.to(t).view(torch.uint8).numpy()
    e = r.uniform(-spread, spread, (NB, Hkv, 2))
    pool[..., :8].view(np.float32)[...] = np.exp2(np.round(e) if powers else e) * 4 / max_finite(fmt)
    return pool


def attention(q, pool, table, ctx, q_start, scale, B, fmt):
    """The oracle's outputs, and a bound for each of them.

    The bound: half a step of the output's type; a softmax weight is rounded to fp16 once, 2^-11 of it at
    most, and below fp16's normal range by 2^-25 of the row's largest contribution; a score is off by the
    tensor core's 32-bit sums, d / 16 truncations of 2^-23 of the sum of |q k| so far; the accumulations of
    weights and outputs lose 2^-23 of the sum of absolute terms at each of the context's 16-key steps."""
    d = q.shape[2]
    k, v = dequantized_pools(pool, B, d, fmt)
    want = decode_multi_ref(q, k, v, table, ctx, q_start, scale)
    size = decode_multi_ref(q, k, np.abs(v), table, ctx, q_start, scale)
    longest = max([1] + [int(c) for c in ctx])
    finite = np.isfinite(k).all(-1) & np.isfinite(v).all(-1)
    kmax = np.abs(np.where(finite[..., None], k, 0)).max() if k.size else 0.0
    vmax = np.abs(np.where(finite[..., None], v, 0)).max() if v.size else 0.0
    qsum = np.abs(q.detach().double().cpu().numpy()).sum(-1, keepdims=True)
    score = qsum * kmax * abs(scale) * (d // 16) * 2.0 ** -23
    steps = (longest / 16 + 2) * 2.0 ** -23
    half = torch.finfo(q.dtype).eps / 2
    bound = half * np.abs(want) + (2.0 ** -11 + 2 * score + 2 * steps) * size * (1 + half)
    return want, bound + longest * 2.0 ** -25 * vmax + torch.finfo(q.dtype).tiny


def check(got, want, bound, what=""):
    g = got.detach().double().cpu().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(want)), f"{what}: NaN in other places"
    real = ~np.isnan(want)
    over = np.where(real, np.abs(np.where(real, g - want, 0)) - np.where(real, bound, 1), -1)
    i = np.unravel_index(int(np.argmax(over)), over.shape) if over.size else None
    assert i is None or over[i] <= 0, f"{what}: at {i} got {g[i]}, want {want[i]}, bound {bound[i]}"
