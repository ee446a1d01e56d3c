"""What attention over the block-scaled 8-bit cache may be off by, row by row, from each row's own weights."""

import numpy as np
import torch

from oracle.bs8 import dequantized_pools, positions, scales_of
from tests.bs8_util import DTYPES, place, random_pool


def rows_of(q, pool, table, ctx, q_start, scale, B, fmt, lost=()):
    """The exact outputs [T, Hq, d] in 64 bits and a bound for each.  ``lost``: (sequence, block) pairs whose keys are
    left out, as by a merge that loses a piece (the mistakes that the tests are to see).

    With W_t = e^(s_t - max s) over the keys that a row sees, L = sum W_t, b_t and c_t the value scale and codes,
    w_t = W_t b_t and M = max w_t, the output is sum w_t c_t / L.  In units of w:
      * a weight is rounded to fp16 once: 2^-11 of it, or 2^-25 of M where it is subnormal beside the largest; a
        chunk's L adds up weights of 11 bits, 2^-11 of it at most;
      * a weight's exponent x_t = s_t + log2 b_t (to the base 2) is off by the tensor core's 32-bit sum of d products,
        (d / 16) 2^-23 sum |q k|, by the roundings of its factors and of itself, 2^-24 (3 |s_t| + |x_t|), and the
        exponential by 2^-21 of its value; log2 b_t by 2^-21 (1 + |log2 b_t|), in the numerator alone;
      * sums over n keys in 32 bits, sixteen at a time, lose 2^-23 of their absolute terms at each of n / 16 steps, and
        at each of as many pieces (a piece has 32 keys at least);
      * the output is rounded once."""
    k, v = dequantized_pools(pool, B, q.shape[2], fmt)
    vs = scales_of(pool)[..., 1].astype(np.float64)
    qn = q.detach().double().cpu().numpy()
    T, Hq, d = qn.shape
    Hkv = k.shape[1]
    g = Hq // Hkv
    want, bound = np.zeros((T, Hq, d)), np.zeros((T, Hq, d))
    half, tiny = torch.finfo(q.dtype).eps / 2, torch.finfo(q.dtype).tiny
    for b, c in enumerate(ctx):
        a, e = int(q_start[b]), int(q_start[b + 1])
        if c <= 0 or e <= a:
            continue
        c = int(c)
        blocks = np.asarray(table[b, :-(-c // B)])
        kept = np.ones(c, bool)
        for s, lb in lost:
            if s == b:
                kept[lb * B:(lb + 1) * B] = False
        seen = np.repeat((np.arange(c) <= np.arange(c - (e - a), c)[:, None]) & kept, g, 0)
        for h in range(Hkv):
            K, V = (x[blocks, h].reshape(-1, d)[:c] for x in (k, v))
            bt = np.repeat(vs[blocks, h], B)[:c]
            Q = qn[a:e, h * g:(h + 1) * g].reshape(-1, d)
            s2 = Q @ K.T * (scale * np.log2(np.e))
            lb = np.log2(np.where(bt > 0, bt, 2.0 ** -126))
            top = np.where(seen, s2, -np.inf).max(1, keepdims=True)
            W = np.where(seen, np.exp2(s2 - np.where(np.isfinite(top), top, 0)), 0.0)
            L = W.sum(1, keepdims=True)
            L[L == 0] = 1
            steps = 2 * (c / 16 + 2) * 2.0 ** -23
            eta = (abs(scale) * np.log2(np.e) * (d // 16) * 2.0 ** -23 * (np.abs(Q) @ np.abs(K).T)
                   + 2.0 ** -24 * (3 * np.abs(s2) + np.abs(s2 + lb))) * np.log(2) + 2.0 ** -21 + steps
            logs = 2.0 ** -21 * (1 + np.abs(lb)) * np.log(2)
            codes = np.abs(V) / np.where(bt > 0, bt, 1)[:, None]
            w = W * bt
            o = W @ V / L
            up = (w * (2.0 ** -11 + eta + logs)) @ codes / L
            up += 2.0 ** -25 * w.max(1, keepdims=True) * (seen.astype(float) @ codes) / L
            down = 2.0 ** -11 + (W * eta).sum(1, keepdims=True) / L
            err = up + np.abs(o) * down
            for x, y in ((want, o), (bound, err * (1 + half) + half * np.abs(o) + tiny)):
                x[a:e, h * g:(h + 1) * g] = y.reshape(e - a, g, d)
    return want, bound


# contexts that are cut into many pieces: (contexts, new tokens (None: a decode), Hq, Hkv, B, d, type)
LONG = [([20000], None, 8, 1, 16, 128, "bf16"), ([20000], None, 8, 1, 16, 128, "fp16"),
        ([9000, 11, 12000, 5000], None, 4, 4, 32, 64, "bf16"), ([20000], [5], 8, 1, 16, 128, "bf16"),
        ([9000, 40, 12000], [20, 3, 40], 8, 1, 16, 128, "fp16"), ([6000, 5000], [300, 17], 4, 4, 32, 64, "bf16")]


def block_by_block(r, pool, table, ctx, B, d):
    """Values by which every block shows: block i of a sequence has values in dimension i mod d alone, positive ones, so
    that a lost block takes a part of one dimension that no rounding takes; keys are small, the softmax nearly flat."""
    key, val = positions(B, d)
    s = scales_of(pool)
    s[..., 0] /= 64
    codes = pool[..., val]                                     # [NB, Hkv, B, d]
    codes &= 0x7F
    shown = np.zeros((len(pool), d), bool)
    for row, c in zip(table, ctx):
        n = -(-int(c) // B)
        shown[row[:n], np.arange(n) % d] = True
    codes[~np.broadcast_to(shown[:, None, None], codes.shape)] = 0
    # (rows past the context are not cached; small codes give way to 1.0, so that each block counts)
    codes[np.broadcast_to(shown[:, None, None], codes.shape) & (codes < 0x38)] = 0x38
    pool[..., val] = codes


def long_case(i, values):
    """Case LONG[i] with values "random" or "block by block": (q, pool, table, ctx, q_start, scale, B)."""
    ctx, n, Hq, Hkv, B, d, dtype = LONG[i]
    r = np.random.default_rng(100 + i)
    table, NB = place(r, ctx, B)
    pool = random_pool(r, NB, Hkv, B, d, "e4m3", spread=4.0 if values == "random" else 1.0)
    if values != "random":
        block_by_block(r, pool, table, ctx, B, d)
    q_start = np.concatenate([[0], np.cumsum(n or [1] * len(ctx))]).astype(np.int32)
    q = torch.from_numpy(r.standard_normal((int(q_start[-1]), Hq, d))).to(DTYPES[dtype])
    return q, pool, table, ctx, q_start, 1 / np.sqrt(d), B
