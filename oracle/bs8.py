"""The 8-bit cache with a scale for each block and KV head.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

The pages: 8-bit keys and values halve the cache (ontq "AI Inference Serving at
Scale", section 6); quantised formats carry scale factors per group
(letsbuildsolutions "How LLM Inference Engines Work", quantization).  They give no
rule for a group's scale.  Reading taken:

  * Group = one (block, KV head), keys and values apart.  The scale that values x need
    is the smallest power of two 2^e, e >= -126, with max |x| <= F 2^e over the finite x,
    F the format's largest value.
  * Appending raises the block's scale s to max(s, need), s counting as 0 when the
    block's first slot is written; the block's older codes c become code(c * (s / s')),
    one fp32 quotient and one fp32 product, when s' > s.  New codes are code(x / s'), one
    fp32 quotient.  code(): nearest, ties to even; infinities become the largest code.
  * Layout: a piece is the two scales (fp32), 24 spare bytes, B key rows of d codes, B
    value rows of d codes.  The 16-byte parts of a row are permuted (``positions``).
"""

from __future__ import annotations

import numpy as np

from .fp8 import decode_array, max_finite, quantize

HEAD = 32


def positions(block_size: int, d: int):
    """Byte offsets in a piece of (row, dim), for keys [B][d] and for values [B][d]."""
    key = np.zeros((block_size, d), dtype=np.int64)
    val = np.zeros((block_size, d), dtype=np.int64)
    for r in range(block_size):
        for c in range(d // 16):
            at = np.arange(16)
            if d == 128:
                kc, vr, vc = c ^ (r % 8), r, c ^ (2 * (r // 8 % 4))
            else:
                kc, vr, vc = c, r ^ (r // 16 % 2), c ^ (2 * (r // 8 % 2))
            key[r, 16 * c:16 * c + 16] = r * d + 16 * kc + at
            val[r, 16 * c:16 * c + 16] = block_size * d + vr * d + 16 * vc + at
    return HEAD + key, HEAD + val


def needed_scale(x, fmt: str) -> np.float32:
    """The power of two that the values need, by trying exponents upwards."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    x = x[np.isfinite(x)]
    top, e, most = (float(x.max()) if x.size else 0.0), -126, max_finite(fmt)
    while top > most * 2.0 ** e:
        e += 1
    return np.float32(2.0 ** e)


def _code(x, scale, fmt):
    """Codes of x / scale; infinities saturate."""
    big = np.finfo(np.float32).max
    x = np.asarray(x, dtype=np.float32)
    with np.errstate(over="ignore"):
        return quantize(np.where(np.isinf(x), np.copysign(big, x), x), scale, fmt)


def scales_of(pool):
    """The scales [NB][Hkv][2] as a writable view of the pool's bytes."""
    return pool[..., :8].view(np.float32)


def append_bs8_ref(pool, k_new, v_new, tables, context_lens, q_start, block_size, fmt):
    """New pool [NB][Hkv][P] with the sequences' last n_b tokens appended."""
    pool = np.array(pool, copy=True)
    d = k_new.shape[2]
    where = positions(block_size, d)
    scales = scales_of(pool)
    for b, ctx in enumerate(np.asarray(context_lens, dtype=np.int64)):
        rows = list(range(int(q_start[b]), int(q_start[b + 1])))
        pos = [int(ctx) - len(rows) + i for i in range(len(rows))]
        for lb in sorted({p // block_size for p in pos}):
            mine = [(r, p % block_size) for r, p in zip(rows, pos) if p // block_size == lb]
            blk, first = int(tables[b, lb]), mine[0][1]
            for i, new in enumerate((k_new, v_new)):
                for h in range(pool.shape[1]):
                    x = np.stack([np.asarray(new[r, h], dtype=np.float32) for r, _ in mine])
                    old = np.float32(0) if first == 0 else np.float32(scales[blk, h, i])
                    now = max(old, needed_scale(x, fmt))
                    piece = pool[blk, h]
                    if first > 0 and now > old:
                        at = where[i][:first]
                        c = decode_array(piece[at], fmt).astype(np.float32) * np.float32(old / now)
                        piece[at] = _code(c, 1.0, fmt)
                    piece[where[i][[o for _, o in mine]]] = _code(x, now, fmt)
                    scales[blk, h, i] = now
    return pool


def pack_bs8_ref(pool, k_pool, v_pool, pairs, fmt):
    """New pool with the 16-bit blocks src (values [NB][Hkv][B][d]) in its blocks dst."""
    pool = np.array(pool, copy=True)
    B, d = k_pool.shape[2:]
    where, scales = positions(B, d), scales_of(pool)
    for src, dst in np.asarray(pairs):
        for i, x in enumerate((k_pool, v_pool)):
            for h in range(pool.shape[1]):
                s = needed_scale(x[src, h], fmt)
                pool[dst, h][where[i]] = _code(x[src, h], s, fmt)
                scales[dst, h, i] = s
    return pool


def dequantized_pools(pool, block_size, d, fmt):
    """fp64 key and value pools in the 16-bit cache's layout [NB][Hkv][B][d]."""
    scales = scales_of(pool).astype(np.float64)
    return tuple(decode_array(pool[..., at], fmt) * scales[..., i, None, None]
                 for i, at in enumerate(positions(block_size, d)))
