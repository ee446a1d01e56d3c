"""The 8-bit cache with a scale for each block of tokens and KV head, as measured cases.

The pool is ``uint8 [NB, Hkv, 32 + 2 * B * d]``: per (block, KV head) the keys' and the values' scale
(fp32), 24 spare bytes, then the codes of B keys and of B values (E4M3 or E5M2, rows of d bytes whose
16-byte parts are permuted, see ``_places``).  Five calls use it:

* ``append`` -- new tokens' keys and values quantised into their blocks; a block whose largest value grows
  gets a larger scale (a power of two) and its older codes are rounded to it (``pa_append_kv_bs8``);
* ``decode`` -- attention of each sequence's newest token over the cache (``pa_decode_bs8``);
* ``chunk``  -- causal attention of a chunk of new tokens per sequence, of a few drafted ones or a whole
  prompt (``pa_decode_multi_bs8``);
* ``pack`` and ``unpack`` -- whole blocks of a 16-bit cache into the 8-bit one and back
  (``pa_pack_blocks_bs8``, ``pa_unpack_blocks_bs8``).

``run`` computes them from elementary torch operations, or (``own``) through the package.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
CODES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
EXPONENT = {"e4m3": 9, "e5m2": 16}           # largest = 0.875 * 2^exponent


def listed():
    serving = dict(q_heads=64, kv_heads=8, head_dim=128, block=16, dtype="bf16", format="e4m3")
    return [
        # one chat's newest token: the append of an interactive decode step
        dict(name="append_one_token", op="append", seqs=1, ctx_lo=4100, ctx_hi=4100, new_lo=1, new_hi=1, kv_heads=8,
             head_dim=128, block=16, dtype="bf16", format="e4m3"),
        # the decode benchmark's batch: one token a sequence, most into a block that has others
        dict(name="append_decode_batch", op="append", seqs=256, ctx_lo=1024, ctx_hi=8192, new_lo=1, new_hi=1,
             kv_heads=8, head_dim=128, block=16, dtype="bf16", format="e4m3"),
        # prompts of ragged lengths, the shortest one token
        dict(name="append_prompts", op="append", seqs=16, ctx_lo=2100, ctx_hi=8192, new_lo=1, new_hi=2047, kv_heads=8,
             head_dim=128, block=16, dtype="bf16", format="e4m3"),
        # one chat, a short context: latency
        dict(name="decode_one_sequence", op="decode", seqs=1, ctx_lo=700, ctx_hi=700, **{**serving, "q_heads": 32}),
        # short ragged contexts down to none, one query head per KV head, small heads, large blocks
        dict(name="decode_short_ragged", op="decode", seqs=13, ctx_lo=0, ctx_hi=2000, q_heads=8, kv_heads=8,
             head_dim=64, block=32, dtype="fp16", format="e5m2"),
        # the serving batch of the decode benchmark
        dict(name="decode_serving_batch", op="decode", seqs=256, ctx_lo=1024, ctx_hi=8192, **serving),
        # long contexts, a KV head for every query head
        dict(name="decode_long_multihead", op="decode", seqs=4, ctx_lo=24576, ctx_hi=32768,
             **{**serving, "kv_heads": 64}),
        # one chat's drafted tokens, verified in one pass
        dict(name="chunk_one_sequence", op="chunk", seqs=1, ctx_lo=700, ctx_hi=700, new_lo=8, new_hi=8,
             **{**serving, "q_heads": 32}),
        # a serving batch's drafted tokens, ragged
        dict(name="chunk_serving_batch", op="chunk", seqs=128, ctx_lo=1024, ctx_hi=8192, new_lo=1, new_hi=16,
             **serving),
        # a long prompt's chunk behind the chunks before it
        dict(name="chunk_long_prompt", op="chunk", seqs=1, ctx_lo=8192, ctx_hi=8192, new_lo=4096, new_hi=4096,
             **serving),
        # cold sequences' blocks of a 16-bit cache, packed to half their size
        dict(name="pack_cold_blocks", op="pack", blocks=4096, kv_heads=8, head_dim=128, block=16, dtype="bf16",
             format="e4m3"),
        # blocks taken back into a 16-bit cache, small heads
        dict(name="unpack_blocks", op="unpack", blocks=777, kv_heads=8, head_dim=64, block=32, dtype="fp16",
             format="e5m2"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["append", "append", "decode", "decode", "decode", "chunk", "chunk", "chunk", "pack", "unpack"])
    heads = rng.choice([1, 2, 4, 8, 16])
    shape = dict(kv_heads=heads, head_dim=rng.choice([64, 128, 128]), block=rng.choice([16, 32]),
                 dtype=rng.choice(["bf16", "fp16"]), format=rng.choice(["e4m3", "e4m3", "e5m2"]))
    if op in ("pack", "unpack"):
        return dict(op=op, blocks=_log(rng, 1, 32768 // heads), **shape)
    q_heads = heads * rng.choice([1, 2, 4, 8, 16])
    if op == "append":
        new = _log(rng, 1, 4096)
        hi = _log(rng, new, 16384)
        most = max(1, min(256, 16384 * 8 // heads // new, 4_000_000 // (heads * hi)))
        return dict(op=op, seqs=_log(rng, 1, most), ctx_lo=rng.randint(new, hi), ctx_hi=hi,
                    new_lo=rng.randint(1, new), new_hi=new, **shape)
    if op == "decode":
        hi = _log(rng, 1, 32768)
        # no more key rows than the largest listed cases
        return dict(op=op, seqs=_log(rng, 1, max(1, min(256, 8_000_000 // (hi * heads)))), ctx_lo=rng.randint(0, hi),
                    ctx_hi=hi, q_heads=q_heads, **shape)
    new = _log(rng, 1, 4096)
    hi = _log(rng, max(new, 40), 24000)
    # no more key rows, and no more products, than the largest listed cases
    most = min(256, 8_000_000 // (hi * heads), 2_000_000_000 // (new * hi * q_heads))
    while most < 1:
        new = max(1, new // 2)
        most = min(256, max(1, 8_000_000 // (hi * heads)), 2_000_000_000 // (new * hi * q_heads))
    return dict(op=op, seqs=_log(rng, 1, most), ctx_lo=rng.randint(new, hi), ctx_hi=hi, new_lo=rng.randint(1, new),
                new_hi=new, q_heads=q_heads, **shape)


# ---------------------------------------------------------------- structure: the case alone says the amounts
def _spread(lo, hi, n):
    """n whole numbers spread evenly over lo .. hi."""
    return np.linspace(lo, hi, n).round().astype(np.int64) if n > 1 else np.array([hi], dtype=np.int64)


def _lengths(case):
    """Context lengths and new tokens of the sequences (the short chunks at the long contexts)."""
    ctx = _spread(case["ctx_lo"], case["ctx_hi"], case["seqs"])
    if "new_hi" not in case:
        return ctx, np.ones_like(ctx)
    return ctx, _spread(case["new_lo"], case["new_hi"], case["seqs"])[::-1].copy()


def work(case):
    d, hkv, B = case["head_dim"], case["kv_heads"], case["block"]
    if case["op"] in ("pack", "unpack"):
        rows = case["blocks"] * hkv * B
        return {"bytes": rows * d * 6 + case["blocks"] * (8 + 8 * hkv), "flops": rows * d * 4}
    ctx, n = _lengths(case)
    T = int(n.sum())
    if case["op"] == "append":
        # the new rows in at 16 bits, out at 8, and the scales of the blocks that they fall into
        blocks = int(((ctx - 1) // B - (ctx - n) // B + 1).sum())
        return {"bytes": T * hkv * d * 6 + blocks * (8 * hkv + 4) + 8 * len(n), "flops": T * hkv * d * 4}
    hq = case["q_heads"]
    if case["op"] == "decode":
        n = (ctx > 0).astype(np.int64)
        T = case["seqs"]
    keys = int(ctx.sum())
    blocks = int((-(-ctx // B)).sum())
    seen = float((n * (ctx - (n - 1) / 2)).sum())              # (query token, key) pairs
    return {"bytes": keys * hkv * d * 2 + blocks * (8 * hkv + 4) + T * hq * d * 4 + 8 * len(ctx),
            "flops": 4 * d * hq * seen}


# ---------------------------------------------------------------- the pool
def _places(B, d):
    """Bytes of a piece's codes at which dimension i of key row r, and of value row r, stand: [2, B, d].  The 16-byte
    parts of a row are permuted, and with d 64 value rows 16 to 31 change places in pairs, so that a plain
    copy in shared memory is read without bank conflicts."""
    r, i = np.arange(B)[:, None], np.arange(d)[None, :]
    part, rest = i // 16, i % 16
    if d == 128:
        k = r * d + (part ^ (r & 7)) * 16 + rest
        v = r * d + (part ^ (2 * ((r >> 3) & 3))) * 16 + rest
    else:
        k = r * d + i
        v = (r ^ ((r >> 4) & 1)) * d + (part ^ (2 * ((r >> 3) & 1))) * 16 + rest
    return np.stack([k, B * d + v])


def _views(s):
    """The pool's codes [NB, Hkv, 2 * B * d] as 8-bit floats, and its scales [NB, Hkv, 2]."""
    return s["pool"][..., 32:].view(CODES[s["format"]]), s["pool"][..., :8].view(torch.float32)


# ---------------------------------------------------------------- inputs
def _place(rng, ctx, block):
    """Scattered blocks for sequences of ctx tokens: the table and the pool's size."""
    need = -(-ctx // block)
    NB = int(math.ceil(need.sum() * 1.1)) + 1
    ids = rng.permutation(NB)[:need.sum()]
    table = np.zeros((len(ctx), max(1, int(need.max()))), dtype=np.int32)
    table[np.arange(table.shape[1])[None, :] < need[:, None]] = ids
    return table, NB


def _normal(shape, dtype, gen):
    return torch.randn(shape, dtype=dtype, device="cuda", generator=gen)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _pool(NB, case, gen):
    """A pool in use: codes up to the format's largest, scales as appended values of size one or so leave them."""
    n, hkv, fmt = 2 * case["block"] * case["head_dim"], case["kv_heads"], case["format"]
    pool = torch.zeros((NB, hkv, 32 + n), dtype=torch.uint8, device="cuda")
    codes = torch.empty((NB, hkv, n), dtype=CODES[fmt], device="cuda")
    for lo in range(0, NB, 4096):
        part = codes[lo:lo + 4096]
        part.copy_((_normal(part.shape, torch.float32, gen) * (LARGEST[fmt] / 4.5)).clamp_(-LARGEST[fmt], LARGEST[fmt]))
    pool[..., 32:] = codes.view(torch.uint8)
    step = torch.randint(-2, 2, (NB, hkv, 2), device="cuda", generator=gen) + 3 - EXPONENT[fmt]
    pool[..., :8] = torch.exp2(step.float()).view(torch.uint8)
    return pool


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    d, hkv, B, dt = case["head_dim"], case["kv_heads"], case["block"], DTYPES[case["dtype"]]
    s = dict(case)
    s["places"] = _dev(_places(B, d))
    if case["op"] in ("pack", "unpack"):
        n = case["blocks"]
        NB8, NB16 = n + n // 8 + 1, n + n // 4 + 1
        a, b = rng.permutation(NB16)[:n], rng.permutation(NB8)[:n]
        s["pairs"] = _dev(np.stack([a, b] if case["op"] == "pack" else [b, a], 1).astype(np.int32))
        s["pool"] = _pool(NB8, case, gen)
        # heads, and blocks of tokens, differ in size
        size = torch.exp2(torch.rand((2, NB16, hkv, 1, 1), device="cuda", generator=gen) * 6 - 4)
        s["k_pool"], s["v_pool"] = ((_normal((NB16, hkv, B, d), torch.float32, gen) * size[i]).to(dt) for i in (0, 1))
        return s
    ctx, n = _lengths(case)
    at = rng.permutation(len(ctx))
    ctx, n = ctx[at], n[at]
    table, NB = _place(rng, ctx, B)
    s.update(table=_dev(table), ctx=_dev(ctx.astype(np.int32)), pool=_pool(NB, case, gen))
    T = int(n.sum())
    if case["op"] != "decode":
        s["q_start"] = _dev(np.concatenate([[0], n.cumsum()]).astype(np.int32))
    if case["op"] == "append":
        # the projection's output; k and v are views of it, and some heads are louder
        size = torch.exp2(torch.rand((T, 2 * hkv, 1), device="cuda", generator=gen) * 4 - 2)
        kv = (_normal((T, 2 * hkv, d), torch.float32, gen) * size).to(dt)
        s.update(k=kv[:, :hkv], v=kv[:, hkv:])
        return s
    rows = case["seqs"] if case["op"] == "decode" else T
    s.update(q=_normal((rows, case["q_heads"], d), dt, gen), scale=1 / math.sqrt(d))
    return s


# ---------------------------------------------------------------- the plain forms
def _steps(top, fmt):
    """The smallest power of two (2^-126 at least) that brings `top` into the format's range."""
    m, e = torch.frexp(top)
    e = e - EXPONENT[fmt] + (m > 0.875).int()
    return torch.ldexp(torch.ones_like(top), torch.where(top > 0, e, -126).clamp(min=-126))


def _round8(x, fmt):
    return x.clamp(-LARGEST[fmt], LARGEST[fmt]).to(CODES[fmt])


def _tops(x):
    """The largest finite absolute value over the last dimension."""
    x = x.abs()
    return torch.where(x.isfinite(), x, 0.0).amax(-1)


def _rows(s, codes, blocks):
    """Codes [n, Hkv, 2, B, d] of the given blocks in their plain order."""
    return codes[blocks][..., s["places"].reshape(-1)].unflatten(-1, s["places"].shape)


def _append(s):
    B, fmt = s["block"], s["format"]
    codes, scales = _views(s)
    start, ctx = s["q_start"].long(), s["ctx"].long()
    n = start.diff()
    t = torch.arange(s["k"].shape[0], device="cuda")
    b = torch.searchsorted(start, t, right=True) - 1
    pos = ctx[b] - n[b] + (t - start[b])
    block, off = s["table"].long()[b, pos // B], pos % B
    opens = (off == 0) | (t == start[b])                       # the first of the call's tokens in its block
    item = opens.long().cumsum(0) - 1
    x = torch.stack([s["k"], s["v"]], 2).float()               # [T, Hkv, 2, d]
    hit, first = block[opens], off[opens]
    old = torch.where(first[:, None, None] == 0, 0.0, scales[hit])
    top = torch.zeros_like(old).index_reduce_(0, item, _tops(x), "amax", include_self=True)
    new = torch.maximum(old, _steps(top, fmt))
    rows = _rows(s, codes.view(torch.uint8), hit).view(CODES[fmt]).float() * (old / new)[..., None, None]
    older = (torch.arange(B, device="cuda") < first[:, None])[:, None, None, :, None]
    out = torch.where(older, _round8(rows, fmt).view(torch.uint8), _rows(s, codes.view(torch.uint8), hit))
    out[item, :, :, off] = _round8(x / new[item][..., None], fmt).view(torch.uint8)
    flat = torch.empty_like(out.flatten(2))
    flat[..., s["places"].reshape(-1)] = out.flatten(2)
    codes.view(torch.uint8)[hit] = flat
    scales[hit] = new
    return {"codes": codes, "scales": scales}


def _values(s, blocks):
    """Keys and values [n, Hkv, 2, B, d] of the given blocks, in 32 bits."""
    codes, scales = _views(s)
    return _rows(s, codes.view(torch.uint8), blocks).view(CODES[s["format"]]).float() * scales[blocks][..., None, None]


def _padded_rows(s):
    """Row numbers [N, new] of each sequence's new tokens in the packed arrays (past its end: row 0), and which of
    them there are."""
    if s["op"] == "decode":
        rows = torch.arange(s["seqs"], device="cuda")[:, None]
        return rows, torch.ones_like(rows, dtype=torch.bool), torch.ones_like(s["ctx"]).long()
    i = torch.arange(s["new_hi"], device="cuda")
    n = s["q_start"].diff().long()
    real = i[None, :] < n[:, None]
    return torch.where(real, s["q_start"][:-1, None].long() + i, 0), real, n


def _attend(s):
    N, hkv, d = s["seqs"], s["kv_heads"], s["head_dim"]
    g = s["q_heads"] // hkv
    rows, real, n = _padded_rows(s)
    k, v = _values(s, s["table"].long()).permute(3, 0, 2, 1, 4, 5).flatten(3, 4)          # [N, hkv, L, d] each
    L = k.shape[2]
    q = s["q"][rows].float().reshape(N, -1, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(N, hkv, -1, d)
    p = q @ k.transpose(-1, -2) * s["scale"]                                              # [N, hkv, new * g, L]
    del k
    last = (s["ctx"].long() - n)[:, None] + torch.arange(rows.shape[1], device="cuda")     # each token's own position
    seen = torch.arange(L, device="cuda") <= torch.where(s["ctx"][:, None] > 0, last, -1)[..., None]
    p = p.masked_fill_(~seen.repeat_interleave(g, 1)[:, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    cached = torch.arange(L, device="cuda") < s["ctx"][:, None]
    o = p @ v.masked_fill(~cached[:, None, :, None], 0.0)
    o = torch.where(total > 0, o / total, 0.0)
    o = o.reshape(N, hkv, -1, g, d).permute(0, 2, 1, 3, 4).reshape(N, -1, hkv * g, d)
    return o[real].to(s["q"].dtype)


def _pack(s):
    fmt = s["format"]
    codes, scales = _views(s)
    src, dst = s["pairs"].long().T
    x = torch.stack([s["k_pool"][src], s["v_pool"][src]], 2).float()                      # [n, Hkv, 2, B, d]
    new = _steps(_tops(x.flatten(3)), fmt)
    flat = torch.empty(x.shape[:2] + (s["places"].numel(),), dtype=torch.uint8, device="cuda")
    flat[..., s["places"].reshape(-1)] = _round8(x / new[..., None, None], fmt).view(torch.uint8).flatten(2)
    codes.view(torch.uint8)[dst] = flat
    scales[dst] = new
    return {"codes": codes, "scales": scales}


def _unpack(s):
    src, dst = s["pairs"].long().T
    x = _values(s, src).to(s["k_pool"].dtype)
    s["k_pool"][dst], s["v_pool"][dst] = x[:, :, 0], x[:, :, 1]
    return {"k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def run(s):
    if not own:
        return {"append": _append, "decode": _attend, "chunk": _attend, "pack": _pack, "unpack": _unpack}[s["op"]](s)
    import paged_kv_cache_254_gb300 as pa
    if s["op"] == "decode":
        return pa.pa_decode_bs8(s["q"], s["pool"], s["table"], s["ctx"], s["scale"], kv_format=s["format"])
    if s["op"] == "chunk":
        return pa.pa_decode_multi_bs8(s["q"], s["pool"], s["table"], s["ctx"], s["q_start"], s["scale"],
                                      kv_format=s["format"], max_q_len=s["new_hi"])
    if s["op"] == "unpack":
        pa.pa_unpack_blocks_bs8(s["pairs"], s["pool"], s["k_pool"], s["v_pool"], kv_format=s["format"])
        return {"k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    if s["op"] == "append":
        pa.pa_append_kv_bs8(s["k"], s["v"], s["table"], s["ctx"], s["q_start"], s["pool"], kv_format=s["format"],
                            max_new=s["new_hi"])
    else:
        pa.pa_pack_blocks_bs8(s["pairs"], s["k_pool"], s["v_pool"], s["pool"], kv_format=s["format"])
    codes, scales = _views(s)
    return {"codes": codes, "scales": scales}


# ---------------------------------------------------------------- the definitions in 64 bits
def _grid(fmt):
    """The format's finite values that are not negative, ascending, from its fields."""
    bits, bias = (3, 7) if fmt == "e4m3" else (2, 15)
    top = np.array([(m / 2 ** bits if e == 0 else 1 + m / 2 ** bits) * 2.0 ** (max(e, 1) - bias)
                    for e in range(2 * bias + 2) for m in range(2 ** bits)])
    return torch.from_numpy(top[top <= LARGEST[fmt]]).cuda()


def _nearest(x, fmt):
    """The format's value nearest to each x, in 64 bits: the even one of two that are as near (their places in the
    list of values are their codes)."""
    grid = _grid(fmt)
    a = x.abs().clamp(max=float(grid[-1]))
    hi = torch.searchsorted(grid, a).clamp(1, len(grid) - 1)
    below, above = a - grid[hi - 1], grid[hi] - a
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return torch.where(up, grid[hi], grid[hi - 1]).copysign(x)


def _exact_scales(top, fmt):
    """The power of two for each largest value (64 bits)."""
    e = torch.log2(top / LARGEST[fmt]).ceil()
    e = e + (torch.exp2(e) * LARGEST[fmt] < top).double() - (torch.exp2(e - 1) * LARGEST[fmt] >= top).double()
    return torch.exp2(torch.where(top > 0, e, -126.0).clamp(min=-126.0))


def exact(case, seed):
    s = prepare(case, seed)
    B, d, fmt, hkv = case["block"], case["head_dim"], case["format"], case["kv_heads"]
    codes, scales = (x.double() for x in _views(s))
    where = s["places"]
    if case["op"] == "unpack":
        out = {"k_pool": s["k_pool"].double(), "v_pool": s["v_pool"].double()}
        src, dst = s["pairs"].long().unbind(1)
        rows = codes[src]
        for i, x in enumerate(out.values()):
            x[dst] = torch.stack([rows[:, :, where[i, r]] for r in range(B)], 2) * scales[src][:, :, i, None, None]
        return out
    if case["op"] == "pack":
        src, dst = s["pairs"].long().unbind(1)
        for i, pool in enumerate((s["k_pool"], s["v_pool"])):
            x = pool.double()[src]
            scale = _exact_scales(x.abs().amax((-1, -2)), fmt)
            new = codes[dst]
            for r in range(B):
                new[:, :, where[i, r]] = _nearest(x[:, :, r] / scale[..., None], fmt)
            codes[dst] = new
            scales[dst, :, i] = scale
        return {"codes": codes, "scales": scales}
    ctx, table = s["ctx"].tolist(), s["table"].tolist()
    if case["op"] == "append":
        start = s["q_start"].tolist()
        for b in range(case["seqs"]):
            first, row = ctx[b] - (start[b + 1] - start[b]), start[b]
            while first < ctx[b]:
                blk, lo = table[b][first // B], first % B
                hi = min(B, lo + ctx[b] - first)
                for i, x in enumerate((s["k"], s["v"])):
                    x = x[row:row + hi - lo].double()
                    scale = _exact_scales(x.abs().amax((0, 2)), fmt)
                    if lo > 0:
                        scale = torch.maximum(scale, scales[blk, :, i])
                        old = where[i, :lo].reshape(-1)
                        codes[blk][:, old] = _nearest(codes[blk][:, old] * (scales[blk, :, i] / scale)[:, None], fmt)
                    new = where[i, lo:hi].reshape(-1)
                    codes[blk][:, new] = _nearest((x / scale[None, :, None]).transpose(0, 1).flatten(1), fmt)
                    scales[blk, :, i] = scale
                first, row = first + hi - lo, row + hi - lo
        return {"codes": codes, "scales": scales}
    g = case["q_heads"] // hkv
    start = s["q_start"].tolist() if case["op"] == "chunk" else list(range(case["seqs"] + 1))
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    del codes
    codes8 = _views(s)[0]
    for b in range(case["seqs"]):
        lo, hi, c = start[b], start[b + 1], ctx[b]
        if c == 0:
            continue
        blocks = s["table"][b, :-(-c // B)].long()
        x = codes8.view(torch.uint8)[blocks].view(CODES[fmt]).double()
        k, v = (torch.stack([x[:, :, where[i, r]] for r in range(B)], 2) * scales[blocks][:, :, i, None, None]
                for i in (0, 1))
        k, v = (y.permute(1, 0, 2, 3).flatten(1, 2)[:, :c] for y in (k, v))
        behind = torch.arange(c, device="cuda") > torch.arange(c - (hi - lo), c, device="cuda")[:, None]
        for h in range(hkv):                                                 # a head at a time: long prompts
            q = s["q"][lo:hi, h * g:(h + 1) * g].double().transpose(0, 1)
            a = (q @ k[h].T * s["scale"]).masked_fill(behind, -math.inf).softmax(-1)
            out[lo:hi, h * g:(h + 1) * g] = (a @ v[h]).transpose(0, 1)
    return out
