"""The serving operators around a tree of drafted tokens, as measured cases.

One step of tree speculation over the paged cache makes four calls:

* ``append``  -- per-head norms and rotary positions of the drafted tokens' queries and keys, and the
  append of their keys and values to the pools, in one pass (``pa_rope_append_kv``);
* ``tree``    -- attention of every drafted token over its sequence's cache and its own ancestors
  (``pa_decode_tree``);
* ``verify``  -- the drafted path that the target model's tokens agree with (``pa_tree_verify``);
* ``keep``    -- the accepted tokens' keys and values moved to consecutive positions (``pa_keep_kv``).

``run`` computes them from elementary torch operations, or (``own``) through the package.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
VOCAB = 50000


def listed():
    return [
        # one sequence's newest token: the append of an interactive decode step
        dict(name="append_one_token", op="append", tokens=1, q_heads=32, kv_heads=8, head_dim=128, block=16,
             dtype="bf16", rotary=128, interleaved=False, norm=True, far=False),
        # a long prompt's chunk at far positions, frequencies scaled for a long context
        dict(name="append_prompt_chunk", op="append", tokens=8192, q_heads=64, kv_heads=8, head_dim=128, block=16,
             dtype="bf16", rotary=128, interleaved=False, norm=True, far=True),
        # a ragged batch with half of a small head rotated, pairs side by side
        dict(name="append_partial_pairs", op="append", tokens=1531, q_heads=8, kv_heads=8, head_dim=64, block=32,
             dtype="fp16", rotary=32, interleaved=True, norm=False, far=False),
        # one chat, a small tree: latency
        dict(name="tree_one_sequence", op="tree", seqs=1, ctx_lo=700, ctx_hi=700, nodes=8, ragged=False, q_heads=32,
             kv_heads=8, head_dim=128, block=16, dtype="bf16"),
        # short contexts, ragged trees (down to one token), one query head per KV head
        dict(name="tree_short_ragged", op="tree", seqs=12, ctx_lo=13, ctx_hi=2000, nodes=13, ragged=True, q_heads=8,
             kv_heads=8, head_dim=64, block=32, dtype="fp16"),
        # the serving batch of the decode benchmark, eight drafted tokens a sequence
        dict(name="tree_serving_batch", op="tree", seqs=256, ctx_lo=1024, ctx_hi=8192, nodes=8, ragged=False,
             q_heads=64, kv_heads=8, head_dim=128, block=16, dtype="bf16"),
        # the widest trees: 64 nodes, 512 query rows per KV head
        dict(name="tree_wide", op="tree", seqs=64, ctx_lo=1024, ctx_hi=8192, nodes=64, ragged=False, q_heads=64,
             kv_heads=8, head_dim=128, block=16, dtype="bf16"),
        # long contexts, a KV head for every query head
        dict(name="tree_long_multihead", op="tree", seqs=4, ctx_lo=24576, ctx_hi=32768, nodes=24, ragged=False,
             q_heads=64, kv_heads=64, head_dim=128, block=16, dtype="bf16"),
        # one chat's verification
        dict(name="verify_one_sequence", op="verify", seqs=1, nodes=8, ragged=False),
        # a serving batch of the widest trees
        dict(name="verify_batch", op="verify", seqs=256, nodes=64, ragged=True),
        # one chat's accepted path
        dict(name="keep_one_sequence", op="keep", seqs=1, nodes=8, accepted=4, q_heads=32, kv_heads=8, head_dim=128,
             block=16, dtype="bf16"),
        # a serving batch's accepted paths through wide trees
        dict(name="keep_batch", op="keep", seqs=256, nodes=64, accepted=12, q_heads=64, kv_heads=8, head_dim=128,
             block=16, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["append", "append", "tree", "tree", "tree", "verify", "keep"])
    if op == "verify":
        return dict(op=op, seqs=_log(rng, 1, 256), nodes=_log(rng, 1, 64), ragged=rng.random() < 0.5)
    heads = rng.choice([1, 2, 4, 8])
    shape = dict(q_heads=heads * rng.choice([1, 2, 4, 8, 16]), kv_heads=heads, head_dim=rng.choice([64, 128]),
                 block=rng.choice([16, 32]), dtype=rng.choice(["bf16", "fp16"]))
    if op == "append":
        d = shape["head_dim"]
        return dict(op=op, tokens=_log(rng, 1, 8192 * 80 // max(80, shape["q_heads"] + 2 * heads)), **shape,
                    rotary=rng.choice([d, d, d // 2, d // 4]), interleaved=rng.random() < 0.5,
                    norm=rng.random() < 0.6, far=rng.random() < 0.4)
    if op == "keep":
        nodes = _log(rng, 2, 64)
        return dict(op=op, seqs=_log(rng, 1, 256), nodes=nodes, accepted=min(nodes, 12, _log(rng, 1, 64)), **shape)
    nodes = _log(rng, 1, 64)
    hi = _log(rng, max(nodes, 40), 24000)
    # no more key rows, and no more products, than the largest listed cases
    per = max(1, hi * heads * max(1, shape["q_heads"] // heads * nodes // 32))
    return dict(op=op, seqs=_log(rng, 1, max(1, min(256, 9_500_000 // per))), ctx_lo=rng.randint(nodes, hi),
                ctx_hi=hi, nodes=nodes, ragged=rng.random() < 0.5, **shape)


# ---------------------------------------------------------------- structure: the case alone says the amounts
def _spread(lo, hi, n):
    """n whole numbers spread evenly over lo .. hi."""
    return np.linspace(lo, hi, n).round().astype(np.int64) if n > 1 else np.array([hi], dtype=np.int64)


def _counts(case):
    n = case["nodes"]
    return _spread(1, n, case["seqs"]) if case["ragged"] else np.full(case["seqs"], n, dtype=np.int64)


def work(case):
    op = case["op"]
    if op == "verify":
        n = _counts(case)
        # masks, drafted and target tokens in; the path and three numbers a sequence out
        return {"bytes": int(n.sum()) * 24 + case["seqs"] * (8 + 4 * case["nodes"] + 16), "flops": 0}
    d, hq, hkv = case["head_dim"], case["q_heads"], case["kv_heads"]
    if op == "append":
        t = case["tokens"]
        return {"bytes": t * ((2 * hq + 4 * hkv) * d * 2 + 12),
                "flops": t * (hq + hkv) * (3 * case["rotary"] + (4 * d if case["norm"] else 0))}
    if op == "keep":
        # K and V rows of the accepted tokens behind the first, read and written
        return {"bytes": case["seqs"] * ((case["accepted"] - 1) * hkv * d * 8 + 4 * case["nodes"] + 8), "flops": 0}
    ctx, n = _spread(case["ctx_lo"], case["ctx_hi"], case["seqs"]), _counts(case)
    rows = int(n.sum())
    keys = int(ctx.sum())
    return {"bytes": keys * hkv * d * 4 + rows * hq * d * 4 + rows * 8 + keys // case["block"] * 4,
            "flops": 4 * d * hq * float(n.mean()) * float((ctx - n.mean() / 2).clip(1).sum())}


# ---------------------------------------------------------------- inputs
def _trees(rng, n, nodes):
    """Ancestor masks [N, nodes] of random trees (node i's parent is an earlier node), and the parents."""
    N = len(n)
    parent = np.full((N, nodes), -1, dtype=np.int64)
    mask = np.zeros((N, nodes), dtype=np.uint64)
    mask[:, 0] = 1
    rows = np.arange(N)
    for i in range(1, nodes):
        parent[:, i] = rng.integers(max(0, i - 9), i, size=N)
        mask[:, i] = mask[rows, parent[:, i]] | np.uint64(1 << i)
    return mask, parent


def _packed(a, n):
    """The first n[b] entries of each row, end to end."""
    return a[np.arange(a.shape[1])[None, :] < n[:, None]]


def _place(rng, ctx, block):
    """Scattered blocks for sequences of ctx tokens: the table and the pool's size."""
    need = -(-ctx // block)
    NB = int(math.ceil(need.sum() * 1.1)) + 1
    ids = rng.permutation(NB)[:need.sum()]
    table = np.zeros((len(ctx), int(need.max())), dtype=np.int32)
    table[np.arange(table.shape[1])[None, :] < need[:, None]] = ids
    return table, NB


def _normal(shape, dtype, gen):
    return torch.randn(shape, dtype=dtype, device="cuda", generator=gen)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op == "verify":
        n = rng.permutation(_counts(case))
        mask, parent = _trees(rng, n, case["nodes"])
        N = len(n)
        draft = rng.integers(0, VOCAB, size=mask.shape)
        target = rng.integers(0, VOCAB, size=mask.shape)
        # the target model agrees with some child of most nodes
        for i in range(1, case["nodes"]):
            hit = rng.random(N) < 0.6
            target[hit, parent[hit, i]] = draft[hit, i]
        start = np.concatenate([[0], n.cumsum()])
        s.update(masks=_dev(_packed(mask, n).astype(np.int64)), draft=_dev(_packed(draft, n)),
                 target=_dev(_packed(target, n)), q_start=_dev(start.astype(np.int32)),
                 ctx=_dev((n + rng.integers(0, 4096, size=N)).astype(np.int32)))
        return s
    d, hq, hkv, B, dt = case["head_dim"], case["q_heads"], case["kv_heads"], case["block"], DTYPES[case["dtype"]]
    if op == "append":
        T = case["tokens"]
        NB = T // B + 17
        qkv = _normal((T, (hq + 2 * hkv) * d), dt, gen)      # the projection's output; q, k, v are views of it
        half = case["rotary"] // 2
        freq = 10000.0 ** (-np.arange(half) / max(half, 1))
        if case["far"]:                                       # low frequencies stretched for a long context
            freq = np.where(np.arange(half) * 2 > half, freq / 8, freq)
        base = int(rng.integers(0, 1_000_000 if case["far"] else 4096))
        s.update(q=qkv[:, :hq * d].unflatten(1, (hq, d)), k=qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
                 v=qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d)),
                 positions=_dev((base + np.arange(T)).astype(np.int32)),
                 slots=_dev(rng.permutation(NB * B)[:T].astype(np.int64)),
                 inv_freq=_dev(freq.astype(np.float32)), scale=1.2 if case["far"] else 1.0,
                 qw=1 + 0.1 * _normal((d,), dt, gen) if case["norm"] else None,
                 kw=1 + 0.1 * _normal((d,), dt, gen) if case["norm"] else None,
                 k_pool=_normal((NB, hkv, B, d), dt, gen), v_pool=_normal((NB, hkv, B, d), dt, gen))
        return s
    N = case["seqs"]
    if op == "keep":
        n = np.full(N, case["nodes"], dtype=np.int64)
        ctx = n + rng.permutation(_spread(0, 99, N))
        path = np.full((N, case["nodes"]), -1, dtype=np.int32)
        behind = np.argsort(rng.random((N, case["nodes"] - 1)), axis=1)[:, :case["accepted"] - 1] + 1
        path[:, 0] = 0
        path[:, 1:case["accepted"]] = np.sort(behind, axis=1)
        s.update(path=_dev(path))
    else:
        ctx, n = rng.permutation(_spread(case["ctx_lo"], case["ctx_hi"], N)), rng.permutation(_counts(case))
        mask, _ = _trees(rng, n, case["nodes"])
        s.update(masks=_dev(_packed(mask, n).astype(np.int64)), q=_normal((int(n.sum()), hq, d), dt, gen),
                 scale=1 / math.sqrt(d))
    table, NB = _place(rng, ctx, B)
    s.update(q_start=_dev(np.concatenate([[0], n.cumsum()]).astype(np.int32)), ctx=_dev(ctx.astype(np.int32)),
             table=_dev(table), k_pool=_normal((NB, hkv, B, d), dt, gen), v_pool=_normal((NB, hkv, B, d), dt, gen))
    return s


# ---------------------------------------------------------------- the plain forms
def _rotated(x, w, s):
    """x [T, H, d] in 32 bits: normed per head, the first `rotary` values of each head rotated."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    # angles of far positions need 64 bits
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()[None, :]
    c, t = (torch.cos(angle) * s["scale"]).float()[:, None], (torch.sin(angle) * s["scale"]).float()[:, None]
    r = s["rotary"]
    if s["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * c - b * t, b * c + a * t], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * c - b * t, b * c + a * t], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _append(s):
    dt, B = s["k_pool"].dtype, s["block"]
    q = _rotated(s["q"], s["qw"], s).to(dt)
    blk, off = s["slots"] // B, s["slots"] % B
    s["k_pool"][blk, :, off] = _rotated(s["k"], s["kw"], s).to(dt)
    s["v_pool"][blk, :, off] = s["v"]
    return {"q": q, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _padded_rows(s):
    """Row numbers [N, nodes] of each sequence's drafted tokens in the packed arrays (past its end: row 0), and
    which of them there are."""
    i = torch.arange(s["nodes"], device="cuda")
    n = s["q_start"].diff().long()
    real = i[None, :] < n[:, None]
    return torch.where(real, s["q_start"][:-1, None].long() + i, 0), real, n


def _tree(s):
    N, hkv, d, B = s["seqs"], s["kv_heads"], s["head_dim"], s["block"]
    g = s["q_heads"] // hkv
    rows, real, n = _padded_rows(s)
    L = s["table"].shape[1] * B
    table = s["table"].long()
    k = s["k_pool"][table].transpose(1, 2).reshape(N, hkv, L, d).float()
    v = s["v_pool"][table].transpose(1, 2).reshape(N, hkv, L, d).float()
    q = s["q"][rows].float().reshape(N, -1, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(N, hkv, -1, d)
    p = q @ k.transpose(-1, -2) * s["scale"]                             # [N, hkv, nodes * g, L]
    del k
    at = torch.arange(L, device="cuda")[None, :] - (s["ctx"].long() - n)[:, None]   # < 0: cached before the tree
    bit = (s["masks"][rows][:, :, None] >> at.clamp(0, 63)[:, None, :]) & 1
    seen = (at < 0)[:, None, :] | ((at < n[:, None])[:, None, :] & (at >= 0)[:, None, :] & (bit == 1))
    seen = seen.repeat_interleave(g, 1)[:, None]
    p = p.masked_fill_(~seen, -math.inf)
    top = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = p @ v.masked_fill_((at >= n[:, None])[:, None, :, None], 0.0)
    o = torch.where(total > 0, o / total, 0.0)
    o = o.reshape(N, hkv, -1, g, d).permute(0, 2, 1, 3, 4).reshape(N, -1, hkv * g, d)
    return o[real].to(s["q"].dtype)


def _verify(s):
    rows, real, n = _padded_rows(s)
    masks, draft, target = s["masks"][rows], s["draft"][rows], s["target"][rows]
    i = torch.arange(s["nodes"], device="cuda")
    has = ((masks[:, :, None] >> i) & 1) == 1                            # [N, i, j]: i has j on its way
    below = has & (i[None, :] < i[:, None])
    parent = torch.where(below, i, -1).amax(-1)
    match = (parent >= 0) & (draft == target.gather(1, parent.clamp(min=0)))
    same = (parent[:, :, None] == parent[:, None, :]) & (i[None, :] < i[:, None]) & match[:, None, :]
    ok = (((match & ~same.any(-1)) & (i > 0)) | (i == 0)) & real
    accepted = ok & (~below | ok[:, None, :]).all(-1)
    count = accepted.sum(-1)
    path = torch.where(accepted, i, s["nodes"]).sort(-1).values
    path = torch.where(path < s["nodes"], path, -1).int()
    last = torch.where(accepted, i, -1).amax(-1, keepdim=True)
    following = torch.where(last >= 0, target.gather(1, last.clamp(min=0)), -1)[:, 0]
    return {"path": path, "accepted": count.int(), "next": following,
            "ctx": (s["ctx"] - n + count).int()}


def _keep(s):
    B = s["block"]
    path = s["path"].long()
    base = (s["ctx"] - s["q_start"].diff()).long()[:, None]
    to = torch.where(path >= 0, torch.arange(s["nodes"], device="cuda"), 0)
    src, dst = base + path.clamp(min=0), base + to                       # past the path: the first token to itself
    sb, db = s["table"].long().gather(1, src // B), s["table"].long().gather(1, dst // B)
    k, v = s["k_pool"][sb, :, src % B], s["v_pool"][sb, :, src % B]
    s["k_pool"][db, :, dst % B] = k
    s["v_pool"][db, :, dst % B] = v
    return {"k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def run(s):
    if not own:
        return {"append": _append, "tree": _tree, "verify": _verify, "keep": _keep}[s["op"]](s)
    import paged_kv_cache_254_gb300 as pa
    if s["op"] == "append":
        q = pa.pa_rope_append_kv(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["k_pool"], s["v_pool"],
                                 s["inv_freq"], interleaved=s["interleaved"], rope_scale=s["scale"], q_weight=s["qw"],
                                 k_weight=s["kw"], eps=1e-6)
        return {"q": q, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    if s["op"] == "tree":
        return pa.pa_decode_tree(s["q"], s["k_pool"], s["v_pool"], s["table"], s["ctx"], s["q_start"], s["masks"],
                                 s["scale"], max_nodes=s["nodes"])
    if s["op"] == "verify":
        path, accepted, following, ctx = pa.pa_tree_verify(s["masks"], s["draft"], s["target"], s["q_start"],
                                                           s["ctx"], max_nodes=s["nodes"])
        return {"path": path, "accepted": accepted, "next": following, "ctx": ctx}
    pa.pa_keep_kv(s["path"], s["q_start"], s["ctx"], s["table"], s["k_pool"], s["v_pool"])
    return {"k_pool": s["k_pool"], "v_pool": s["v_pool"]}


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_turn(x, w, s):
    """x [T, H, d] as complex pairs turned by e^(i position frequency)."""
    x = x.double()
    if w is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * w.double()
    r = s["rotary"]
    pair = torch.arange(r, device=x.device)
    pair = pair.reshape(-1, 2) if s["interleaved"] else pair.reshape(2, -1).T
    z = torch.complex(x[..., pair[:, 0]], x[..., pair[:, 1]])
    w64 = torch.outer(s["positions"].double(), s["inv_freq"].double())
    z = z * torch.polar(torch.full_like(w64, s["scale"]), w64)[:, None]
    y = x.clone()
    y[..., pair[:, 0]], y[..., pair[:, 1]] = z.real, z.imag
    return y


def _exact_tree(s):
    hkv, B, d = s["kv_heads"], s["block"], s["head_dim"]
    g = s["q_heads"] // hkv
    starts, ctx, masks = s["q_start"].tolist(), s["ctx"].tolist(), s["masks"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(s["seqs"]):
        lo, hi, c = starts[b], starts[b + 1], ctx[b]
        blocks = s["table"][b, :-(-c // B)].long()
        k, v = (pool[blocks].permute(1, 0, 2, 3).flatten(1, 2)[:, :c].double() for pool in (s["k_pool"], s["v_pool"]))
        tree = torch.tensor([[(m >> j) & 1 for j in range(hi - lo)] for m in masks[lo:hi]], dtype=torch.bool)
        seen = torch.cat([torch.ones(hi - lo, c - (hi - lo), dtype=torch.bool), tree], 1).cuda()
        q = s["q"][lo:hi].double().unflatten(1, (hkv, g))
        a = torch.einsum("nhgd,hld->hgnl", q, k) * s["scale"]
        a = a.masked_fill(~seen, -math.inf).softmax(-1)
        out[lo:hi] = torch.einsum("hgnl,hld->nhgd", a, v).flatten(1, 2)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "verify":
        return None                                  # whole numbers
    if case["op"] == "tree":
        return _exact_tree(s)
    k, v = s["k_pool"].double(), s["v_pool"].double()
    if case["op"] == "append":
        slots = s["slots"].tolist()
        kt, vt = _exact_turn(s["k"], s["kw"], s), s["v"].double()
        where = torch.tensor([divmod(x, case["block"]) for x in slots], device="cuda")
        k[where[:, 0], :, where[:, 1]], v[where[:, 0], :, where[:, 1]] = kt, vt
        return {"q": _exact_turn(s["q"], s["qw"], s), "k_pool": k, "v_pool": v}
    k0, v0 = k.clone(), v.clone()
    starts, ctx, path, table = (s[x].tolist() for x in ("q_start", "ctx", "path", "table"))
    moves = []
    for b in range(case["seqs"]):
        first = ctx[b] - (starts[b + 1] - starts[b])
        for to, node in enumerate(x for x in path[b] if x >= 0):
            (si, so), (di, do) = divmod(first + node, case["block"]), divmod(first + to, case["block"])
            moves.append((table[b][si], so, table[b][di], do))
    m = torch.tensor(moves, device="cuda").T
    k[m[2], :, m[3]], v[m[2], :, m[3]] = k0[m[0], :, m[1]], v0[m[0], :, m[1]]
    return {"k_pool": k, "v_pool": v}
