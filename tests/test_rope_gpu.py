"""pa_rope_append_kv against the fp64 oracle.

Tolerance, per element: half a step of the 16-bit output (finfo.eps / 2 of the
value; 2^-25 below fp16's normal range) plus the fp32 work in front of it.
Angles are off by at most 2^-32 turns for the fixed point and half a step of the
fp32 argument of sincospif (2^-25 half turns), 1.0e-7 radians in all; sincospif
adds 2 steps; the products, the sum of squares (16 terms a lane, 4 rounds),
rsqrtf (2 steps) and the two multiplications of the norm add at most 16 steps.
Together below 32 * 2^-24 = 2^-19 of the pair's length, taken here as the row's
largest normed value times 1.5 > sqrt(2), times the scale."""

import numpy as np
import pytest
import torch

from oracle.kv_ops import bits
from oracle.rope import norm_ref, rotate_ref
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def pa():
    import paged_kv_cache_254_gb300 as m
    return m


DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def values(shape, dt, seed, mult=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device="cuda", generator=g) * mult).to(dt)


def expected(x, w, eps, positions, freq, interleaved, scale):
    y = norm_ref(x, w, eps) if w is not None else x.double().cpu().numpy()
    return rotate_ref(y, positions, freq, interleaved, scale), np.abs(y).max(-1, keepdims=True) * max(1.0, abs(scale))


def close(got, want, top):
    eps = torch.finfo(got.dtype).eps / 2
    err = np.abs(got.double().cpu().numpy() - want)
    bound = eps * np.abs(want) + 1.5 * 2.0 ** -19 * top + 2.0 ** -25
    assert np.isfinite(err).all() and (err <= bound).all(), f"worst {np.max(err - bound):.3e} over the bound"


def case(T, Hq, Hkv, d, B, dt, seed=0, strided=True, extra=5):
    NB = -(-T // B) + extra
    if strided:
        qkv = values((T, (Hq + 2 * Hkv) * d), dt, seed)
        q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], 1))
    else:
        q, k, v = values((T, Hq, d), dt, seed), values((T, Hkv, d), dt, seed + 1), values((T, Hkv, d), dt, seed + 2)
    slots = np.random.default_rng(seed).permutation(NB * B)[:T].astype(np.int64)
    return q, k, v, slots, values((NB, Hkv, B, d), dt, seed + 3), values((NB, Hkv, B, d), dt, seed + 4)


def check(q, k, v, slots, kp, vp, positions, freq, interleaved=False, scale=1.0, qw=None, kw=None, eps=1e-6,
          live=None, **kwargs):
    """Run the call and compare queries, both pools and every untouched slot."""
    B = kp.shape[2]
    k0, v0 = bits(kp), bits(vp)
    fq = np.asarray([] if freq is None else freq.cpu())
    want_q, top_q = expected(q, qw, eps, positions, fq, interleaved, scale)
    want_k, top_k = expected(k, kw, eps, positions, fq, interleaved, scale)
    vb = bits(v)
    out = pa().pa_rope_append_kv(q, k, v, torch.tensor(positions, dtype=torch.int32, device="cuda"),
                                 torch.from_numpy(slots).cuda(), kp, vp, freq, interleaved=interleaved,
                                 rope_scale=scale, q_weight=qw, k_weight=kw, eps=eps, **kwargs)
    torch.cuda.synchronize()
    close(out, want_q, top_q)
    live = np.arange(len(slots)) if live is None else live
    blk, at = slots[live] // B, slots[live] % B
    close(kp[torch.from_numpy(blk), :, torch.from_numpy(at)], want_k[live], top_k[live])
    k1, v1 = bits(kp), bits(vp)
    v0[blk, :, at] = vb[live]
    assert np.array_equal(v1, v0)                          # values bit for bit, the rest untouched
    k0[blk, :, at] = k1[blk, :, at]
    assert np.array_equal(k1, k0)
    return out


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("d,rotary,B,Hq,Hkv", [(64, 64, 16, 8, 8), (64, 16, 32, 4, 1), (128, 128, 16, 32, 8),
                                               (128, 64, 32, 16, 1), (256, 256, 16, 4, 2), (96, 96, 16, 6, 3),
                                               (80, 32, 16, 5, 5), (32, 32, 16, 3, 1), (16, 16, 32, 2, 2)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_layouts(dt, d, rotary, B, Hq, Hkv, interleaved, norm):
    dt = DT[dt]
    T = 37
    c = case(T, Hq, Hkv, d, B, dt, seed=d + rotary + Hq)
    freq, _ = pa().rope_inv_freq(rotary)
    qw, kw = (values((d,), dt, 91), values((d,), dt, 92)) if norm else (None, None)
    check(*c, positions=list(range(100, 100 + T)), freq=freq, interleaved=interleaved, qw=qw, kw=kw)


@pytest.mark.parametrize("T", [1, 2, 7, 511, 1531])
@pytest.mark.parametrize("strided", [False, True])
def test_token_counts(T, strided):
    c = case(T, 8, 2, 128, 16, torch.bfloat16, seed=T, strided=strided)
    freq, _ = pa().rope_inv_freq(128)
    w = values((128,), torch.bfloat16, 5)
    check(*c, positions=list(range(T)), freq=freq, qw=w, kw=w)


def test_far_and_negative_positions():
    pos = [0, 1, -1, 131071, 1_000_003, -1_000_003, 2 ** 31 - 1, -2 ** 31, 16_777_217, 123_456_789]
    c = case(len(pos), 4, 2, 64, 16, torch.float16, seed=9)
    freq, _ = pa().rope_inv_freq(64)
    check(*c, positions=pos, freq=freq)


def test_unusual_frequencies():
    # zero, negative, tiny, above a turn a position; all with exact turns at these positions
    freq = torch.tensor([0.0, -0.5, 1e-12, 1e-30, 7.25, 100.5, 3.0, 1e-3], device="cuda")
    c = case(6, 2, 1, 16, 16, torch.bfloat16, seed=3)
    check(*c, positions=[0, 1, 5, 1000, 65536, -77], freq=freq)


@pytest.mark.parametrize("scaling,kw", [("linear", {}), ("ntk", {}), ("yarn", dict(original_len=4096))])
def test_long_context_scalings(scaling, kw):
    freq, scale = pa().rope_inv_freq(128, scaling=scaling, factor=16.0, **kw)
    c = case(50, 4, 2, 128, 16, torch.bfloat16, seed=11)
    check(*c, positions=[1311 * i for i in range(50)], freq=freq, scale=scale)


def test_one_sided_norm_no_rotation_and_large_values():
    c = case(20, 4, 2, 64, 16, torch.bfloat16, seed=13)
    w = values((64,), torch.bfloat16, 14)
    check(*c, positions=[0] * 20, freq=None, kw=w, eps=0.5)
    q, k, v, slots, kp, vp = case(20, 4, 2, 64, 16, torch.bfloat16, seed=15)
    big = torch.full_like(k, 3.0) * 2.0 ** 40             # squares near fp32's range, and tiny ones
    small = torch.full_like(q, 2.0 ** -60)
    check(small, big, v, slots, kp, vp, positions=list(range(20)), freq=None, qw=w, kw=w, eps=0.0)


def test_skipped_and_bad_slots():
    q, k, v, slots, kp, vp = case(12, 4, 2, 64, 16, torch.float16, seed=17)
    slots[[0, 5, 11]] = -1
    freq, _ = pa().rope_inv_freq(64)
    live = np.flatnonzero(slots >= 0)
    check(q, k, v, slots, kp, vp, positions=list(range(12)), freq=freq, live=live)
    err = pa().new_error_word("cuda")
    slots[[2, 3]] = [kp.shape[0] * 16, 2 ** 40]
    live = np.flatnonzero((slots >= 0) & (slots < kp.shape[0] * 16))
    check(q, k, v, slots, kp, vp, positions=list(range(12)), freq=freq, live=live, err=err)
    assert pa().pa_read_error(err) == 4 and int(err.item()) == 4


def test_values_keep_their_bits_and_bad_rows_stay_alone():
    q, k, v, slots, kp, vp = case(9, 2, 2, 64, 16, torch.bfloat16, seed=19, strided=False)
    v.view(torch.int16)[4] = 0x7fa5                       # a NaN with a payload
    v[5, 1, 3] = float("-inf")
    freq, _ = pa().rope_inv_freq(32)
    check(q, k, v, slots, kp, vp, positions=list(range(9)), freq=freq)
    # an infinity in an unrotated value of a key leaves the others as they are
    k[3, 0, 60] = float("inf")
    out = pa().pa_rope_append_kv(q, k, v, torch.arange(9, dtype=torch.int32, device="cuda"),
                                 torch.from_numpy(slots).cuda(), kp, vp, freq)
    row = kp[slots[3] // 16, 0, slots[3] % 16]
    assert torch.isinf(row[60]) and torch.isfinite(row[:60]).all() and torch.isfinite(out).all()


def test_in_place_queries_and_refusals():
    q, k, v, slots, kp, vp = case(33, 8, 2, 128, 16, torch.bfloat16, seed=21, strided=False)
    freq, _ = pa().rope_inv_freq(128)
    pos = torch.arange(33, dtype=torch.int32, device="cuda")
    sl = torch.from_numpy(slots).cuda()
    want = pa().pa_rope_append_kv(q, k, v, pos, sl, kp, vp, freq)
    got = pa().pa_rope_append_kv(q, k, v, pos, sl, kp, vp, freq, out=q)
    assert got is q and torch.equal(got, want)
    E = (ValueError, TypeError, pa().PagedAttentionError)
    bad = [dict(q=q.float()), dict(q=q.transpose(0, 1)), dict(k_new=k[:5]), dict(positions=pos.long()),
           dict(slot_mapping=sl.int()), dict(inv_freq=freq.double()), dict(inv_freq=freq[:20]),
           dict(inv_freq=torch.cat([freq, freq])), dict(q_weight=freq), dict(q_weight=q[0, :2].flatten()),
           dict(out=q[:, :4]), dict(out=q[:5]), dict(v_pool=vp[:, :1]), dict(q=q[:, :, ::2]),
           dict(q=q[:1].expand(33, 8, 128)), dict(positions=pos[:3]), dict(k_pool=kp.cpu())]
    good = dict(q=q, k_new=k, v_new=v, positions=pos, slot_mapping=sl, k_pool=kp, v_pool=vp, inv_freq=freq)
    before = bits(kp)
    for b in bad:
        with pytest.raises(E):
            pa().pa_rope_append_kv(**{**good, **b})
    assert np.array_equal(bits(kp), before)
    # no tokens
    assert pa().pa_rope_append_kv(q[:0], k[:0], v[:0], pos[:0], sl[:0], kp, vp, freq).shape == (0, 8, 128)


def test_captured_and_on_another_stream():
    q, k, v, slots, kp, vp = case(40, 8, 2, 128, 16, torch.bfloat16, seed=23)
    freq, _ = pa().rope_inv_freq(128)
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    sl = torch.from_numpy(slots).cuda()
    want = pa().pa_rope_append_kv(q, k, v, pos, sl, kp, vp, freq)
    wk = bits(kp)
    kp.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = pa().pa_rope_append_kv(q, k, v, pos, sl, kp, vp, freq, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = pa().pa_rope_append_kv(q, k, v, pos, sl, kp, vp, freq)
    pos.add_(1000)                                        # a replay reads what is there now
    g.replay()
    moved = out.clone()
    pos.sub_(1000)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and not torch.equal(moved, want)
    got = bits(kp)
    blk, at = slots // 16, slots % 16
    assert np.array_equal(got[blk, :, at], wk[blk, :, at])
