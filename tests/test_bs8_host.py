"""Host side of the block-scaled 8-bit cache: refusals that answer without touching a GPU."""

import ctypes

import pytest
import torch

from paged_kv_cache_254_gb300 import _build, _lib, ops
from tests.test_abi import BUF_BYTES, FAKE, NULL, shape

E4M3, E5M2 = ops.KV_FORMATS["e4m3"], ops.KV_FORMATS["e5m2"]


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _lib.load()


def off(k):
    return ctypes.c_void_p(FAKE.value + k)


POOL = off(1 << 17)        # 64 blocks of 2 heads of 32 + 2 * 16 * 64 bytes: 266,240
SMALL = dict(num_q_heads=4, num_kv_heads=2, num_blocks=64)


@pytest.mark.parametrize("kw,status", [
    (dict(max_new=0), 1), (dict(total=-1), 1), (dict(fmt=7), 1), (dict(k=NULL), 1), (dict(v=NULL), 1), (dict(qs=NULL), 1),
    (dict(pool=NULL), 1), (dict(table=NULL), 1), (dict(k=off(8)), 1), (dict(v=off(4)), 1), (dict(pool=off((1 << 17) + 16)), 1),
    (dict(qs=off(2)), 1), (dict(ks=120), 1), (dict(vs=127), 1), (dict(ks=132), 1),
    (dict(k=POOL), 1), (dict(v=off((1 << 17) + 266240 - 256)), 1),           # inside the pool
    (dict(sh=dict(head_dim=96)), 2), (dict(sh=dict(block_size=8)), 2), (dict(sh=dict(block_size=64)), 2),
    (dict(sh=dict(dtype=2)), 1), (dict(sh=dict(num_seqs=-1)), 1), (dict(sh=dict(max_blocks_per_seq=0)), 1),
    (dict(sh=dict(max_blocks_per_seq=1 << 27)), 2), (dict(sh=dict(num_seqs=0)), 0),
])
def test_append_checks(lib, kw, status):
    kw = dict(kw)
    sh = shape(**{**SMALL, **kw.pop("sh", {})})
    a = {**dict(max_new=4, total=8, fmt=E4M3, k=FAKE, v=off(1 << 16), qs=FAKE, pool=POOL, table=FAKE, ks=128, vs=128), **kw}
    assert lib.pa_append_kv_bs8(sh, a["fmt"], a["max_new"], a["total"], a["k"], a["ks"], a["v"], a["vs"], a["qs"],
                                a["table"], FAKE, a["pool"], NULL, NULL) == status


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=5), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(q=NULL), 1), (dict(out=NULL), 1),
    (dict(pool=NULL), 1), (dict(table=NULL), 1), (dict(q=off(8)), 1), (dict(pool=off((1 << 17) + 16)), 1),
    (dict(out=FAKE), 1), (dict(out=off(1024)), 1), (dict(out=off(2)), 1),                  # over q, or half of it
    (dict(ws=NULL), 6), (dict(ws=off(64)), 6),
    (dict(sh=dict(head_dim=96)), 2), (dict(sh=dict(block_size=8)), 2), (dict(sh=dict(num_q_heads=6)), 2),
    (dict(sh=dict(num_q_heads=64)), 2), (dict(sh=dict(num_q_heads=5)), 1), (dict(sh=dict(dtype=2)), 1),
    (dict(sh=dict(num_seqs=-1)), 1), (dict(sh=dict(num_seqs=0)), 0),
])
@pytest.mark.parametrize("multi", [False, True])
def test_attention_checks(lib, kw, status, multi):
    kw = dict(kw)
    sh = shape(**{**SMALL, **kw.pop("sh", {})})
    a = {**dict(fmt=E5M2, q=FAKE, pool=POOL, table=FAKE, scale=0.1, out=off(1 << 16), ws=FAKE), **kw}
    if status == 6 and not torch.cuda.is_available():
        status = (3, 6)                                   # (without a device the grid's size is not known)
    mid = (a["table"], FAKE, a["scale"], a["out"], a["ws"], BUF_BYTES, NULL, NULL)
    if multi:
        got = lib.pa_decode_multi_bs8(sh, a["fmt"], 4, 4, a["q"], FAKE, a["pool"], *mid)
    else:
        got = lib.pa_decode_bs8(sh, a["fmt"], a["q"], a["pool"], *mid)
    assert got in (status if isinstance(status, tuple) else (status,))


def test_multi_checks(lib):
    def m(max_q=4, total=4, qs=FAKE, **sh):
        return lib.pa_decode_multi_bs8(shape(**{**SMALL, **sh}), E4M3, max_q, total, FAKE, qs, POOL, FAKE, FAKE, 0.1,
                                       off(1 << 16), FAKE, BUF_BYTES, NULL, NULL)
    assert m(max_q=0) == 1 and m(max_q=-3) == 1 and m(total=-1) == 1 and m(qs=NULL) == 1 and m(qs=off(2)) == 1


def test_workspaces_of_bad_shapes_are_zero(lib):
    assert lib.pa_decode_bs8_workspace_bytes(shape(head_dim=80), E4M3) == 0
    assert lib.pa_decode_bs8_workspace_bytes(shape(), 9) == 0
    assert lib.pa_decode_bs8_workspace_bytes(None, E4M3) == 0
    assert lib.pa_decode_multi_bs8_workspace_bytes(shape(), E4M3, 0) == 0
    assert lib.pa_decode_multi_bs8_workspace_bytes(shape(block_size=8), E4M3, 4) == 0
    assert lib.pa_decode_multi_bs8_workspace_bytes(None, E4M3, 4) == 0


def test_copy_and_convert_checks(lib):
    def c(n=2, pairs=FAKE, pool=POOL, **sh):
        return lib.pa_copy_blocks_bs8(shape(**{**SMALL, **sh}), pairs, n, pool, NULL, NULL)
    assert c(n=-1) == 1 and c(pairs=NULL) == 1 and c(pool=NULL) == 1 and c(pool=off((1 << 17) + 8)) == 1
    assert c(head_dim=96) == 2 and c(block_size=8) == 2 and c(dtype=2) == 1 and c(n=0) == 0

    for name in ("pa_pack_blocks_bs8", "pa_unpack_blocks_bs8"):
        def f(n=2, nb=3, fmt=E4M3, pairs=FAKE, k=FAKE, v=off(1 << 16), pool=POOL, **sh):
            three = (k, v, pool) if "un" not in name else (pool, k, v)
            return getattr(lib, name)(shape(**{**SMALL, **sh}), fmt, nb, pairs, n, *three, NULL, NULL)
        assert f(n=-1) == 1 and f(nb=-1) == 1 and f(fmt=4) == 1 and f(pairs=NULL) == 1 and f(k=NULL) == 1
        assert f(v=NULL) == 1 and f(pool=NULL) == 1 and f(k=off(8)) == 1 and f(pool=off((1 << 17) + 16)) == 1
        assert f(k=POOL) == 1 and f(v=off((1 << 17) - 16)) == 1 and f(v=FAKE) == 1 and f(v=off(64)) == 1   # over another
        assert f(head_dim=96) == 2 and f(block_size=8) == 2 and f(dtype=2) == 1 and f(n=0) == 0


def test_python_calls_refuse_host_tensors():
    x = torch.zeros(2, 2, 64, dtype=torch.float16)
    wide = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    pool = ops.bs8_pool(4, 2, 16, 64, device="cpu")
    i = torch.zeros(3, dtype=torch.int32)
    pairs = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ops.pa_append_kv_bs8(x, x, i[None], i, i, pool)
    with pytest.raises(ValueError, match="CUDA"):
        ops.pa_decode_bs8(x, pool, i[None], i, 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        ops.pa_decode_multi_bs8(x, pool, i[None], i, i, 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        ops.pa_copy_blocks_bs8(pairs, pool)
    with pytest.raises(ValueError, match="CUDA"):
        ops.pa_pack_blocks_bs8(pairs, wide, wide, pool)
    with pytest.raises(ValueError, match="CUDA"):
        ops.pa_unpack_blocks_bs8(pairs, pool, wide, wide)


def test_formats_by_name():
    for bad in ("fp8", "E4M3", None, 1):
        with pytest.raises(ValueError, match="kv_format"):
            ops._bs8_format(bad)


def test_an_empty_pool():
    pool = ops.bs8_pool(3, 2, 16, 64, device="cpu")
    assert pool.shape == (3, 2, 32 + 2 * 16 * 64) and pool.dtype == torch.uint8 and not pool.any()
    s = ops.bs8_scales(pool)
    assert s.shape == (3, 2, 2) and s.dtype == torch.float32
    s[1, 1, 0] = 2.0
    assert pool[1, 1, :4].tolist() == [0, 0, 0, 0x40]
