"""Sizes of the block-scaled calls whose product passes 32 bits: what is refused goes by the work there is."""

import ctypes

import pytest
import torch

from paged_kv_cache_254_gb300 import _build, _lib, ops
from tests.test_abi import BUF_BYTES, FAKE, NULL, shape

E4M3 = ops.KV_FORMATS["e4m3"]


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _lib.load()


@pytest.mark.skipif(torch.cuda.is_available(), reason="the operands are no device memory")
@pytest.mark.parametrize("kw,ok", [
    (dict(num_seqs=32, max_q=2 ** 31 - 1, total=64), True),    # 2^27 groups of 16 tokens by the bound alone
    (dict(num_seqs=1 << 20, max_q=1 << 20, total=1 << 20, max_blocks_per_seq=8), True),
    (dict(num_seqs=1 << 20, max_q=2 ** 31 - 1, total=1 << 20, max_blocks_per_seq=1 << 20), False),   # 2^36 in earnest
])
def test_a_chunk_bound_far_above_the_chunks_is_no_reason_to_refuse(lib, kw, ok):
    kw = dict(kw)
    max_q, total = kw.pop("max_q"), kw.pop("total")
    sh = shape(num_q_heads=16, num_kv_heads=1, num_blocks=64, **kw)
    off = lambda k: ctypes.c_void_p(FAKE.value + k)  # noqa: E731
    st = lib.pa_decode_multi_bs8(sh, E4M3, max_q, total, FAKE, FAKE, FAKE, FAKE, FAKE, 0.1, off(1 << 40), FAKE, BUF_BYTES,
                                 NULL, NULL)
    assert st == (3 if ok else 2)                              # without a device: the grid's size is not known
