"""Waits of the block-scaled chunk kernel that run out: the call returns, says so, and leaves nothing that
could be taken for an answer."""

import numpy as np
import pytest
import torch

from tests.bs8_util import attention, check, dev, pa, place, random_pool
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("dtype,B,d", [(torch.bfloat16, 16, 128), (torch.float16, 32, 64)])
@pytest.mark.parametrize("ctx,n", [
    ([3000, 17, 5000, 33], [3, 5, 4, 1]),                      # rows of few tiles, most of them cut among CTAs
    ([700, 4000, 90], [300, 40, 90]),                          # groups of 256 rows
    ([40, 33, 50] * 120, [2, 1, 16] * 120),                    # several whole pairs to a CTA
])
def test_a_wait_that_runs_out(dtype, B, d, ctx, n):
    """The converting warps of every CTA wait, for 100 us at most, on a barrier that nothing completes, in a
    workspace that holds the states of a whole call before."""
    r = np.random.default_rng(len(ctx))
    table, NB = place(r, ctx, B)
    pool = random_pool(r, NB, 2, B, d, "e4m3")
    qs = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    q = torch.from_numpy(r.standard_normal((int(qs[-1]), 16, d))).to(dtype)
    args = [q.cuda(), dev(pool), dev(table), dev(np.array(ctx, np.int32)), dev(qs), 0.1]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(args[0])
    call = lambda err: pa().pa_decode_multi_bs8(*args, max_q_len=max(n), out=out, workspace=ws, err=err)  # noqa: E731
    want = call(pa().new_error_word("cuda")).clone()
    if len(ctx) < 10:
        check(want, *attention(q, pool, table, ctx, qs, 0.1, B, "e4m3"))
    pa().pa_set_decode_stall_ns(100_000)
    try:
        err = pa().new_error_word("cuda")
        call(err)
        assert pa().pa_read_error(err) == 5                    # PA_ERR_TIMEOUT
        assert int(err.item()) == 16 and out.isnan().all()     # cut rows too, through the merge
    finally:
        pa().pa_set_decode_stall_ns(0)
    err = pa().new_error_word("cuda")
    assert torch.equal(call(err), want) and int(err.item()) == 0
