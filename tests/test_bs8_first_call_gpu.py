"""The first block-scaled call of a process, whatever its sizes are."""

import os
import subprocess
import sys

import pytest

from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import numpy as np, torch
import paged_kv_cache_254_gb300 as pa
from tests.bs8_util import dev, place, random_pool
most, n = {most}, {n}
r = np.random.default_rng(1)
table, NB = place(r, [200, 90], 16)
pool = dev(random_pool(r, NB, 2, 16, 128, "e4m3"))
q = torch.randn(2 * n, 8, 128, device="cuda").bfloat16()
args = (q, pool, dev(table), dev(np.array([200, 90], np.int32)), dev(np.array([0, n, 2 * n], np.int32)), 0.09)
first = pa.pa_decode_multi_bs8(*args, max_q_len=most)
assert torch.equal(first, pa.pa_decode_multi_bs8(*args, max_q_len=max(n, 1)))
print("same")
"""


@pytest.mark.parametrize("most,n", [(1000, 3), (1000, 0), (33, 16), (1000, 60), (5, 5)])
def test_a_chunk_call_with_a_loose_bound(most, n):
    """The bound alone asks for groups of 256 query rows, the call's rows (8 n, at most 128) for the other kernel."""
    need_gpu()
    p = subprocess.run([sys.executable, "-c", CHILD.format(most=most, n=n)], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert p.returncode == 0 and p.stdout.strip() == "same", p.stderr[-2000:]
