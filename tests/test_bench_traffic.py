"""The benchmark's DRAM traffic: captured from the kernel sources as they are."""

import os
import re

import pytest

import bench

CSRC = os.path.join(bench.ROOT, "paged_kv_cache_254_gb300", "csrc")


def test_captures_are_keyed_by_all_that_the_kernel_includes():
    seen, todo = set(), ["decode_kernel.cuh"]
    while todo:
        name = todo.pop()
        if name not in seen:
            seen.add(name)
            with open(os.path.join(CSRC, name)) as f:
                todo += re.findall(r'#include "([a-z0-9_]+[.]cuh)"', f.read())
    assert set(bench.KERNEL_SOURCES) == seen


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3", "int4"])
def test_the_present_kernels_have_a_capture(kv):
    """(After a change of these sources: the capture in profiles/pa_decode_*.md, and its key, anew.)"""
    got = bench.scaled_traffic(bench.kernel_hash(), kv, "llama3_70b_b256", 4_820_000_000)
    assert got is not None and 0.98 < got / 4_820_000_000 < 1.05
