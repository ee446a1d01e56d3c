"""Rotary frequencies, each band by its formula."""

import math

import pytest

from paged_kv_cache_254_gb300 import rope_inv_freq


@pytest.mark.parametrize("dim,base,factor,length,fast,slow", [(64, 1e4, 16.0, 4096, 32.0, 1.0), (128, 1e4, 16.0, 4096, 32.0, 1.0),
                                                              (128, 5e5, 8.0, 8192, 32.0, 1.0), (64, 1e6, 4.0, 32768, 16.0, 2.0)])
def test_yarn_frequencies_by_their_number_of_turns(dim, base, factor, length, fast, slow):
    f, scale = rope_inv_freq(dim, base=base, scaling="yarn", factor=factor, original_len=length, beta_fast=fast,
                             beta_slow=slow, device="cpu")
    assert scale == 0.1 * math.log(factor) + 1
    bands = set()
    for j, got in enumerate(f.tolist()):
        plain = math.pow(base, -2 * j / dim)
        turns = length * plain / (2 * math.pi)
        if turns >= fast:
            band, stay = "fast", 1.0
        elif turns <= slow:
            band, stay = "slow", 0.0
        else:
            band, stay = "middle", (turns - slow) / (fast - slow)
        bands.add(band)
        # one rounding to fp32, 2^-24; the fp64 arithmetic on both sides is off by less than 2^-45
        assert math.isclose(got, stay * plain + (1 - stay) * plain / factor, rel_tol=2.0 ** -24 + 2.0 ** -45)
    assert bands == {"fast", "middle", "slow"}
