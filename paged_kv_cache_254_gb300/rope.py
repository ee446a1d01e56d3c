"""Rotary frequencies for ``pa_rope_append_kv``, plain and stretched for
contexts longer than the trained one."""

from __future__ import annotations

import math

import torch

SCALINGS = (None, "linear", "ntk", "yarn")


def rope_inv_freq(rotary_dim: int, base: float = 10000.0, scaling=None, factor: float = 1.0, original_len=None,
                  beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
    """Return (inv_freq, rope_scale): radians per position, fp32
    [rotary_dim / 2], and the factor of cos and sin.

    The plain frequencies are base ** (-2 j / rotary_dim).  ``scaling``
    stretches them by ``factor``:

    * ``"linear"``: every frequency divided by factor (position interpolation);
    * ``"ntk"``: base multiplied by factor ** (r / (r - 2)), which leaves the
      fastest frequency alone and divides the slowest by factor;
    * ``"yarn"`` (Peng et al. 2023): a frequency that turns more than beta_fast
      times within original_len positions stays, one that turns less than
      beta_slow times is divided by factor, the ones between are blended
      linearly in their number of turns, and rope_scale is
      0.1 ln(factor) + 1.  A checkpoint whose frequencies were blended
      otherwise (linearly in the pair's index, with rounded ends) has others
      in the middle band, by up to a factor of 3: give those as inv_freq."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be a positive even number")
    if not base > 0 or not factor >= 1:
        raise ValueError("base must be positive and factor at least 1")
    if scaling not in SCALINGS:
        raise ValueError(f"scaling must be one of {SCALINGS}")
    j = torch.arange(rotary_dim // 2, dtype=torch.float64)
    rope_scale = 1.0
    if scaling == "ntk" and rotary_dim > 2:
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    freq = base ** (-2.0 * j / rotary_dim)
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "yarn":
        if original_len is None or not original_len > 0 or not beta_fast > beta_slow:
            raise ValueError("yarn needs original_len > 0 and beta_fast > beta_slow")
        turns = original_len * freq / (2 * math.pi)
        stay = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0.0, 1.0)
        freq = freq * stay + freq / factor * (1.0 - stay)
        rope_scale = 0.1 * math.log(factor) + 1.0
    return freq.float().to(device), rope_scale
