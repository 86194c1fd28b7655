"""Inverse frequencies of rotary positions, also scaled for long contexts.

Host code, run once: the frequencies are weights of sas_rotary and
sas_cache_append, which take them as an fp32 tensor with their amplitude.
"""
from __future__ import annotations

import math

import torch


def inv_freq(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
             trained: int = 8192, slow: float = 1.0, fast: float = 32.0,
             device=None) -> tuple[torch.Tensor, float]:
    """(inv_freq [rot/2] fp32, amplitude) of a rotated width.

    Pair p turns by base^(-2p/rot) radians a position. For contexts `factor`
    times the `trained` length:
      none    as trained;
      linear  every frequency divided by factor (positions interpolated);
      base    the base raised to base * factor^(rot/(rot-2)): the fastest pair
              is kept, the slowest slowed by factor (one pair, rot 2, is kept);
      parts   pairs that turn fewer than `slow` times over the trained length
              are slowed by factor, those above `fast` turns kept, a linear
              ramp over the turns between; amplitude 1 + 0.1 ln factor for
              factor > 1 (on q and k alike, so the logits get its square).
    Computed in fp64, rounded once.
    """
    if rot < 2 or rot % 2:
        raise ValueError(f"rot must be even and at least 2 (got {rot})")
    if not 0 < base < math.inf or not 1 <= factor < math.inf:
        raise ValueError(f"base must be positive, factor at least 1, both finite (got {base}, {factor})")
    amplitude = 1.0
    p = torch.arange(rot // 2, dtype=torch.float64) * 2.0 / rot
    if scaling == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = float(base) ** -p
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        if not -math.inf < slow < fast < math.inf or not 0 < trained < math.inf:
            raise ValueError(f"fast must be above slow, both finite, and trained positive "
                             f"(got {fast}, {slow}, {trained})")
        turns = trained * f / (2.0 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
        if factor > 1:
            amplitude = 1.0 + 0.1 * math.log(factor)
    elif scaling not in ("none", "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.float().to(device) if device is not None else f.float(), amplitude
