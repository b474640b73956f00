"""Rotary frequencies for lsa_qk_norm_rope: one small table per model, made once on the host.

The kernel takes the frequencies as they are, so a rotation scaled for longer
contexts than the model was trained on is only another table (and, for one of
the scalings, another ``rope_scale``).
"""
from __future__ import annotations

import math
from typing import Optional

import torch

SCALINGS = ("none", "linear", "base", "parts")


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_context: Optional[int] = None, slow: float = 1.0, fast: float = 32.0, device=None):
    """``(inv_freq, rope_scale)``: fp32 [rot_dim / 2] on ``device`` and the factor of the rotated values.

    The unscaled frequency of pair i is base^(-2i / rot_dim).  ``scaling``:

    * ``"none"``: as it is;
    * ``"linear"``: every frequency divided by ``factor`` (position interpolation);
    * ``"base"``: the base multiplied by factor^(rot_dim / (rot_dim - 2)), which leaves the fastest pair alone and
      divides the slowest one by ``factor``;
    * ``"parts"``: by the turns r that a pair makes in ``original_context`` tokens: r > ``fast`` stays, r < ``slow``
      is divided by ``factor``, a linear ramp in r between them; ``rope_scale`` = 0.1 ln(factor) + 1 (interpolation by
      parts, Peng et al. 2023, "YaRN", section 3).  Tables that ramp linearly in the pair's index i instead, between
      the two bounds' indexes, differ from these inside the ramp: a model trained with such a table needs its own.

    Computed in fp64 and rounded once to fp32.
    """
    if rot_dim <= 0 or rot_dim > 128 or rot_dim % 8:
        raise ValueError("rot_dim must be a multiple of 8 in [8, 128]")
    if scaling not in SCALINGS:
        raise ValueError(f"scaling must be one of {SCALINGS}")
    if not base > 0 or not factor >= 1 or not math.isfinite(base) or not math.isfinite(factor):
        raise ValueError("base must be positive and factor at least 1")
    if scaling == "base":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    freq = base ** (-2.0 * i / rot_dim)
    scale = 1.0
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "parts":
        if not original_context or not original_context > 0 or not 0 <= slow < fast:   # (NaN too)
            raise ValueError("scaling by parts needs original_context > 0 and 0 <= slow < fast")
        turns = original_context * freq / (2 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0, 1)
        freq = freq * keep + freq / factor * (1 - keep)
        scale = 0.1 * math.log(factor) + 1.0
    return freq.to(torch.float32).to(device or "cpu"), scale
