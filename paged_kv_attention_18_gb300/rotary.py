"""Tables of rotary frequencies for :func:`binding.rotary_reshape_and_cache`.

A table is float64 [rotary_dim / 2], radians per position, made once per model; how a model
stretches its positions for contexts longer than those it was trained on is all in it:

    plain          f_i = theta ^ (-2 i / R)
    factor         f_i / factor: every position counts as 1 / factor of one
    theta_factor   theta * theta_factor ^ (R / (R - 2)) for theta: the lowest frequency falls
                   by theta_factor, the highest stays
    by wavelength  f_i / factor where the wavelength 2 pi / f_i exceeds original_len / low,
                   f_i where it is under original_len / high, and between them a blend that
                   is linear in original_len / wavelength
"""
from __future__ import annotations

import math

import torch


def axes(sections, interleaved: bool = False, device=None) -> torch.Tensor:
    """int32 [sum(sections)]: the axis of every frequency of
    :func:`binding.rotary_axes_reshape_and_cache`, sections[a] of them on axis a: one section
    behind another, or (interleaved) the axes in turns as long as each has frequencies left."""
    left = [int(n) for n in sections]
    if not left or any(n < 0 for n in left) or sum(left) == 0:
        raise ValueError("sections must be counts, one at least above 0")
    if not interleaved:
        table = [a for a, n in enumerate(left) for _ in range(n)]
    else:
        table = []
        for turn in range(max(left)):
            table += [a for a, n in enumerate(left) if n > turn]
    return torch.tensor(table, dtype=torch.int32, device=device)


def frequencies(rotary_dim: int, theta: float = 10000.0, factor: float = 1.0,
                theta_factor: float = 1.0, original_len: int | None = None, low: float = 1.0,
                high: float = 4.0, device=None) -> torch.Tensor:
    """float64 [rotary_dim / 2] frequencies. With original_len the factor goes by wavelength,
    else it applies to every frequency."""
    if rotary_dim <= 0 or rotary_dim % 2:
        raise ValueError("rotary_dim must be a positive even number")
    if not (theta > 0 and factor > 0 and theta_factor > 0):
        raise ValueError("theta and the factors must be positive")
    if theta_factor != 1.0:
        if rotary_dim < 4:
            raise ValueError("theta_factor needs rotary_dim >= 4")
        theta = theta * theta_factor ** (rotary_dim / (rotary_dim - 2))
    f = theta ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim)
    if original_len is None:
        f = f / factor
    else:
        if not (original_len > 0 and 0 < low < high):
            raise ValueError("original_len must be positive and 0 < low < high")
        turns = original_len * f / (2 * math.pi)  # over the trained context
        keep = ((turns - low) / (high - low)).clamp(0.0, 1.0)
        f = keep * f + (1.0 - keep) * f / factor
    return f.to(device) if device is not None else f
