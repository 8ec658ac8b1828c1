"""fp64 CPU oracle of the rotary embedding with a position per axis (test
infrastructure only)."""

from __future__ import annotations

import numpy as np

from . import rope_cache


def rope_axes(x: np.ndarray, positions: np.ndarray, cos_sin: np.ndarray, pair_axis, rot_dim: int,
              is_neox: bool) -> np.ndarray:
    """``rope_cache.rope`` with a position per axis, positions [axes, T]: pair i by the
    angle at positions[pair_axis[i], t]."""
    out = np.array(x, dtype=np.float64, copy=True)
    half = rot_dim // 2
    a, b = rope_cache.pair_index(rot_dim, is_neox)
    for i in range(half):
        p = positions[pair_axis[i]]
        c, s = cos_sin[p, i][:, None], cos_sin[p, half + i][:, None]
        x1, x2 = x[:, :, a[i]], x[:, :, b[i]]
        out[:, :, a[i]] = x1 * c - x2 * s
        out[:, :, b[i]] = x2 * c + x1 * s
    return out
