"""fp64 CPU oracle of the 8-bit paged cache (test infrastructure only): e4m3
rounding, the write that quantises and the read back, block by block from their
definitions; it shares nothing with the CUDA path."""

from __future__ import annotations

import numpy as np
import torch

TOKENS = 16  # of a scale
LEAST = -64  # exponent of the least scale

# the magnitudes that codes stand for, ascending: 0x00 .. 0x7e
MAGNITUDES = np.array([(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
                       for e in range(16) for m in range(8)][:127])


def values(codes: np.ndarray) -> np.ndarray:
    """What codes (uint8) stand for."""
    mag = np.where((codes & 0x7F) == 0x7F, np.nan, MAGNITUDES[np.minimum(codes & 0x7F, 126)])
    return np.where(codes & 0x80, -mag, mag)


def encode(x: np.ndarray) -> np.ndarray:
    """The nearest codes, ties to the even code; past 448: 448; NaN: 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    hi = np.clip(np.searchsorted(MAGNITUDES, np.where(np.isnan(a), 0.0, a)), 1, 126)
    lo = hi - 1
    below, above = a - MAGNITUDES[lo], MAGNITUDES[hi] - a
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    code = np.where(up, hi, lo)
    code = np.where(a >= 448.0, 126, code).astype(np.uint8)
    code = np.where(np.signbit(x), code | 0x80, code).astype(np.uint8)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def least_scale(a: float) -> float:
    """The smallest power of two, 2^LEAST at least, with a <= 448 times it."""
    e = LEAST
    while a > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def magnitude(x: np.ndarray) -> float:
    """The largest finite magnitude (0: none)."""
    a = np.abs(x[np.isfinite(x)])
    return float(a.max()) if a.size else 0.0


def store(x: np.ndarray, slots, codes: np.ndarray, scale: np.ndarray):
    """Rows x [T, H, D] (fp64) at the slots, in place: codes [pages, P, H, D] uint8,
    scale [pages, P / 16, H]."""
    P = codes.shape[1]
    runs = {}
    for t, s in enumerate(slots):
        if s >= 0:
            runs.setdefault(int(s) // TOKENS, []).append((int(s) % TOKENS, t))
    for block, tokens in runs.items():
        page, sub = block * TOKENS // P, block * TOKENS % P // TOKENS
        at = codes[page, sub * TOKENS:(sub + 1) * TOKENS]
        named = {o for o, _ in tokens}
        for h in range(x.shape[1]):
            need = least_scale(magnitude(np.stack([x[t, h] for _, t in tokens])))
            old = float(scale[page, sub, h])
            held = np.isfinite(old) and old > 0 and 0 not in named
            now = max(old, need) if held else need
            if held and now > old:
                for o in set(range(TOKENS)) - named:
                    at[o, h] = encode(values(at[o, h]) * (old / now))
            for o, t in tokens:
                at[o, h] = encode(x[t, h] / now)
            scale[page, sub, h] = now


def dequantised(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """codes [pages, P, H, D] and scale [pages, P / 16, H] as values."""
    return values(codes) * np.repeat(scale.astype(np.float64), TOKENS, axis=1)[..., None]


def read(pool: np.ndarray, table, lens, out_table, out: np.ndarray):
    """Pages of a dequantised pool to a staging pool, in place."""
    P = pool.shape[1]
    for s, L in enumerate(lens):
        for j in range(min(-(-int(L) // P), len(table[s]))):
            if table[s][j] >= 0 and out_table[s][j] >= 0:
                n = min(P, int(L) - j * P)
                out[out_table[s][j], :n] = pool[table[s][j], :n]


def by_token(pool: torch.Tensor, layout: int) -> np.ndarray:
    """A pool of codes as [page, token, kv head, d] uint8."""
    t = pool.view(torch.uint8).cpu()
    return np.ascontiguousarray((t if layout == 0 else t.permute(0, 2, 1, 3)).numpy())
