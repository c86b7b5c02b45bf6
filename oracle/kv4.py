"""The 4-bit cache as plain fp64 NumPy: quantising a row and what the row holds.

Test infrastructure only (see the package docstring).

A row of d values is d / 2 bytes of codes (4-bit floats, the even value of a pair
in the low half) and d / 16 scale bytes (e4m3); value = t * scale * code.  The
scale of 16 values is max |x| / t / 6 on the e4m3 grid (at most 448), a code
x / t / scale on the code grid, both to nearest, ties to the even grid index.
"""

import numpy as np

# code grid and e4m3 grid (bytes 0 .. 126; byte 127 is NaN), by their bits
CODES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([i * 2.0 ** -9 if i < 8 else (1 + i % 8 / 8) * 2.0 ** (i // 8 - 7) for i in range(127)])


def nearest(x, grid):
    """Index of the grid value nearest to each x >= 0, ties to the even index;
    everything above the grid goes to its last value."""
    x = np.asarray(x, dtype=np.float64)
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    with np.errstate(invalid="ignore"):
        up, down = grid[hi] - x, x - grid[lo]
    return np.where(up < down, hi, np.where(down < up, lo, np.where(lo % 2 == 0, lo, hi)))


def quantise(x, t=1.0):
    """x [.., d]: code bytes [.., d / 2] and scale bytes [.., d / 16], uint8."""
    x = np.asarray(x, dtype=np.float64) / t
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    a = np.abs(g).max(axis=-1)
    broken = np.isnan(g).any(axis=-1)
    sf = np.where(broken, 127, nearest(np.where(broken | np.isinf(a), 1e300, a) / 6, E4M3)).astype(np.uint8)
    scale = E4M3[np.minimum(sf, 126)][..., None]
    live = (scale > 0) & ~broken[..., None]
    mag = np.where(live, np.minimum(np.abs(np.where(live, g, 0)), 1e300) / np.where(scale > 0, scale, 1), 0)
    code = nearest(mag, CODES) | (np.signbit(g).astype(np.int64) << 3)
    code = code.reshape(x.shape).astype(np.uint8)
    return code[..., 0::2] | code[..., 1::2] << 4, sf


def values(codes, sf, t=1.0):
    """What codes [.., d / 2] and scale bytes [.., d / 16] hold, fp64 [.., d]."""
    both = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], 2 * codes.shape[-1]).astype(np.int64)
    code = np.where(both >= 8, -1.0, 1.0) * CODES[both & 7]
    scale = np.append(E4M3, np.nan)[(sf & 127).astype(np.int64)] * np.where(sf >= 128, -1.0, 1.0)
    return code * np.repeat(scale, 16, axis=-1) * t
