"""Rows of 8 and 4 bits with a power of two per 32 values, in 64 bits, in
NumPy: a plain restatement of the definitions in include/s2_ops.h for the tests
of the kernels."""

import numpy as np

GROUP, EMIN, EMAX = 32, -126, 120


def _grid(lowest, highest, mantissas):
    """Non-negative values of a small float type, in the order of their codes."""
    below = [2.0 ** lowest * m / mantissas for m in range(mantissas)]
    return np.array(below + [2.0 ** e * (1 + m / mantissas) for e in range(lowest, highest + 1)
                             for m in range(mantissas)])


E4M3 = _grid(-6, 8, 8)[:-1]          # its last code is NaN
E2M1 = _grid(0, 2, 2)
VALUE8 = np.concatenate([E4M3, [np.nan], -E4M3, [np.nan]])
VALUE4 = np.concatenate([E2M1, -E2M1])


def up(n, m):
    return (n + m - 1) // m * m


def exponents(x, top):
    """Smallest e with each group's largest finite magnitude <= top * 2^e; x float64 [rows, K]."""
    n, K = x.shape
    a = np.zeros((n, up(K, GROUP)))
    a[:, :K] = np.where(np.isfinite(x), np.abs(x), 0)
    a = a.reshape(n, -1, GROUP).max(-1)
    powers = np.array([top * 2.0 ** e for e in range(EMIN, EMAX + 1)])
    return np.minimum(np.searchsorted(powers, a), EMAX - EMIN) + EMIN


def nearest(z, grid):
    """Codes of the grid's values next to z, the even code on a tie, sign in the top bit."""
    a = np.minimum(np.abs(z), grid[-1])
    hi = np.minimum(np.searchsorted(grid, a), len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    down, up_ = a - grid[lo], grid[hi] - a
    return np.where((down < up_) | ((down == up_) & (lo % 2 == 0)), lo, hi)


def scaled(x, e):
    return x * 2.0 ** -np.repeat(e, GROUP, 1)[:, :x.shape[1]].astype(np.float64)


def round8(x):
    """(values on the e4m3 grid, exponents); NaN and infinities become NaN."""
    x = np.asarray(x, np.float64)
    e = exponents(x, 448.0)
    z = scaled(np.where(np.isfinite(x), x, 0), e)
    v = np.copysign(E4M3[nearest(z, E4M3)], z)
    return np.where(np.isfinite(x), v, np.nan), e


def round4(w):
    """(values on the e2m1 grid, exponents, groups that are NaN)."""
    w = np.asarray(w, np.float64)
    n, K = w.shape
    bad = np.zeros((n, up(K, GROUP)), bool)
    bad[:, :K] = ~np.isfinite(w)
    bad = bad.reshape(n, -1, GROUP).any(-1)
    e = exponents(w, 6.0)
    z = scaled(np.where(np.isfinite(w), w, 0), e)
    return np.copysign(E2M1[nearest(z, E2M1)], z), e, bad


def tile_index(n, K):
    """Place of the scale byte of each row < n and group < 4 ceil(K / 128)."""
    r, g = np.arange(n)[:, None], np.arange(up(K, 128) // 32)
    return ((r // 128) * (up(K, 128) // 128) + g // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + g % 4


def tiles(byte, K, fill=0):
    """Scale bytes [rows, groups] in their tiles; rows that do not exist hold ``fill``."""
    n = byte.shape[0]
    at = tile_index(n, K)
    out = np.full(up(n, 128) * up(K, 128) // 32, fill, np.uint8)
    full = np.full(at.shape, 127, np.uint8)
    full[:, :byte.shape[1]] = byte
    out[at] = full
    return out


def pack4(w):
    """Codes and scale tiles of weights."""
    n, K = w.shape
    v, e, bad = round4(w)
    code = nearest(v, E2M1) + 8 * (v < 0)
    code[np.repeat(bad, GROUP, 1)[:, :K]] = 0
    full = np.zeros((n, up(K, 128)), np.uint8)
    full[:, :K] = code
    return full[:, 0::2] | (full[:, 1::2] << 4), tiles(np.where(bad, 255, e + 127).astype(np.uint8), K)


def pack8(x):
    """Bytes [rows, ld] and scale tiles of rows."""
    n, K = x.shape
    v, e = round8(x)
    code = np.zeros((n, up(K, 16)), np.uint8)
    code[:, :K] = np.where(np.isnan(v), 127, nearest(np.nan_to_num(v), E4M3) + 128 * (v < 0))
    return code, tiles((e + 127).astype(np.uint8), K)


def power(byte):
    return np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))


def unpack4(codes, scale, n, K):
    full = np.empty((n, 2 * codes.shape[1]), np.uint8)
    full[:, 0::2], full[:, 1::2] = codes & 15, codes >> 4
    s = power(scale.reshape(-1)[tile_index(n, K)])
    return (VALUE4[full] * np.repeat(s, GROUP, 1))[:, :K]


def unpack8(codes, scale, n, K):
    s = power(scale.reshape(-1)[tile_index(n, K)])
    return VALUE8[codes[:, :K]] * np.repeat(s, GROUP, 1)[:, :K]


def rows(rs, n, K):
    """Rows as a model's layers have them: of unlike size, a few channels loud."""
    x = rs.standard_normal((n, K)) * 2.0 ** rs.uniform(-1, 1, (n, 1))
    return x * np.where(rs.uniform(size=K) < 0.01, 8.0, 1.0)
