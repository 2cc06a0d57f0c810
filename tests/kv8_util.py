"""The 8-bit KV cache in 64 bits, in NumPy: a plain restatement of the
definitions in include/s2_ops.h for the tests of its kernels."""

import numpy as np

PAGE, EMIN, EMAX = 16, -32, 32

# value of every e4m3 code: sign, 4 exponent bits (bias 7), 3 mantissa bits,
# 0x7f / 0xff NaN
_c = np.arange(128)
_pos = np.where(_c // 8 == 0, (_c % 8) / 512.0, (1 + (_c % 8) / 8.0) * 2.0 ** (_c // 8 - 7.0))
_pos[127] = np.nan
VALUE = np.concatenate([_pos, -_pos])


def encode(x):
    """Codes of the nearest e4m3 values, ties to even, saturating; NaN 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    nan = np.isnan(x)
    a = np.where(nan, 0.0, a)
    hi = np.minimum(np.searchsorted(_pos[:127], a), 126)
    lo = np.maximum(hi - 1, 0)
    down, up = a - _pos[lo], _pos[hi] - a
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    code = np.where(nan, 127, code)
    return (code + np.where(np.signbit(x) & ~nan, 128, 0)).astype(np.uint8)


def same_codes(a, b):
    """Equal codes, any NaN equal to any NaN and -0 to 0."""
    va, vb = VALUE[a], VALUE[b]
    return (va == vb) | (np.isnan(va) & np.isnan(vb))


def exponent(x):
    """The scale exponent of blocks over the last two dimensions."""
    m = np.where(np.isnan(x), 0.0, np.abs(x))
    m = m.max((-1, -2), initial=0.0)
    e = np.full(m.shape, EMAX)
    for k in range(EMAX - 1, EMIN - 1, -1):
        e = np.where(m <= 448.0 * 2.0 ** k, k, e)
    return e


def norm_rope(x, gain, cos, sin, eps):
    """x [n, heads, hd] normed, rotated; cos, sin [n, hd/2]."""
    x = x.astype(np.float64)
    h = x.shape[-1] // 2
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + float(np.float32(eps))) * gain.astype(np.float64)
    c, s = cos.astype(np.float64)[:, None], sin.astype(np.float64)[:, None]
    return np.concatenate([y[..., :h] * c - y[..., h:] * s, y[..., h:] * c + y[..., :h] * s], -1)


class Cache:
    """codes uint8 [pages, 2, Hkv, 16, hd], exponents int [pages, 2, Hkv]."""

    def __init__(self, codes, exps):
        self.codes, self.exps = codes.copy(), exps.copy()

    def append(self, table, pos, k, v):
        """Rows k, v [n, Hkv, hd] at positions pos.. of the sequence with this table row."""
        n, n_pages = len(k), len(self.codes)
        if n == 0:
            return
        for j in range(pos // PAGE, (pos + n - 1) // PAGE + 1):
            p = int(table[j])
            if not 0 <= p < n_pages:
                continue
            lo, hi = max(pos, j * PAGE), min(pos + n, (j + 1) * PAGE)
            had = lo - j * PAGE
            for t, x in ((0, k), (1, v)):
                z = x[lo - pos:hi - pos].transpose(1, 0, 2).astype(np.float64)
                e_old = self.exps[p, t] if had else np.full(z.shape[0], EMIN)
                e = np.maximum(exponent(z), e_old)
                grow = 2.0 ** (e_old - e)[:, None, None]
                moved = encode(VALUE[self.codes[p, t, :, :had]] * grow)
                keep = (e_old == e)[:, None, None]
                self.codes[p, t, :, :had] = np.where(keep, self.codes[p, t, :, :had], moved)
                self.codes[p, t, :, had:had + hi - lo] = encode(z / 2.0 ** e[:, None, None])
                self.exps[p, t] = e

    def keys_values(self, table, n):
        """k, v [n, Hkv, hd] and which of the n keys have a page."""
        j = np.arange(n) // PAGE
        pages = np.asarray(table)[j].astype(np.int64)
        ok = (pages >= 0) & (pages < len(self.codes))
        q = np.where(ok, pages, 0)
        x = VALUE[self.codes[q, :, :, np.arange(n) % PAGE]] * 2.0 ** self.exps[q][..., None].astype(np.float64)
        return x[:, 0], x[:, 1], ok


def attention(cache, qkv, H, Hkv, hd, row0, pos, table, q_gain, k_gain, eps, cos, sin, max_pos, o):
    """Appends and attends; sequence b has the rows row0[b]..row0[b+1]-1 of
    qkv at pos[b].. .  Writes o [T, H, hd] (float64), and returns for each row
    (S, V): the largest sum |q_i k_ij| / sqrt(hd) over its keys, and the
    largest |v|, the scale of the rounding errors."""
    B = len(pos)
    T = len(o)
    SV = np.zeros((T, H, 2))
    G = H // Hkv
    work = []
    for b in range(B):
        r0, n, p0 = int(row0[b]), int(row0[b + 1] - row0[b]), int(pos[b])
        if n <= 0:
            continue
        if p0 < 0 or p0 + n > max_pos:
            o[r0:r0 + n] = 0
            continue
        x = qkv[r0:r0 + n].reshape(n, H + 2 * Hkv, hd)
        q = norm_rope(x[:, :H], q_gain, cos[p0:p0 + n], sin[p0:p0 + n], eps)
        k = norm_rope(x[:, H:H + Hkv], k_gain, cos[p0:p0 + n], sin[p0:p0 + n], eps)
        cache.append(table[b], p0, k, x[:, H + Hkv:])
        work.append((b, r0, n, p0, q))
    for b, r0, n, p0, q in work:
        k, v, ok = cache.keys_values(table[b], p0 + n)
        for h in range(H):
            g = h // G
            s = q[:, h] @ k[:, g].T / np.sqrt(hd)
            sa = np.abs(q[:, h]) @ np.abs(k[:, g]).T / np.sqrt(hd)
            see = ok[None] & (np.arange(p0 + n)[None] <= (p0 + np.arange(n))[:, None])
            s = np.where(see, s, -np.inf)
            m = s.max(-1, keepdims=True)
            w = np.where(see, np.exp(s - np.where(np.isfinite(m), m, 0)), 0.0)
            l = w.sum(-1, keepdims=True)
            vg = v[:, g]
            bad = np.isnan(vg)
            y = w @ np.where(bad, 0.0, vg) / np.where(l > 0, l, 1)
            y = np.where((see.astype(np.float64) @ bad) > 0, np.nan, y)   # NaN only where it is seen
            o[r0:r0 + n, h] = np.where(l == 0, 0.0, y)
            SV[r0:r0 + n, h, 0] = np.where(see, np.nan_to_num(sa), 0).max(-1)
            SV[r0:r0 + n, h, 1] = np.where(see[..., None], np.nan_to_num(np.abs(vg))[None], 0).max((1, 2))
    return SV


def tolerance(SV, ref, bf16, planes=2):
    """How far an output may be from the 64-bit one.

    o = sum p_j v_j with weights that sum to 1: an error d in every score and
    a relative error e in every weight move o by at most (2 d + 2 e) max |v|.
    d <= S u, S = sum |q_i k_i| / sqrt(hd).  u for f16 pairs (planes = 2):
    the norm, gain and rotation of q in fp32 (at most 8 roundings of 2^-24),
    the pair (2^-22 = 4 x 2^-24), at most 32 accumulating steps in fp32
    (2 x 2^-24 each) and the scaling: under 2^-17.  For one f16 plane: 2^-11
    more.  e: the exponent's argument (beyond |x| = 2^6 a weight is nothing:
    2^6 x 2^-24 = 2^-18), exp2 itself and the pair (2^-21), and the sums of
    weights and products: fp32 in runs of one tile, joined over at most 2^9
    tiles and 2^6 parts, whose errors of at most 2^-24 a step add up like a
    random walk at the lengths here (sqrt(2^9) x 2^-24 < 2^-19): together
    under 2^-16; one f16 plane: 2^-11 more.
    bf16 output: half a step, 2^-8 of the value."""
    u = 2.0 ** -17 + (2.0 ** -11 if planes == 1 else 0)
    e = 2.0 ** -16 + (2.0 ** -11 if planes == 1 else 0)
    t = (2 * SV[..., :1] * u + 2 * e) * SV[..., 1:]
    r = np.where(np.isfinite(ref), np.abs(ref), 0)
    return t + (2.0 ** -8 * r if bf16 else 2.0 ** -23 * r) + 1e-30
