"""Attention over the 8-bit cache where the pages' values differ by many powers
of two and so do their weights, against a 64-bit restatement.

The bound is in terms of what a row sums up: A = sum p_j |v_j|, weighted, and
not the largest |v|.  A relative error e in every weight and an error d in every
score (see kv8_util.tolerance) move o = sum p_j v_j / sum p_j by at most
(2 d + 2 e) A.  A weight times its block's scale 2^e_j goes into the products as
f16 values: the largest p_j 2^e_j of the row stands at 2^6 at least, so that
f16's smallest step, 2^-24, rounds every key's by at most 2^-31 of the largest;
with codes of at most 448, n keys add n 2^-31 C, C = 448 max p_j 2^e_j.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import kv8_util as ref  # noqa: E402
from test_kv8_gpu import EPS, Setup, b  # noqa: E402, F401  (b: the fixture)


def weighted(s, cache):
    """(A, C, n): A [T, H, hd], C [T, H] and the number of keys [T] of each row."""
    A, C, n_keys = np.zeros((s.T, s.H, s.hd)), np.zeros((s.T, s.H)), np.ones(s.T)
    for i in range(s.B):
        r0, n, p0 = int(s.row0[i]), int(s.new[i]), int(s.pos[i])
        if n == 0 or p0 < 0:
            continue
        x = s.qkv[r0:r0 + n, :(s.H + 2 * s.Hkv) * s.hd].reshape(n, -1, s.hd)
        q = ref.norm_rope(x[:, :s.H], s.qg, s.cos[p0:p0 + n], s.sin[p0:p0 + n], EPS)
        k, v, ok = cache.keys_values(s.table[i], p0 + n)
        pages = np.where(ok, s.table[i][np.arange(p0 + n) // 16], 0)
        see = ok[None] & (np.arange(p0 + n)[None] <= (p0 + np.arange(n))[:, None])
        n_keys[r0:r0 + n] = p0 + n
        for h in range(s.H):
            g = h // (s.H // s.Hkv)
            z = np.where(see, q[:, h] @ k[:, g].T / np.sqrt(s.hd), -np.inf)
            top = z.max(-1, keepdims=True)
            w = np.where(see, np.exp(z - np.where(np.isfinite(top), top, 0)), 0.0)
            w /= np.maximum(w.sum(-1, keepdims=True), 1e-300)
            A[r0:r0 + n, h] = w @ np.abs(v[:, g])
            C[r0:r0 + n, h] = 448 * (w * 2.0 ** cache.exps[pages, 1, g].astype(float)).max(-1)
    return A, C, n_keys


def check(s, o, bf16, planes):
    cache, want, SV = s.want()
    got = o.float().cpu().numpy()[:s.T, :s.H * s.hd].reshape(want.shape).astype(np.float64)
    A, C, n = weighted(s, cache)
    u = 2.0 ** -17 + (2.0 ** -11 if planes == 1 else 0)
    e = 2.0 ** -16 + (2.0 ** -11 if planes == 1 else 0)
    tol = (2 * SV[..., :1] * u + 2 * e) * A + (n[:, None] * 2.0 ** -31 * C)[..., None]
    tol += (2.0 ** -8 if bf16 else 2.0 ** -23) * np.abs(want) + 1e-40
    err = np.abs(got - want)
    assert (err <= tol).all(), (float((err / tol).max()), np.argwhere(err > tol)[:5].tolist())
    return want


def shifted(s, by):
    """All values, cached and new, times 2^by."""
    s.exps[:, 1] = np.clip(s.exps[:, 1] + by, -32, 32)
    s.qkv[:, (s.H + s.Hkv) * s.hd:(s.H + 2 * s.Hkv) * s.hd] *= np.float32(2.0 ** by)


def turned_away(s, i, page, lam, by):
    """Keys of this page of sequence i away from all queries (scores of about
    -lam sqrt(hd)), its values times 2^by.  Every query is one vector in the dims
    that turn slowly, so that rows at all positions see it alike."""
    half = s.hd // 2
    u = np.zeros(s.hd, np.float32)
    u[half // 2:half] = u[half + half // 2:] = 1.0
    s.qkv[:, :s.H * s.hd] = np.tile(u, s.H)
    p0 = int(s.pos[i])
    q = ref.norm_rope(u[None, None], s.qg, s.cos[p0:p0 + 1], s.sin[p0:p0 + 1], EPS)[0, 0]
    x = np.broadcast_to(-lam * q * np.sqrt(s.hd) / np.linalg.norm(q), (s.Hkv, 16, s.hd))
    p = s.table[i, page]
    s.exps[p, 0] = ref.exponent(x)
    s.codes[p, 0] = ref.encode(x / 2.0 ** s.exps[p, 0][:, None, None])
    s.exps[p, 1] += by
    assert np.abs(s.exps[p]).max() <= 32


# ---------------------------------------------------------------- pages that are not there

@pytest.mark.parametrize("kind", ["decode", "prefill"])
@pytest.mark.parametrize("missing", [0, 2, 4])
def test_small_values_beside_a_missing_page(b, kind, missing):
    s = Setup([100, 70], [2, 1] if kind == "prefill" else [2, 2], 4, 2, 128, seed=31)
    s.table[0, missing] = -1
    s.table[1, missing] = s.n_pages
    shifted(s, -26)
    s.upload()
    o, _ = s.run(b, kind, False)
    torch.cuda.synchronize()
    want = check(s, o, False, 2)
    assert (want != 0).any()
