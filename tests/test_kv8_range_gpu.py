"""Attention over the 8-bit cache where the pages' values differ by many powers
of two and so do their weights, against a 64-bit restatement.

The bound is in terms of what a row sums up: A = sum p_j |v_j|, weighted, and
not the largest |v|.  A relative error e in every weight and an error d in every
score (see kv8_util.tolerance) move o = sum p_j v_j / sum p_j by at most
(2 d + 2 e) A.  A weight times its block's scale, p_j 2^e_j, goes into the products
as f16 values: the row's largest stands at 2^6 at least, so that f16's smallest
step, 2^-24, rounds every other by at most 2^-31 of it.  A block's scale may be far
above what the row sees of the block, so the largest one counts only among blocks
whose scale is at most 2^10 times key j's; if it is in another block, key j's
block stands at 2^-4 at least or by itself: 2^-21 of the block's largest p_j 2^e_j,
or 2^-95 of the row's largest.  That times the key's largest code is its error.
In prompts the largest stands at 2^11 at least (2^7 with a bf16 output), a step is
2^-36 (2^-32) of it, and the blocks of 128 keys count as of the largest of their
scales, which is at most 2^14 times the scale of each: 2^-22 (2^-18) of the row's
largest p_j 2^e_j.  And a block more than 2^14 below the largest scale met stands by
itself, so that no more than the largest weight among blocks of up to 2^14 times key
j's scale counts for j, at that scale: 2^-22 (2^-18) of this weight times 2^e_j.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import kv8_util as ref  # noqa: E402
from test_kv8_gpu import EPS, Setup, b  # noqa: E402, F401  (b: the fixture)


def weighted(s, cache, prompt, bf16):
    """(A, D): A [T, H, hd], and D [T, H], the sum over a row's keys of what f16's smallest step can move."""
    A, D = np.zeros((s.T, s.H, s.hd)), np.zeros((s.T, s.H))
    for i in range(s.B):
        r0, n, p0 = int(s.row0[i]), int(s.new[i]), int(s.pos[i])
        if n == 0 or p0 < 0:
            continue
        x = s.qkv[r0:r0 + n, :(s.H + 2 * s.Hkv) * s.hd].reshape(n, -1, s.hd)
        q = ref.norm_rope(x[:, :s.H], s.qg, s.cos[p0:p0 + n], s.sin[p0:p0 + n], EPS)
        k, v, ok = cache.keys_values(s.table[i], p0 + n)
        v = np.where(ok[:, None, None], v, 0.0)
        at = np.arange(p0 + n) // 16
        pages = np.where(ok, s.table[i][at], 0)
        see = ok[None] & (np.arange(p0 + n)[None] <= (p0 + np.arange(n))[:, None])
        for h in range(s.H):
            g = h // (s.H // s.Hkv)
            z = np.where(see, q[:, h] @ k[:, g].T / np.sqrt(s.hd), -np.inf)
            top = z.max(-1, keepdims=True)
            w = np.where(see, np.exp(z - np.where(np.isfinite(top), top, 0)), 0.0)
            w /= np.maximum(w.sum(-1, keepdims=True), 1e-300)
            A[r0:r0 + n, h] = w @ np.abs(v[:, g])
            e = cache.exps[pages, 1, g]
            c = w * 2.0 ** e.astype(float)                                   # [n, keys]
            block = np.stack([c[:, at == p].max(-1) for p in range(at[-1] + 1)], -1)
            far = np.stack([np.where(e <= e[16 * p] + 10, c, 0).max(-1) for p in range(at[-1] + 1)], -1)
            step = np.maximum(np.maximum(2.0 ** -31 * far, 2.0 ** -21 * block),
                              2.0 ** -95 * block.max(-1, keepdims=True))
            if prompt:
                near = np.stack([np.where(e <= e[16 * p] + 14, w, 0).max(-1) for p in range(at[-1] + 1)], -1)
                step = (2.0 ** -18 if bf16 else 2.0 ** -22) * np.minimum(near * 2.0 ** e[::16],
                                                                       block.max(-1, keepdims=True))
            D[r0:r0 + n, h] = step[:, at] @ (np.abs(v[:, g]).max(-1) / 2.0 ** e)     # codes of 448 at most
    return A, D


def check(s, o, bf16, planes, prompt=False):
    cache, want, SV = s.want()
    got = o.float().cpu().numpy()[:s.T, :s.H * s.hd].reshape(want.shape).astype(np.float64)
    A, D = weighted(s, cache, prompt, bf16)
    u = 2.0 ** -17 + (2.0 ** -11 if planes == 1 else 0)
    e = 2.0 ** -16 + (2.0 ** -11 if planes == 1 else 0)
    tol = (2 * SV[..., :1] * u + 2 * e) * A + D[..., None]
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
    if by == "zeros":
        s.codes[p, 1], by = 0, 40
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
    want = check(s, o, False, 2, kind == "prefill")
    assert (want != 0).any()


# ---------------------------------------------------------------- large values with little weight

# lam: the page's weights are e^(-lam sqrt(hd)) of the others'; by: its values are 2^by of theirs
FAR = [
    (4.5, 24),     # nothing of the page is left: the others' values stand alone
    (3.0, 12),     # the same with values that f16 holds beside each other
    (3.0, 14),     # the last scale that prompts take together with the others'
    (3.0, 15),     # the first that they do not
    (3.0, 45),     # weights of 2^-49, values of 2^45: both count
    (2.0, 48),     # weights of 2^-33: the page is all that counts
    (-3.0, -12),   # the page has all the weight, the others values of 2^12: both count
    (0.0, 40),     # equal weights
    (0.0, "zeros"),   # equal weights, and zeros in a block whose scale is 2^40 times the others'
    (-2.0, "zeros"),  # the same with the weight on the zeros
]


@pytest.mark.parametrize("page", [0, 3, 5])
@pytest.mark.parametrize("lam,by", FAR)
def test_decode_of_far_values(b, lam, by, page):
    s = Setup([100, 99], [2, 2], 8, 4, 128, seed=32)
    shifted(s, -8 if by == -12 else -20)
    for i in range(2):
        turned_away(s, i, page, lam, by)
    s.upload()
    o, _ = s.run(b, "decode", False)
    torch.cuda.synchronize()
    check(s, o, False, 2)


@pytest.mark.parametrize("lam,by", FAR)
def test_decode_of_far_values_in_another_run(b, lam, by):
    """A long sequence, cut into runs: pages of the kind in different ones."""
    s = Setup([3000, 40], [1, 1], 8, 2, 64, seed=33)
    shifted(s, -8 if by == -12 else -20)
    turned_away(s, 0, 3, lam, by)
    turned_away(s, 0, 150, lam, by)
    s.upload()
    o, ws = s.run(b, "decode", True)
    torch.cuda.synchronize()
    check(s, o, True, 2)


@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
@pytest.mark.parametrize("page", [0, 5])
@pytest.mark.parametrize("lam,by", FAR)
def test_prompt_of_far_values(b, lam, by, page, bf16):
    s = Setup([150, 99, 600], [70, 1, 3], 4, 2, 128, seed=34)
    shifted(s, -8 if by == -12 else -20)
    for i in range(3):
        turned_away(s, i, page, lam, by)
    s.upload()
    o, _ = s.run(b, "prefill", bf16)
    torch.cuda.synchronize()
    check(s, o, bf16, 1 if bf16 else 2, True)


@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
@pytest.mark.parametrize("lam,by", FAR)
def test_prompt_of_far_values_in_another_range(b, lam, by, bf16):
    """Few rows behind many keys, which are cut into ranges."""
    s = Setup([2000], [3], 4, 2, 64, seed=35)
    shifted(s, -8 if by == -12 else -20)
    turned_away(s, 0, 3, lam, by)
    turned_away(s, 0, 100, lam, by)
    s.upload()
    o, _ = s.run(b, "prefill", bf16)
    torch.cuda.synchronize()
    check(s, o, bf16, 1 if bf16 else 2, True)


@pytest.mark.parametrize("seed", range(30))
def test_calls_at_random(b, seed):
    """Head layouts, lengths, value scales, missing pages and blocks of zeros at random."""
    r = np.random.default_rng(1000 + seed)
    Hkv, G, hd, B = r.choice([1, 2, 3, 5]), r.choice([1, 2, 3, 4, 8]), int(r.choice([64, 128])), r.choice([1, 2, 3, 7])
    H, Hkv, kind, bf16 = int(Hkv * G), int(Hkv), ["decode", "prefill"][seed % 2], bool(r.integers(2))
    pos = r.choice([0, 3, 15, 16, 40, 130, 300, 777, 1500], B) + r.integers(0, 20, B)
    new = np.full(B, r.integers(1, 8 // G + 1)) if kind == "decode" else r.choice([1, 2, 17, 64, 150], B)
    s = Setup(pos, new, H, Hkv, hd, seed=seed, pad=int(r.choice([0, 4, 3])), spread=float(r.choice([0, 2, 6, 9, 18])))
    s.exps[:, 0] = np.clip(s.exps[:, 0], -9, -6)              # keys of ordinary sizes
    s.qg *= np.float32(r.choice([1, 1, 4]))
    v = s.qkv[:, (H + Hkv) * hd:(H + 2 * Hkv) * hd]
    v *= (2.0 ** (r.integers(-20, 21, s.T + 2) * r.integers(0, 2)))[:, None].astype(np.float32)
    if seed % 3 == 0:
        for i in r.integers(0, B, 3):
            s.table[i, r.integers(0, (pos[i] + new[i] + 15) // 16)] = r.choice([-1, s.n_pages, 1 << 30])
    if seed % 4 == 0:
        s.codes[r.integers(0, s.n_pages, 4), 1] = 0
    s.upload()
    o, _ = s.run(b, kind, bf16)
    torch.cuda.synchronize()
    check(s, o, bf16, 1 if bf16 and kind == "prefill" else 2, kind == "prefill")
