"""4-bit weights and 8-bit rows with scales on the GPU, against their definitions in 64 bits (mx_util.py)."""

import numpy as np
import pytest

import mx_util as U

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def s2():
    from serving_dual_ar_gb300 import buildlib
    buildlib.build()
    from serving_dual_ar_gb300 import binding
    assert torch.cuda.is_available()
    return binding


TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def dev(a, kind=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if kind is None else t.to(TYPES[kind])


def host(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def strided(a, kind, ld, shift=0):
    """Rows a at pitch ld, ``shift`` elements into a buffer of NaN."""
    n, K = a.shape
    buf = torch.full((shift + n * ld + 8,), float("nan"), dtype=TYPES[kind], device="cuda")
    view = buf[shift:shift + n * ld].view(n, ld)
    view[:, :K] = dev(a).to(TYPES[kind])
    return view


def guarded(nbytes, fill=0xAB):
    return torch.full((nbytes,), fill, dtype=torch.uint8, device="cuda")


def same(a, b):
    return np.array_equal(a, b) or bool(((a == b) | (np.isnan(a) & np.isnan(b))).all())


# ---------------------------------------------------------------- packing

def special_rows(K, rs, top):
    """Rows with what rounding and scales can go wrong on."""
    x = rs.standard_normal((12, K))
    x[0] = 0
    x[1] = top * 2.0 ** rs.randint(-8, 8, K)                   # largest magnitudes on the border of a scale
    x[2] = np.nextafter(np.float32(top), np.float32(1e9)) * np.sign(x[2])
    x[3] *= 1e-41                                              # fp32 subnormals
    x[4] *= 1e30
    x[5, ::7] = 0.0
    x[6] = (rs.randint(0, 512, K) - 256) / 32.0                # many ties
    x[7, K // 2] = 2.0 ** 40                                   # all else far below
    x[8] = 2.0 ** -30
    x[9, 0] = 3.3e38
    return x


SHAPES = [(1, 1), (12, 31), (12, 32), (12, 33), (12, 129), (40, 1000), (130, 256)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 1)])
@pytest.mark.parametrize("n,K", SHAPES)
def test_mx8_pack(s2, n, K, kind, pad, shift):
    rs = np.random.RandomState(n * 1000 + K)
    x = U.rows(rs, n, K) if n != 12 else special_rows(K, rs, 448.0)
    t = strided(x, kind, K + pad, shift)
    x = host(t[:, :K])
    ld8 = U.up(K, 16) + 16
    y8, sc = guarded(n * ld8), guarded(s2.s2op_mx_scale_bytes(n, K))
    s2.s2op_mx8_pack(t, kind == "bf16", K + pad, n, K, y8, ld8, sc)
    y8 = host(y8).reshape(n, ld8)
    v, e = U.round8(x)
    assert same(U.VALUE8[y8[:, :K]], v)
    assert (y8[:, K:] == 0xAB).all()                           # behind the rows nothing is written
    assert np.array_equal(host(sc), U.tiles((e + 127).astype(np.uint8), K, 0xAB))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_mx8_pack_nan_and_infinities(s2, kind):
    x = np.random.RandomState(1).standard_normal((3, 96))
    x[0, 3], x[1, 40], x[2, 95] = np.nan, np.inf, -np.inf
    x[2, 64:] = np.nan                                         # a group with nothing else
    t = strided(x, kind, 96)
    y8, sc = guarded(3 * 96), guarded(512)
    s2.s2op_mx8_pack(t, kind == "bf16", 96, 3, 96, y8, 96, sc)
    v, e = U.round8(host(t))
    assert same(U.VALUE8[host(y8).reshape(3, 96)], v)
    assert np.array_equal(host(sc), U.tiles((e + 127).astype(np.uint8), 96, 0xAB))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 1)])
@pytest.mark.parametrize("n,K", SHAPES)
def test_w4_pack_and_unpack(s2, n, K, kind, pad, shift):
    rs = np.random.RandomState(n * 1000 + K)
    w = 0.02 * rs.standard_normal((n, K)) if n != 12 else special_rows(K, rs, 6.0)
    t = strided(w, kind, K + pad, shift)
    w = host(t[:, :K])
    codes, sc = guarded(s2.s2op_w4_code_bytes(n, K)), guarded(s2.s2op_mx_scale_bytes(n, K))
    s2.s2op_w4_pack(t, kind == "bf16", n, K, K + pad, codes, sc)
    v, e, bad = U.round4(w)
    got = host(codes).reshape(n, -1)
    full = np.empty((n, 2 * got.shape[1]), np.uint8)
    full[:, 0::2], full[:, 1::2] = got & 15, got >> 4
    assert np.array_equal(U.VALUE4[full[:, :K]], v) and not full[:, K:].any()
    assert np.array_equal(host(sc), U.tiles((e + 127).astype(np.uint8), K, 0xAB))
    for back in ("f32", "bf16"):
        out = strided(np.zeros((n, K)), back, K + pad, shift)
        s2.s2op_w4_unpack(codes, sc, n, K, out, back == "bf16", K + pad)
        assert np.array_equal(host(out[:, :K]), U.unpack4(got, host(sc), n, K))
        assert bool(torch.isnan(out[:, K:]).all())


def test_w4_pack_nan(s2):
    w = np.random.RandomState(2).standard_normal((4, 128)).astype(np.float32)
    w[0, 5], w[1, 64], w[3, 127] = np.nan, np.inf, -np.inf
    codes, sc, out = guarded(4 * 64), guarded(512), torch.zeros(4, 128, device="cuda")
    s2.s2op_w4_pack(dev(w), False, 4, 128, 128, codes, sc)
    s2.s2op_w4_unpack(codes, sc, 4, 128, out, False, 128)
    v, e, bad = U.round4(w)
    assert same(host(out), np.where(np.repeat(bad, 32, 1), np.nan, v * 2.0 ** np.repeat(e, 32, 1)))


# ---------------------------------------------------------------- residual and norm

def norm64(h, gain, eps):
    with np.errstate(all="ignore"):
        return h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * gain


def run_norm(s2, x, r, gain, eps, tx, tr, pad=0, shift=0, in_place=False):
    n, K = x.shape
    ld8 = U.up(K, 16)
    X = strided(x, tx, K + pad, shift)
    R = None if r is None else strided(r, tr, K + pad, shift)
    H = X if in_place else strided(np.zeros((n, K)), tx, K + pad, shift)
    x0, r0 = host(X[:, :K]), 0 if r is None else host(R[:, :K])
    y8, sc = guarded(n * ld8), guarded(s2.s2op_mx_scale_bytes(n, K))
    s2.s2op_add_rmsnorm_mx8(X, tx == "bf16", K + pad, R, tr == "bf16", K + pad, n, K, dev(gain.astype(np.float32)), eps,
                            H, K + pad, y8, ld8, sc)
    h = host(dev((x0 + r0).astype(np.float32), tx))             # rounded to fp32, then to x's type
    assert same(host(H[:, :K]), h)
    y8 = host(y8).reshape(n, ld8)
    assert (y8[:, K:] == 0xAB).all()
    return h, y8[:, :K], host(sc)


@pytest.mark.parametrize("tx,tr", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("n,K,pad,shift", [(1, 1, 0, 0), (1, 2560, 0, 0), (3, 33, 1, 1), (130, 256, 8, 0), (5, 1000, 0, 0),
                                           (2, 4104, 0, 0), (2, 9728, 0, 0), (2, 17000, 3, 1)])
def test_add_rmsnorm(s2, n, K, pad, shift, tx, tr):
    rs = np.random.RandomState(K)
    gain = rs.uniform(0.5, 1.5, K).astype(np.float32)
    h, y8, sc = run_norm(s2, U.rows(rs, n, K), 0.3 * U.rows(rs, n, K), gain, 1e-6, tx, tr, pad, shift)
    v, e = U.round8(norm64(h, gain.astype(np.float64), float(np.float32(1e-6))))
    assert same(U.VALUE8[y8], v)
    assert np.array_equal(sc, U.tiles((e + 127).astype(np.uint8), K, 0xAB))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("with_r", [False, True])
def test_add_rmsnorm_in_place_and_without_residual(s2, with_r, in_place):
    rs = np.random.RandomState(5)
    x, r, gain = U.rows(rs, 7, 768), U.rows(rs, 7, 768), rs.uniform(-2, 2, 768).astype(np.float32)
    h, y8, sc = run_norm(s2, x, r if with_r else None, gain, 1e-5, "f32", "f32", in_place=in_place)
    v, e = U.round8(norm64(h, gain.astype(np.float64), float(np.float32(1e-5))))
    assert same(U.VALUE8[y8], v)


@pytest.mark.parametrize("K", [64, 3000, 20000])
def test_add_rmsnorm_range(s2, K):
    """Rows whose squares leave fp32's range, rows of zeros, NaN and infinities."""
    rs = np.random.RandomState(6)
    x = U.rows(rs, 9, K)
    for i, f in enumerate([1e-40, 1e-25, 1e-15, 1e-6, 1e15, 1e25, 1e37]):
        x[i] *= f
    x[5] = np.where(rs.uniform(size=K) < 0.1, x[5], 1e-3)
    x = np.clip(x, -3e38, 3e38)
    x[8, K // 2] = np.nan
    gain = rs.uniform(0.5, 1.5, K).astype(np.float32)
    for eps in (0.0, 1e-12, 1e-6):
        h, y8, sc = run_norm(s2, x, None, gain, eps, "f32", "f32")
        v, e = U.round8(norm64(h, gain.astype(np.float64), float(np.float32(eps))))
        assert np.isnan(U.VALUE8[y8[8]]).all()
        assert same(U.VALUE8[y8[:8]], v[:8]), eps
    x[3], x[4, 1] = 0, np.inf
    h, y8, sc = run_norm(s2, x, None, gain, 1e-6, "f32", "f32")
    assert not U.VALUE8[y8[3]].any() and np.isnan(U.VALUE8[y8[4]]).all()
    h, y8, sc = run_norm(s2, x, None, gain, 0.0, "f32", "f32")
    assert np.isnan(U.VALUE8[y8[3]]).all()


# ---------------------------------------------------------------- products

# Error of one output, relative to A = sum_k |x w| (the sum may cancel): products are exact; a tensor core adds 32 of
# them to the running sum and cuts each term below 2^-23 of the largest, at most 34 terms; at most 32 such steps run
# into one another before the sum goes to fp32 registers; then one rounding of 2^-24 for each 512 of K and each of at
# most 16 parts of a sum.  Terms that are cut one after another do not all lean one way to their full size, but the
# bound lets them.
def sum_bound(K):
    return 34 * 32 * 2.0 ** -23 / 32 + (K / 512 + 17) * 2.0 ** -24


def bounds(A, v, y0, want, kind, mode, K):
    """Allowed error of each output; v: the products in 64 bits (both, for SwiGLU)."""
    d = sum_bound(K) * A
    if mode == 2:
        g, u, dg, du = v[:, 0::2], v[:, 1::2], d[:, 0::2], d[:, 1::2]
        silu = g / (1 + np.exp(-g))
        # |silu'| < 1.1; exp, quotient and product round to a few units each
        d = 1.1 * dg * (np.abs(u) + du) + (np.abs(silu) + 1.1 * dg) * du + 8 * 2.0 ** -24 * np.abs(silu * u)
    if mode == 1:
        d = d + 2.0 ** -24 * (np.abs(want) + d)
    return d + (2.0 ** -8 if kind == "bf16" else 2.0 ** -24) * (np.abs(want) + d) + 1e-45


def product64(x, w, y0, mode):
    v = x @ w.T
    if mode == 2:
        with np.errstate(over="ignore"):
            return v, v[:, 0::2] / (1 + np.exp(-v[:, 0::2])) * v[:, 1::2]
    return v, y0 + v if mode == 1 else v


def weights(rs, N, K):
    w = rs.standard_normal((N, K)) * 2.0 ** rs.uniform(0, 1, (N, 1)) * K ** -0.5
    codes, sc = U.pack4(w)
    return U.unpack4(codes, sc, N, K), dev(codes), dev(sc)


def check_product(s2, rs, T, N, K, ty, mode, x_kind=None, pad=0, shift=0, x=None, w=None):
    wv, codes, sc = weights(rs, N, K) if w is None else w
    x = U.rows(rs, T, K) if x is None else x
    cols = N // 2 if mode == 2 else N
    y0 = rs.standard_normal((T, cols))
    Y = strided(y0, ty, cols + pad, shift)
    y0 = host(Y[:, :cols])
    if x_kind is None:
        x8, xs = U.pack8(x)
        xv = U.unpack8(x8, xs, T, K)
        s2.s2op_w4_gemm(codes, sc, N, K, dev(x8), x8.shape[1], dev(xs), T, Y, ty == "bf16", cols + pad, mode)
    else:
        X = strided(x, x_kind, K + pad, shift)
        xv = host(X[:, :K])
        ws = guarded(s2.s2op_w4_gemv_workspace_bytes(K, T), 0xFF)
        s2.s2op_w4_gemv(codes, sc, N, K, X, x_kind == "bf16", K + pad, T, Y, ty == "bf16", cols + pad, mode, ws)
    v, want = product64(xv, wv, y0, mode)
    got = host(Y[:, :cols])
    A = np.abs(xv) @ np.abs(wv).T
    off = np.abs(got - want) / bounds(A, v, y0, want, ty, mode, K)
    assert off.max() <= 1, (off.max(), np.unravel_index(off.argmax(), off.shape))
    assert bool(torch.isnan(Y[:, cols:]).all())
    return got


MODES = [("f32", 0), ("bf16", 0), ("f32", 1), ("bf16", 1), ("f32", 2), ("bf16", 2)]


@pytest.mark.parametrize("ty,mode", MODES)
@pytest.mark.parametrize("T,N,K", [(1, 2, 1), (1, 256, 256), (5, 130, 100), (16, 2560, 1024), (17, 1000, 424), (33, 34, 2816),
                                   (128, 640, 768), (129, 256, 9728), (200, 1538, 1000), (300, 130, 33), (640, 512, 256)])
def test_gemm(s2, T, N, K, ty, mode):
    check_product(s2, np.random.RandomState(T * 31 + N + K), T, N, K, ty, mode)


@pytest.mark.parametrize("x_kind", ["f32", "bf16"])
@pytest.mark.parametrize("ty,mode", [("f32", 0), ("bf16", 1), ("f32", 2)])
@pytest.mark.parametrize("T,N,K", [(1, 2, 1), (1, 6144, 2560), (2, 130, 100), (3, 512, 4096), (5, 1000, 424), (8, 2560, 9728),
                                   (8, 34, 33)])
def test_gemv(s2, T, N, K, ty, mode, x_kind):
    check_product(s2, np.random.RandomState(T * 31 + N + K), T, N, K, ty, mode, x_kind)


@pytest.mark.parametrize("x_kind", [None, "f32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(2, 0), (3, 1), (8, 8)])
def test_product_pitches(s2, pad, shift, x_kind):
    for mode in (0, 1, 2):
        check_product(s2, np.random.RandomState(pad), 7, 386, 424, "f32", mode, x_kind, pad, shift)
        check_product(s2, np.random.RandomState(pad), 7, 386, 424, "bf16", mode, x_kind, pad, shift)


@pytest.mark.parametrize("x_kind", [None, "f32", "bf16"])
def test_product_of_unlike_sizes(s2, x_kind):
    """Groups, rows and values whose sizes lie far apart: each output is held to its own sum."""
    rs = np.random.RandomState(9)
    T, N, K = 6, 200, 640
    x = U.rows(rs, T, K) * np.repeat(2.0 ** rs.randint(-20, 20, (T, K // 32)), 32, 1)
    x *= np.where(rs.uniform(size=(T, K)) < 0.3, 2.0 ** -12, 1)
    w = rs.standard_normal((N, K)) * np.repeat(2.0 ** rs.randint(-20, 20, (N, K // 32)), 32, 1)
    codes, sc = U.pack4(w)
    check_product(s2, rs, T, N, K, "f32", 0, x_kind, x=x, w=(U.unpack4(codes, sc, N, K), dev(codes), dev(sc)))


def test_scale_bytes_of_rows_that_do_not_exist(s2):
    """Bytes behind the last row may be anything, NaN scales among them."""
    rs = np.random.RandomState(10)
    T, N, K = 5, 130, 100
    wv, codes, sc = weights(rs, N, K)
    x8, xs = U.pack8(U.rows(rs, T, K))
    xv = U.unpack8(x8, xs, T, K)
    live = np.zeros(xs.size, bool)
    live[U.tile_index(T, K)] = True
    xs[~live] = 255
    s = host(sc).copy()
    live = np.zeros(s.size, bool)
    live[U.tile_index(N, K)] = True
    s[~live] = 255
    x8[:, K:] = 127                                             # bytes behind the rows, too
    Y = torch.zeros(T, N, device="cuda")
    s2.s2op_w4_gemm(codes, dev(s), N, K, dev(x8), x8.shape[1], dev(xs), T, Y, False, N, 0)
    A = np.abs(xv) @ np.abs(wv).T
    assert (np.abs(host(Y) - xv @ wv.T) <= sum_bound(K) * A + 2.0 ** -24 * np.abs(xv @ wv.T)).all()


@pytest.mark.parametrize("x_kind", [None, "f32"])
def test_nan_stays_in_its_row(s2, x_kind):
    rs = np.random.RandomState(11)
    T, N, K = 4, 140, 256
    w = rs.standard_normal((N, K))
    w[70, 100] = np.nan
    codes, sc = U.pack4(w)
    x = rs.standard_normal((T, K))
    x[2, 200] = np.nan
    Y = torch.zeros(T, N, device="cuda")
    if x_kind is None:
        x8, xs = U.pack8(x)
        s2.s2op_w4_gemm(dev(codes), dev(sc), N, K, dev(x8), K, dev(xs), T, Y, False, N, 0)
    else:
        ws = guarded(s2.s2op_w4_gemv_workspace_bytes(K, T))
        s2.s2op_w4_gemv(dev(codes), dev(sc), N, K, dev(x, "f32"), False, K, T, Y, False, N, 0, ws)
    want = np.zeros((T, N), bool)
    want[2], want[:, 70] = True, True
    assert np.array_equal(np.isnan(host(Y)), want)


# ---------------------------------------------------------------- together, in graphs and on streams

class Layer:
    """A small gated MLP: x += r, norm, gate and up with SwiGLU, rounding, down onto the residual."""

    def __init__(self, s2, rs, T, K, F):
        self.s2, self.T, self.K, self.F = s2, T, K, F
        self.w1v, self.c1, self.s1 = weights(rs, 2 * F, K)
        self.w2v, self.c2, self.s2_ = weights(rs, K, F)
        self.gain = dev(rs.uniform(0.5, 1.5, K).astype(np.float32))
        self.y8 = torch.zeros(T, K, dtype=torch.uint8, device="cuda")
        self.ys = guarded(s2.s2op_mx_scale_bytes(T, K), 0)
        self.a = torch.zeros(T, F, device="cuda")
        self.a8 = torch.zeros(T, F, dtype=torch.uint8, device="cuda")
        self.as_ = guarded(s2.s2op_mx_scale_bytes(T, F), 0)
        self.h = torch.zeros(T, K, device="cuda")

    def run(self, x, r, stream=None):
        s2, T, K, F = self.s2, self.T, self.K, self.F
        s2.s2op_add_rmsnorm_mx8(x, False, K, r, True, K, T, K, self.gain, 1e-6, self.h, K, self.y8, K, self.ys, stream)
        s2.s2op_w4_gemm(self.c1, self.s1, 2 * F, K, self.y8, K, self.ys, T, self.a, False, F, 2, stream)
        s2.s2op_mx8_pack(self.a, False, F, T, F, self.a8, F, self.as_, stream)
        s2.s2op_w4_gemm(self.c2, self.s2_, K, F, self.a8, F, self.as_, T, self.h, False, K, 1, stream)
        return self.h

    def check(self, x, r):
        T, K, F = self.T, self.K, self.F
        h = host((x + r.float()))
        v, e = U.round8(norm64(h, host(self.gain), float(np.float32(1e-6))))
        n = v * 2.0 ** np.repeat(e, 32, 1)
        p, a = product64(n, self.w1v, None, 2)
        A = np.abs(n) @ np.abs(self.w1v).T
        assert (np.abs(host(self.a) - a) <= bounds(A, p, None, a, "f32", 2, K)).all()
        av, ae = U.round8(host(self.a))              # of the values that the product gave
        a = av * 2.0 ** np.repeat(ae, 32, 1)
        p, y = product64(a, self.w2v, h, 1)
        A = np.abs(a) @ np.abs(self.w2v).T
        assert (np.abs(host(self.h) - y) <= bounds(A, p, h, y, "f32", 1, F)).all()


@pytest.mark.parametrize("T", [1, 9, 130])
def test_layer(s2, T):
    rs = np.random.RandomState(T)
    m = Layer(s2, rs, T, 256, 768)
    x, r = dev(U.rows(rs, T, 256), "f32"), dev(U.rows(rs, T, 256), "bf16")
    m.run(x, r)
    torch.cuda.synchronize()
    m.check(x, r)


def test_layer_in_a_graph_and_on_a_stream(s2):
    rs = np.random.RandomState(3)
    m = Layer(s2, rs, 5, 256, 768)
    x, r = dev(U.rows(rs, 5, 256), "f32"), dev(U.rows(rs, 5, 256), "bf16")
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        m.run(x, r, st)
        st.synchronize()
        m.check(x, r)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            m.run(x, r, st)
    for seed in (1, 2):
        x.copy_(dev(U.rows(np.random.RandomState(seed), 5, 256), "f32"))
        m.h.zero_()
        g.replay()
        torch.cuda.synchronize()
        m.check(x, r)


def test_calls_repeat_bit_for_bit(s2):
    rs = np.random.RandomState(4)
    _, codes, sc = weights(rs, 2560, 2560)
    for T in (1, 24, 150):
        x8, xs = U.pack8(U.rows(rs, T, 2560))
        x8, xs = dev(x8), dev(xs)
        out = []
        for _ in range(3):
            Y = torch.zeros(T, 2560, device="cuda")
            s2.s2op_w4_gemm(codes, sc, 2560, 2560, x8, 2560, xs, T, Y, False, 2560, 0)
            out.append(Y)
        assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])


def test_graphs_share_a_gemv_workspace_one_after_the_other(s2):
    rs = np.random.RandomState(7)
    ws = guarded(s2.s2op_w4_gemv_workspace_bytes(1024, 8))
    st = torch.cuda.Stream()
    todo = []
    for T, N, K, kind in ((8, 512, 1024, "f32"), (1, 256, 256, "bf16")):
        wv, codes, sc = weights(rs, N, K)
        X = dev(U.rows(rs, T, K), kind)
        Y = torch.zeros(T, N, device="cuda")
        args = (codes, sc, N, K, X, kind == "bf16", K, T, Y, False, N, 0, ws, st)
        with torch.cuda.stream(st):
            s2.s2op_w4_gemv(*args)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                s2.s2op_w4_gemv(*args)
        todo.append((g, wv, X, Y, K))
    for g, wv, X, Y, K in todo * 2:
        Y.zero_()
        with torch.cuda.stream(st):
            g.replay()
    torch.cuda.synchronize()
    for g, wv, X, Y, K in todo:
        x = host(X)
        A = np.abs(x) @ np.abs(wv).T
        assert (np.abs(host(Y) - x @ wv.T) <= (sum_bound(K) + 2.0 ** -24) * A).all()


# ---------------------------------------------------------------- sizes

def on_gpu(codes, sc, N, K, x, rows):
    """The products of x (float64) with some rows of the weights, on the GPU in 64 bits; A of each."""
    rows = torch.as_tensor(rows, device="cuda")
    nib = torch.stack([codes[rows] & 15, codes[rows] >> 4], -1).view(len(rows), -1)[:, :K].long()
    g = torch.arange((K + 31) // 32, device="cuda")
    r = rows[:, None]
    at = ((r // 128) * ((K + 127) // 128) + g // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + g % 4
    s = torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), sc.view(-1)[at].int() - 127)
    w = torch.from_numpy(U.VALUE4).cuda()[nib] * s.repeat_interleave(32, 1)[:, :K]
    return x @ w.T, x.abs() @ w.abs().T


def random_weights(N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (N, U.up(K, 128) // 2), dtype=torch.uint8, device="cuda", generator=g)
    sc = torch.randint(118, 126, (U.up(N, 128) * U.up(K, 128) // 32,), dtype=torch.uint8, device="cuda", generator=g)
    return codes, sc


def many(s2, T, N, K, ty, mode, seed, rows=None):
    codes, sc = random_weights(N, K, seed)
    x = U.rows(np.random.RandomState(seed), T, K)
    x8, xs = U.pack8(x)
    xv = torch.from_numpy(U.unpack8(x8, xs, T, K)).cuda()
    cols = N // 2 if mode == 2 else N
    Y = torch.full((T, cols), 0.5, dtype=TYPES[ty], device="cuda")
    s2.s2op_w4_gemm(codes, sc, N, K, dev(x8), x8.shape[1], dev(xs), T, Y, ty == "bf16", cols, mode)
    rows = np.arange(N) if rows is None else np.asarray(rows)
    v, A = on_gpu(codes, sc, N, K, xv, rows)
    if mode == 2:
        want = torch.nn.functional.silu(v[:, 0::2]) * v[:, 1::2]
        got = Y.double()[:, torch.as_tensor(rows[0::2] // 2, device="cuda")]
    else:
        want = v + 0.5 if mode == 1 else v
        got = Y.double()[:, torch.as_tensor(rows, device="cuda")]
    tol = torch.from_numpy(bounds(A.cpu().numpy(), v.cpu().numpy(), 0.5, want.cpu().numpy(), ty, mode, K)).cuda()
    # bf16 outputs of many rows are summed in the tensor core over up to 16,384 k
    if ty == "bf16":
        tol = tol + 34 * 2.0 ** -23 / 32 * (K / 32) * (A if mode != 2 else A[:, 0::2] * A[:, 1::2])
    off = ((got - want).abs() / tol).max().item()
    assert off <= 1, off


# tiles of 128, 192 and 256 rows by CTAs that stay, ends of tiles and of K inside them, and tiles of 128 in parts of K
@pytest.mark.parametrize("ty,mode", [("f32", 0), ("bf16", 0), ("f32", 1), ("bf16", 2)])
@pytest.mark.parametrize("T,N,K", [(1000, 19456, 256), (1024, 19456, 384), (700, 6144, 640), (160, 19500, 300), (250, 20000, 130),
                                   (385, 10000, 64), (150, 2560, 2560), (130, 25000, 256), (120, 20000, 100), (3000, 700, 1000)])
def test_gemm_many(s2, T, N, K, ty, mode):
    many(s2, T, N, K, ty, mode, T + N)


@pytest.mark.parametrize("T", [1, 3, 17, 40, 70])
def test_gemm_more_tiles_than_sms(s2, T):
    rs = np.random.RandomState(T)
    for N in (19457, 40000):
        rows = np.unique(np.concatenate([[0, 1, 127, 128, N - 2, N - 1], rs.randint(0, N, 500)]))
        many(s2, T, N, 700, "f32", 0, N + T, rows)


def test_weights_beyond_32_bits(s2):
    """Codes of more than 4 GB, and scale tiles and outputs that lie as far: a few rows of them."""
    N, K = (1 << 21) + 3, 4160
    rs = np.random.RandomState(0)
    rows = np.unique(np.concatenate([[0, N - 1, N - 2], rs.randint(0, N, 300)]))
    many(s2, 2, N, K, "f32", 0, 3, rows)
    codes, sc = random_weights(N, K, 3)
    X = dev(U.rows(rs, 1, K), "f32")
    Y = torch.zeros(1, N, device="cuda")
    s2.s2op_w4_gemv(codes, sc, N, K, X, False, K, 1, Y, False, N, 0, guarded(s2.s2op_w4_gemv_workspace_bytes(K, 1)))
    v, A = on_gpu(codes, sc, N, K, X.double(), rows)
    assert bool(((Y[:, torch.as_tensor(rows, device="cuda")].double() - v).abs() <= sum_bound(K) * A).all())


def test_rows_beyond_32_bits(s2):
    """Rows whose pitch takes the last ones beyond 2^31 elements."""
    T, K, N, ld = 70000, 96, 40, 32768
    codes, sc = random_weights(N, K, 5)
    g = torch.Generator(device="cuda").manual_seed(5)
    X = torch.empty(T, ld, dtype=torch.bfloat16, device="cuda")
    X[:, :K] = torch.randn(T, K, device="cuda", generator=g).bfloat16()
    y8 = torch.zeros(T, ld, dtype=torch.uint8, device="cuda")
    ys = guarded(s2.s2op_mx_scale_bytes(T, K))
    s2.s2op_mx8_pack(X, True, ld, T, K, y8, ld, ys)
    H = torch.empty(T, ld, dtype=torch.bfloat16, device="cuda")
    z8, zs = torch.zeros(T, 96, dtype=torch.uint8, device="cuda"), guarded(s2.s2op_mx_scale_bytes(T, K))
    gain = torch.ones(K, device="cuda")
    s2.s2op_add_rmsnorm_mx8(X, True, ld, X, True, ld, T, K, gain, 1e-6, H, ld, z8, 96, zs)
    Y = torch.empty(T, ld, device="cuda")
    s2.s2op_w4_gemm(codes, sc, N, K, y8, ld, ys, T, Y, False, ld, 0)
    at = torch.tensor([0, 1, 65535, 65536, 69998, 69999], device="cuda")
    x = host(X[at, :K])
    v, e = U.round8(x)
    assert np.array_equal(U.VALUE8[host(y8[at, :K])], v)
    p, A = on_gpu(codes, sc, N, K, torch.from_numpy(v * 2.0 ** np.repeat(e, 32, 1)).cuda(), np.arange(N))
    assert bool(((Y[at, :N].double() - p).abs() <= sum_bound(K) * A).all())
    h = host(dev(2 * x, "bf16"))
    assert np.array_equal(host(H[at, :K]), h)
    v, e = U.round8(norm64(h, np.ones(K), float(np.float32(1e-6))))
    assert np.array_equal(U.VALUE8[host(z8[at])], v)


def test_nothing_to_do(s2):
    none = torch.zeros(0, 64, device="cuda")
    s2.s2op_mx8_pack(none, False, 64, 0, 64, none, 64, none)
    s2.s2op_w4_pack(none, False, 0, 64, 64, none, none)
    s2.s2op_w4_gemm(none, none, 0, 64, none, 64, none, 0, none, False, 0, 0)
    torch.cuda.synchronize()


def test_first_call_may_be_captured():
    """A process whose first calls are under capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    child = """
import sys
sys.path[:0] = ["tests", "."]
import numpy as np, torch
import test_mx_gpu as m
from serving_dual_ar_gb300 import binding as s2
rs = np.random.RandomState(3)
layer = m.Layer(s2, rs, 5, 256, 768)
x, r = m.dev(m.U.rows(rs, 5, 256), "f32"), m.dev(m.U.rows(rs, 5, 256), "bf16")
torch.cuda.synchronize()
st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=st):
    layer.run(x, r, st)
g.replay()
torch.cuda.synchronize()
layer.check(x, r)
print("CAPTURED_OK")
"""
    r = subprocess.run([sys.executable, "-c", child], cwd=root, capture_output=True, text=True, timeout=300)
    assert "CAPTURED_OK" in r.stdout, r.stdout[-500:] + r.stderr[-2000:]


def test_two_streams_at_once(s2):
    """Products that overlap on the GPU, of kernels that take all of an SM's tensor memory and of ones that do not."""
    rs = np.random.RandomState(8)
    jobs = []
    for T, N, K in ((600, 4096, 1024), (1, 2560, 2560), (100, 2560, 1024), (20, 20000, 512)):
        codes, sc = random_weights(N, K, T)
        x8, xs = U.pack8(U.rows(rs, T, K))
        args = (codes, sc, N, K, dev(x8), K, dev(xs), T)
        Y, want = torch.zeros(T, N, device="cuda"), torch.zeros(T, N, device="cuda")
        s2.s2op_w4_gemm(*args, want, False, N, 0)
        jobs.append((args, Y, want, N, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(40):
        for args, Y, want, N, st in jobs:
            s2.s2op_w4_gemm(*args, Y, False, N, 0, st)
    torch.cuda.synchronize()
    for args, Y, want, N, st in jobs:
        assert torch.equal(Y, want)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("K", [96, 99, 256])
def test_w4_pack_nan_in_any_place(s2, K, kind):
    """A NaN or an infinity makes its group NaN and no other, aligned rows or not."""
    rs = np.random.RandomState(K)
    w = rs.standard_normal((40, K))
    at = rs.randint(0, K, 40)
    w[np.arange(40), at] = rs.choice([np.nan, np.inf, -np.inf], 40)
    t = dev(w, kind)
    codes, sc = guarded(s2.s2op_w4_code_bytes(40, K)), guarded(s2.s2op_mx_scale_bytes(40, K))
    out = torch.zeros(40, K, device="cuda")
    s2.s2op_w4_pack(t, kind == "bf16", 40, K, K, codes, sc)
    s2.s2op_w4_unpack(codes, sc, 40, K, out, False, K)
    v, e, bad = U.round4(host(t))
    assert bad.sum() == 40
    assert same(host(out), np.where(np.repeat(bad, 32, 1)[:, :K], np.nan, v * 2.0 ** np.repeat(e, 32, 1)[:, :K]))


@pytest.mark.parametrize("tx,tr", [("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("T,K", [(4000, 2560), (3000, 256), (1000, 9728)])
def test_add_rmsnorm_of_many_rows(s2, T, K, tx, tr):
    """Codes and scales of millions of values, next to ties among them, are those of 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, K, device="cuda", generator=g).to(TYPES[tx])
    r = (0.3 * torch.randn(T, K, device="cuda", generator=g)).to(TYPES[tr])
    gain = torch.rand(K, device="cuda", generator=g) + 0.5
    h, y8 = torch.empty_like(x), torch.zeros(T, K, dtype=torch.uint8, device="cuda")
    ys = guarded(s2.s2op_mx_scale_bytes(T, K))
    s2.s2op_add_rmsnorm_mx8(x, tx == "bf16", K, r, tr == "bf16", K, T, K, gain, 2.0 ** -20, h, K, y8, K, ys)
    want = (x.float() + r.float()).to(TYPES[tx])
    assert torch.equal(h, want)
    v = want.double()
    v = v / torch.sqrt(v.square().mean(-1, keepdim=True) + 2.0 ** -20) * gain.double()
    power = torch.tensor([448 * 2.0 ** e for e in range(U.EMIN, U.EMAX + 1)], dtype=torch.float64, device="cuda")
    e = torch.searchsorted(power, v.abs().view(T, -1, 32).amax(-1)) + U.EMIN
    grid = torch.from_numpy(U.E4M3).cuda()
    z = v / (power / 448)[(e - U.EMIN).repeat_interleave(32, 1)]
    hi = torch.searchsorted(grid, z.abs()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    down, up = z.abs() - grid[lo], grid[hi] - z.abs()
    code = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    assert torch.equal((y8 & 127).long(), code)
    assert bool(((y8 >= 128) == torch.signbit(z)).all())
    assert np.array_equal(host(ys), U.tiles((e + 127).byte().cpu().numpy(), K, 0xAB))


def test_add_rmsnorm_onto_the_residual(s2):
    rs = np.random.RandomState(12)
    for K in (768, 99, 20000):
        x, r = dev(U.rows(rs, 5, K), "f32"), dev(U.rows(rs, 5, K), "f32")
        gain = torch.ones(K, device="cuda")
        y8, ys = torch.zeros(2, 5, U.up(K, 16), dtype=torch.uint8, device="cuda"), guarded(2 * s2.s2op_mx_scale_bytes(5, K))
        h = torch.empty_like(x)
        s2.s2op_add_rmsnorm_mx8(x, False, K, r, False, K, 5, K, gain, 1e-6, h, K, y8[0], U.up(K, 16), ys)
        s2.s2op_add_rmsnorm_mx8(x, False, K, r, False, K, 5, K, gain, 1e-6, r, K, y8[1], U.up(K, 16),
                                ys[s2.s2op_mx_scale_bytes(5, K):])
        assert torch.equal(h, r) and torch.equal(y8[0], y8[1])


@pytest.mark.parametrize("T", [20, 40])
def test_between_bf16_products(s2, T):
    """Calls that follow one another without a pause, 4-bit products that start under bf16 ones and hold tensor memory on
    the same SMs among them, give what each gives alone."""
    K, N, M = 512, 20000, 512
    rs = np.random.RandomState(T)
    a = dev(rs.standard_normal((M, K)) * K ** -0.5, "bf16")
    b = dev(rs.standard_normal((T, K)), "bf16")
    wv, codes, sc = weights(rs, N, M)
    gain = torch.ones(M, device="cuda")
    h = torch.zeros(T, M, device="cuda")
    y8, ys = guarded(T * M).view(T, M), guarded(s2.s2op_mx_scale_bytes(T, M))
    Y, Z = torch.zeros(T, N, device="cuda"), torch.zeros(2, N, device="cuda")
    ws = guarded(s2.s2op_w4_gemv_workspace_bytes(M, 2))

    def run(after=lambda: None):
        for _ in range(3):
            s2.s2op_tc_gemm(a, M, K, b, T, K, h, M, split_k=1)
            after()
        s2.s2op_w4_gemv(codes, sc, N, M, h, False, M, 2, Z, False, N, 0, ws)
        after()
        s2.s2op_tc_gemm(a, M, K, b, T, K, h, M, epi=1, split_k=1)
        after()
        s2.s2op_add_rmsnorm_mx8(h, False, M, None, False, 0, T, M, gain, 1e-6, None, 0, y8, M, ys)
        after()
        s2.s2op_w4_gemm(codes, sc, N, M, y8, M, ys, T, Y, False, N, 0)
        after()
        return h.clone(), y8.clone(), Y.clone(), Z.clone()

    alone = run(torch.cuda.synchronize)
    v = host(alone[0])[:2] / 2
    want = v @ wv.T
    assert (np.abs(host(alone[3]) - want) <= bounds(np.abs(v) @ np.abs(wv).T, want, 0, want, "f32", 0, M)).all()
    for _ in range(20):
        for got, want in zip(run(), alone):
            assert torch.equal(got, want)


# ---------------------------------------------------------------- weights written just ahead

@pytest.mark.parametrize("kind,T,N,K", [("f32", 1, 640, 2560), ("bf16", 2, 300, 20000), ("f32", 5, 640, 2560), ("bf16", 8, 640, 2560),
                                        ("f32", 1, 20000, 512), (None, 1, 640, 2560), (None, 40, 20000, 512),
                                        (None, 100, 640, 2560), (None, 100, 12000, 512), (None, 300, 6000, 512)])
def test_weights_packed_just_ahead(s2, kind, T, N, K):
    """A product directly behind the packing of its weights, or with a call between that starts early, takes the new ones;
    a packing directly behind a product does not disturb it."""
    g = torch.Generator(device="cuda").manual_seed(N)
    W = [torch.randn(N, K, device="cuda", generator=g).bfloat16() for _ in range(2)]
    X = dev(U.rows(np.random.RandomState(T), T, K), kind or "f32")
    x8, xs = torch.zeros(T, U.up(K, 16), dtype=torch.uint8, device="cuda"), guarded(s2.s2op_mx_scale_bytes(T, K), 0)
    s2.s2op_mx8_pack(X, kind == "bf16", K, T, K, x8, U.up(K, 16), xs)
    z8, zs = torch.zeros_like(x8), guarded(s2.s2op_mx_scale_bytes(T, K), 0)
    codes, sc = guarded(s2.s2op_w4_code_bytes(N, K)), guarded(s2.s2op_mx_scale_bytes(N, K))
    ws = guarded(s2.s2op_w4_gemv_workspace_bytes(K, min(T, 8)))
    st = torch.cuda.Stream()

    def pack(i):
        s2.s2op_w4_pack(W[i], True, N, K, K, codes, sc, st)

    def product(Y):
        if kind is None:
            s2.s2op_w4_gemm(codes, sc, N, K, x8, U.up(K, 16), xs, T, Y, False, N, 0, st)
        else:
            s2.s2op_w4_gemv(codes, sc, N, K, X, kind == "bf16", K, T, Y, False, N, 0, ws, st)

    def steps(Y):
        for i in range(len(Y)):
            pack(i % 2)
            if i % 4 > 1:
                s2.s2op_mx8_pack(X, kind == "bf16", K, T, K, z8, U.up(K, 16), zs, st)
            product(Y[i])

    want = torch.zeros(2, T, N, device="cuda")
    Y = torch.zeros(16, T, N, device="cuda")
    torch.cuda.synchronize()
    for i in range(2):
        pack(i)
        torch.cuda.synchronize()
        product(want[i])
        torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        steps(Y)
    for run in (lambda: steps(Y), graph.replay):
        for _ in range(3):
            Y.zero_()
            torch.cuda.synchronize()
            run()
            torch.cuda.synchronize()
            assert torch.equal(Y, want.repeat(8, 1, 1))


# ---------------------------------------------------------------- sums that cancel

@pytest.mark.parametrize("T,N,K,ty", [(1, 256, 16384, "bf16"), (64, 256, 16384, "bf16"), (300, 12000, 2560, "bf16"),
                                      (1000, 2560, 16384, "bf16"), (600, 19456, 4096, "bf16"), (520, 6144, 17000, "bf16"),
                                      (1000, 2560, 16384, "f32")])
def test_sums_that_cancel(s2, T, N, K, ty):
    """Positive products added to what takes all but their last bits away: what is left shows how the sum was made.
    Each step of 32 k on the tensor core may cut 2^-23 of the sum so far, four times what it does on the average over a
    sum that grows evenly (2^-24 of half of it), up to 16,384 k where the output is bf16 and T above 64, 896 otherwise."""
    codes, sc = random_weights(N, K, K)
    codes &= 0x77                                               # no signs
    x8, xs = U.pack8(np.abs(U.rows(np.random.RandomState(T), T, K)))
    xv = torch.from_numpy(U.unpack8(x8, xs, T, K)).cuda()
    rows = np.unique(np.concatenate([[0, 127, N - 1], np.random.RandomState(N).randint(0, N, 200)]))
    v, A = on_gpu(codes, sc, N, K, xv, rows)
    at = torch.as_tensor(rows, device="cuda")
    Y = torch.zeros(T, N, dtype=TYPES[ty], device="cuda")
    Y[:, at] = (-v).to(TYPES[ty])
    y0 = Y[:, at].double()
    s2.s2op_w4_gemm(codes, sc, N, K, dev(x8), x8.shape[1], dev(xs), T, Y, ty == "bf16", N, 1)
    want = y0 + v
    steps = min(K, 16384 if ty == "bf16" and T > 64 else 896) / 32
    d = (steps * 2.0 ** -23 + (K / 512 + 17) * 2.0 ** -24) * A
    d = d + 2.0 ** -24 * (want.abs() + d)                       # the addition
    d = d + (2.0 ** -8 if ty == "bf16" else 2.0 ** -24) * (want.abs() + d)
    assert ((Y[:, at].double() - want).abs() / d).max().item() <= 1


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 4, 8])
def test_infinities_of_plain_rows_count_as_nan(s2, T, kind):
    rs = np.random.RandomState(T)
    N, K = 140, 500
    wv, codes, sc = weights(rs, N, K)
    x = U.rows(rs, T, K)
    x[T // 2, 300] = np.inf if T % 4 else -np.inf
    X = dev(x, kind)
    Y = torch.zeros(T, N, device="cuda")
    s2.s2op_w4_gemv(codes, sc, N, K, X, kind == "bf16", K, T, Y, False, N, 0, guarded(s2.s2op_w4_gemv_workspace_bytes(K, T)))
    got = host(Y)
    assert np.isnan(got[T // 2]).all()
    x = np.delete(host(X), T // 2, 0)
    assert (np.abs(np.delete(got, T // 2, 0) - x @ wv.T) <= (sum_bound(K) + 2.0 ** -24) * (np.abs(x) @ np.abs(wv).T)).all()


# ---------------------------------------------------------------- plain rows value by value

def unit_weights(s2, K):
    """The unit matrix: output n of a product with it is value n of the row."""
    codes, sc = guarded(s2.s2op_w4_code_bytes(K, K), 0), guarded(s2.s2op_mx_scale_bytes(K, K), 127)
    n = torch.arange(K, device="cuda")
    codes.view(K, -1)[n, n // 2] = torch.where(n % 2 == 0, 0x02, 0x20).to(torch.uint8)      # 1.0
    return codes, sc


def check_values(s2, x, kind, least):
    T, K = x.shape
    X = dev(x.astype(np.float32), kind)
    codes, sc = unit_weights(s2, K)
    Y = torch.zeros(T, K, device="cuda")
    s2.s2op_w4_gemv(codes, sc, K, K, X, kind == "bf16", K, T, Y, False, K, 0, guarded(s2.s2op_w4_gemv_workspace_bytes(K, T), 0xFF))
    x, got = host(X), host(Y)
    top = np.zeros((T, U.up(K, 32)))
    top[:, :K] = np.abs(x)
    top = np.repeat(top.reshape(T, -1, 32).max(-1), 32, 1)[:, :K]
    near, left = (2.0 ** -13, 2.0 ** -37) if kind == "f32" else (2.0 ** -17, 2.0 ** -25)
    whole = (np.abs(x) >= near * top) & (top >= least)
    assert whole.any() or least > top.max()
    assert np.array_equal(got[whole], x[whole])
    assert (np.abs(got - x) <= np.maximum(left * top, 2.0 ** -136)).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 3, 5, 6, 8])
@pytest.mark.parametrize("K", [100, 1000])
def test_values_of_plain_rows(s2, K, T, kind):
    """Values within 2^13 (bf16: 2^17) of their group's largest are taken whole, smaller ones to 2^-37 (2^-25) of it."""
    rs = np.random.RandomState(K + T)
    group = np.repeat(2.0 ** rs.uniform(-90, 100, (T, U.up(K, 32) // 32)), 32, 1)[:, :K]
    x = group * 2.0 ** rs.uniform(-30, 0, (T, K)) * rs.choice([-1, 1], (T, K))
    x[:, ::7] = group[:, ::7] * 2.0 ** -rs.randint(8, 20, x[:, ::7].shape) * rs.uniform(1, 2, x[:, ::7].shape)
    x[:, 5::32] = group[:, 5::32]
    check_values(s2, x, kind, 2.0 ** -95)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T", [2, 7])
def test_values_of_tiny_and_huge_rows(s2, T, kind):
    """Groups next to fp32's ends, subnormals among them: no part has a scale below 2^-126, so 2^-136 may be missing."""
    rs = np.random.RandomState(T)
    K = 640
    group = np.repeat(2.0 ** np.linspace(-148, -94, T * 20).reshape(T, 20), 32, 1)
    x = group * 2.0 ** rs.uniform(-10, 0, (T, K)) * rs.choice([-1, 1], (T, K))
    check_values(s2, x, kind, np.inf)
    x = 2.0 ** rs.uniform(100, 127.99, (T, K)) * rs.choice([-1, 1], (T, K))
    x[0, :32] = 3.3e38
    check_values(s2, x, kind, 0.0)


# ---------------------------------------------------------------- sizes of a model's larger matrices

@pytest.mark.parametrize("ty,mode", MODES)
@pytest.mark.parametrize("T,N,K", [(65, 9730, 700), (100, 12000, 1300), (128, 19456, 300)])
def test_gemm_of_up_to_128_rows_and_many_weights(s2, T, N, K, ty, mode):
    """Tiles of 128 weights by 128 rows, a CTA each, K whole."""
    many(s2, T, N, K, ty, mode, T + K)


@pytest.mark.parametrize("x_kind", ["f32", "bf16"])
@pytest.mark.parametrize("ty,mode", [("f32", 0), ("bf16", 1), ("f32", 2)])
@pytest.mark.parametrize("T", [1, 2, 3, 5, 6, 8])
def test_gemv_of_more_tiles_than_sms(s2, T, ty, mode, x_kind):
    """Two CTAs share an SM; plain rows' parts made by them, or by a kernel ahead."""
    rs = np.random.RandomState(T)
    for N, K in ((19458, 700), (40000, 1500)):
        codes, sc = random_weights(N, K, N + T)
        X = dev(U.rows(rs, T, K), x_kind)
        cols = N // 2 if mode == 2 else N
        Y = torch.full((T, cols), 0.5, dtype=TYPES[ty], device="cuda")
        ws = guarded(s2.s2op_w4_gemv_workspace_bytes(K, T), 0xFF)
        s2.s2op_w4_gemv(codes, sc, N, K, X, x_kind == "bf16", K, T, Y, ty == "bf16", cols, mode, ws)
        v, A = on_gpu(codes, sc, N, K, X.double(), np.arange(N))
        want = torch.nn.functional.silu(v[:, 0::2]) * v[:, 1::2] if mode == 2 else v + 0.5 * mode
        tol = torch.from_numpy(bounds(A.cpu().numpy(), v.cpu().numpy(), 0.5, want.cpu().numpy(), ty, mode, K)).cuda()
        off = ((Y.double() - want).abs() / tol).max().item()
        assert off <= 1, (N, off)


@pytest.mark.parametrize("x_kind", ["f32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(0, 0), (2, 0), (3, 1), (8, 8)])
def test_pitches_of_one_and_two_plain_rows(s2, pad, shift, x_kind):
    for T in (1, 2):
        for K in (424, 413):
            check_product(s2, np.random.RandomState(pad), T, 386, K, "f32", 0, x_kind, pad, shift)
            check_product(s2, np.random.RandomState(pad), T, 386, K, "bf16", 2, x_kind, pad, shift)


@pytest.mark.parametrize("K", [64, 2560, 99, 20000])
def test_add_rmsnorm_of_a_large_eps(s2, K):
    """eps up to fp32's largest number: its sum with the mean square may lie beyond."""
    rs = np.random.RandomState(K)
    x = U.rows(rs, 4, K) * np.array([1.0, 1e9, 1e17, 1e19])[:, None]
    gain = rs.uniform(0.5, 1.5, K).astype(np.float32)
    for eps in (1e20, 1e36, 3.4028234e38):
        h, y8, sc = run_norm(s2, x, None, gain, eps, "f32", "f32")
        v, e = U.round8(norm64(h, gain.astype(np.float64), float(np.float32(eps))))
        assert same(U.VALUE8[y8], v), eps
        assert np.array_equal(sc, U.tiles((e + 127).astype(np.uint8), K, 0xAB))


@pytest.mark.parametrize("x_kind", [None, "f32", "bf16"])
@pytest.mark.parametrize("T", [1, 7, 300])
def test_product_of_opposite_sizes(s2, T, x_kind):
    """Weights and rows whose scales lie at opposite ends: products of ordinary size."""
    if x_kind and T > 8:
        pytest.skip("plain rows: up to 8")
    rs = np.random.RandomState(T)
    N, K = 200, 640
    e = np.repeat(rs.choice([-118, -100, -40, 0, 40, 100], K // 32), 32)
    w = rs.standard_normal((N, K)) * 2.0 ** np.where(e > 0, e, e + 10.0)
    x = rs.standard_normal((T, K)) * 2.0 ** -e
    codes, sc = U.pack4(w)
    check_product(s2, rs, T, N, K, "f32", 0, x_kind, x=x.astype(np.float32).astype(np.float64),
                  w=(U.unpack4(codes, sc, N, K), dev(codes), dev(sc)))
