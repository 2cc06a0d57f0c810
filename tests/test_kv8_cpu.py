"""Refusals of the 8-bit KV cache calls (no GPU): every bad argument is an
error before any device call, and the binding's own checks."""

import numpy as np
import pytest

import kv8_util as ref


@pytest.fixture(scope="module")
def lib():
    from serving_dual_ar_gb300 import buildlib
    buildlib.build()
    from serving_dual_ar_gb300 import binding
    return binding


P = 4096     # a pointer that no refused call may follow


def decode_args(**kw):
    a = dict(qkv=P, qkv_ld=1536, B=1, m=1, H=8, Hkv=2, hd=128, qg=P, kg=P, eps=1e-6, cos=P, sin=P, n_pos=64, pos=P,
             kv=P, scale=P, n_pages=4, table=P, table_ld=4, o=P, bf16=0, o_ld=1024, ws=P, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return list(a.values())


def prefill_args(**kw):
    a = dict(qkv=P, qkv_ld=1536, T=3, B=1, row0=P, pos=P, H=8, Hkv=2, hd=128, qg=P, kg=P, eps=1e-6, cos=P, sin=P,
             n_pos=64, kv=P, scale=P, n_pages=4, table=P, table_ld=4, o=P, bf16=0, o_ld=1024, ws=P, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return list(a.values())


BOTH = [dict([(k, None)]) for k in ("qkv", "qg", "kg", "cos", "sin", "pos", "kv", "scale", "table", "o", "ws")] + [
    dict(B=0), dict(B=1025), dict(hd=96), dict(H=9), dict(H=0), dict(Hkv=0), dict(H=18, qkv_ld=10000, o_ld=10000),
    dict(n_pos=0), dict(n_pages=0), dict(table_ld=0), dict(qkv_ld=1535), dict(o_ld=1023), dict(kv=P + 8),
    dict(scale=P + 2), dict(o=P + 2), dict(o=P + 1, bf16=1), dict(ws=P + 4), dict(qkv=P + 1), dict(qg=P + 2), dict(kg=P + 1),
    dict(cos=P + 2), dict(sin=P + 1), dict(pos=P + 2), dict(table=P + 1)]


@pytest.mark.parametrize("kw", BOTH + [dict(m=0), dict(m=3), dict(m=-1), dict(H=16, m=2, qkv_ld=4000, o_ld=4000),
                                       dict(m=2 ** 30), dict(B=1024, table_ld=2 ** 20)], ids=str)
def test_decode_refuses(lib, kw):
    assert lib.LIB.s2op_attn_decode_kv8(*decode_args(**kw)) == lib.S2_EINVAL


@pytest.mark.parametrize("kw", BOTH + [dict(T=0), dict(T=-4), dict(T=2 ** 24 + 1), dict(row0=None), dict(row0=P + 2)],
                         ids=str)
def test_prefill_refuses(lib, kw):
    assert lib.LIB.s2op_attn_prefill_kv8(*prefill_args(**kw)) == lib.S2_EINVAL


@pytest.mark.parametrize("change", [
    {0: None}, {3: None}, {5: None}, {6: None}, {8: None}, {2: 0}, {7: 0}, {9: -1}, {10: 0}, {11: 96}, {0: P + 8},
    {5: P + 4}, {6: P + 2}, {3: P + 1}, {8: P + 2}, {9: 2 ** 30, 10: 8}, {9: 2 ** 30 - 1, 10: 1}], ids=str)
def test_pack_refuses(lib, change):
    # kv, bf16, n_src, src, fill, kv8, scale, n_dst, dst, n, Hkv, hd, stream
    a = [P, 0, 4, P, None, P, P, 4, P, 2, 2, 128, None]
    for i, v in change.items():
        a[i] = v
    L = lib.LIB
    assert L.s2op_kv8_pack_pages(*a) == lib.S2_EINVAL
    # kv8, scale, n_src, src, kv, bf16, n_dst, dst, n, Hkv, hd, stream
    u = [a[5], a[6], a[7], a[8], a[0], a[1], a[2], a[3], a[9], a[10], a[11], a[12]]
    assert L.s2op_kv8_unpack_pages(*u) == lib.S2_EINVAL


def test_nothing_to_do_is_ok(lib):
    L = lib.LIB
    assert L.s2op_kv8_pack_pages(P, 0, 4, P, None, P, P, 4, P, 0, 2, 128, None) == lib.S2_OK
    assert L.s2op_kv_copy_pages(P, 16, None, 0, 4, 1, None, None, 0, None) == lib.S2_OK
    assert L.s2op_kv_remap_pages(P, 4, 4, 4, None, None, 0, None) == lib.S2_OK


@pytest.mark.parametrize("src,dst", [
    ([0, 1], [2, 2]),        # a destination twice
    ([0, 2], [2, 3]),        # a chain
    ([1], [1]),              # a page onto itself
    ([0, 1], [1, 0]),        # a swap
    ([4], [0]), ([-1], [0]), ([0], [4]), ([0], [-1]),
    ([0, 0, 0, 0, 0], [1, 2, 3, 1, 2])])
def test_copy_refuses_pairs(lib, src, dst):
    with pytest.raises(lib.S2Error) as e:
        lib.s2op_kv_copy_pages(P, 16, None, 0, 4, 1, src, dst, len(src))
    assert e.value.status == lib.S2_EINVAL


@pytest.mark.parametrize("kw", [dict(kv=None), dict(kv=P + 8), dict(page_bytes=0), dict(page_bytes=24),
                                dict(scale=P, scale_bytes=0), dict(scale=P, scale_bytes=6),
                                dict(scale=P + 2, scale_bytes=8), dict(n_pages=0), dict(layers=0),
                                dict(layers=65536), dict(n=-1), dict(src=None), dict(dst=None)], ids=str)
def test_copy_refuses(lib, kw):
    import ctypes
    arr = (ctypes.c_int32 * 1)(0), (ctypes.c_int32 * 1)(1)
    a = dict(kv=P, page_bytes=16, scale=None, scale_bytes=0, n_pages=4, layers=1, src=ctypes.addressof(arr[0]),
             dst=ctypes.addressof(arr[1]), n=1, stream=None)
    a.update(kw)
    assert lib.LIB.s2op_kv_copy_pages(*a.values()) == lib.S2_EINVAL


@pytest.mark.parametrize("src,dst", [([1, 1], [2, 3]), ([1, 2], [2, 3]), ([1], [1]), ([-1], [0]), ([0], [-1])])
def test_remap_refuses_pairs(lib, src, dst):
    with pytest.raises(lib.S2Error) as e:
        lib.s2op_kv_remap_pages(P, 2, 2, 2, src, dst, len(src))
    assert e.value.status == lib.S2_EINVAL


@pytest.mark.parametrize("args", [(None, 2, 2, 2), (P, -1, 2, 2), (P, 2, -1, 2), (P, 2, 4, 3), (P + 2, 2, 2, 2)])
def test_remap_refuses(lib, args):
    with pytest.raises(lib.S2Error):
        lib.s2op_kv_remap_pages(*args, [0], [1], 1)


def test_binding_wants_enough_host_pairs(lib):
    with pytest.raises(ValueError):
        lib.s2op_kv_copy_pages(P, 16, None, 0, 4, 1, [0], [1], 2)
    with pytest.raises(ValueError):
        lib.s2op_kv_remap_pages(P, 1, 1, 1, [0], [], 1)


def test_workspace_sizes(lib):
    d, p = lib.s2op_attn_decode_kv8_workspace_bytes, lib.s2op_attn_prefill_kv8_workspace_bytes
    assert 0 < d(1, 1, 32, 8, 128) <= d(128, 1, 32, 8, 128)
    assert p(1, 1, 32, 8, 128) > 0 and p(8000, 16, 32, 8, 128) > 0
    assert p(1, 1, 32, 8, 128) == p(8000, 16, 32, 8, 128) == p(8000, 1, 7, 7, 128)   # fewer rows never need more
    assert d(1, 1, 32, 8, 128) == d(128, 1, 32, 8, 128) < d(1, 2, 32, 8, 128)
    assert d(1, 3, 32, 8, 128) == 0 and p(0, 1, 32, 8, 128) == 0      # refused sizes


# the restatement itself, against torch's own conversion

def test_restated_e4m3_is_torchs():
    torch = pytest.importorskip("torch")
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(v, ref.VALUE)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(-448, 448, 20000), rng.standard_normal(20000) * 0.02,
                        ref.VALUE[:126] / 2 + ref.VALUE[1:127] / 2, -ref.VALUE[:127]]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert ref.same_codes(ref.encode(x), want).all()


def test_restated_exponent():
    x = np.zeros((6, 1, 1))
    x[:, 0, 0] = [0, 448, 448.5, 3.5, 3.5000005, np.inf]
    np.testing.assert_array_equal(ref.exponent(x), [-32, 0, 1, -7, -6, 32])


@pytest.mark.parametrize("bad", [np.array([2 ** 32 + 1]), np.array([2 ** 31]), np.array([-2 ** 32]), [2 ** 33],
                                 np.array([2 ** 32 + 1], np.uint64)], ids=str)
def test_page_indices_beyond_32_bits_are_outside_the_pool(lib, bad):
    """Not pages of the pool whose number is what 32 bits of them give."""
    for src, dst in ((bad, [2]), ([2], bad)):
        with pytest.raises(lib.S2Error) as e:
            lib.s2op_kv_copy_pages(P, 16, None, 0, 4, 1, src, dst, 1)
        assert e.value.status == lib.S2_EINVAL
        with pytest.raises(lib.S2Error) as e:
            lib.s2op_kv_remap_pages(P, 0, 2, 2, src, dst, 1)
        assert e.value.status == lib.S2_EINVAL


@pytest.mark.parametrize("bad", [[1.5], np.array([1.0]), [True], ["1"]], ids=str)
def test_page_indices_are_integers(lib, bad):
    with pytest.raises(ValueError):
        lib.s2op_kv_copy_pages(P, 16, None, 0, 4, 1, bad, [2], 1)
    with pytest.raises(ValueError):
        lib.s2op_kv_remap_pages(P, 0, 2, 2, [2], bad, 1)


def test_page_indices_of_any_integer_type(lib):
    for t in (np.int64, np.uint64, np.int16, np.int32):
        lib.s2op_kv_remap_pages(P, 0, 2, 2, np.array([1], t), np.array([2], t), 1)     # no rows: nothing to do
    lib.s2op_kv_remap_pages(P, 0, 2, 2, [], [], 0)
