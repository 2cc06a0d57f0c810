"""4-bit weights and 8-bit rows without a GPU: sizes, refusals before any launch, and the 64-bit restatement itself."""

import numpy as np
import pytest

import mx_util as U


@pytest.fixture(scope="module")
def lib():
    from serving_dual_ar_gb300 import buildlib
    buildlib.build()
    from serving_dual_ar_gb300 import binding
    return binding


def test_grids():
    assert len(U.E4M3) == 127 and U.E4M3[-1] == 448 and U.E4M3[1] == 2.0 ** -9
    assert U.E2M1.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]


@pytest.mark.parametrize("top", [448.0, 6.0])
def test_exponent_is_the_smallest_that_covers(top):
    for e in (-126, -20, 0, 7, 120):
        x = np.zeros((3, 32))
        x[:, 5] = top * 2.0 ** e * np.array([1.0, 1 - 2.0 ** -40, 1 + 2.0 ** -40])
        got = U.exponents(x, top)[:, 0]
        assert got.tolist() == [e, e, min(e + 1, 120)]
    assert U.exponents(np.zeros((1, 1)), top).tolist() == [[-126]]


def test_ties_go_to_the_even_code():
    z = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    assert U.E2M1[U.nearest(z, U.E2M1)].tolist() == [0, 1, 1, 2, 2, 4, 4]


@pytest.mark.parametrize("n,K", [(1, 1), (129, 127), (300, 1000)])
def test_round_trips(n, K):
    rs = np.random.RandomState(n)
    x = U.rows(rs, n, K)
    v, e = U.round8(x)
    assert np.array_equal(U.unpack8(*U.pack8(x), n, K), v * 2.0 ** np.repeat(e, 32, 1)[:, :K])
    v, e, _ = U.round4(x)
    assert np.array_equal(U.unpack4(*U.pack4(x), n, K), v * 2.0 ** np.repeat(e, 32, 1)[:, :K])


def test_sizes(lib):
    assert lib.s2op_w4_code_bytes(3, 129) == 3 * 128
    assert lib.s2op_mx_scale_bytes(129, 129) == 4 * 512
    assert lib.s2op_mx_scale_bytes(0, 1) == 0
    assert lib.s2op_mx_scale_bytes(-1, 1) == lib.s2op_w4_code_bytes(1, 0) == 0
    assert lib.s2op_mx_scale_bytes(1 << 24, 1 << 20) == (1 << 17) * (1 << 13) * 512      # beyond 32 bits
    assert lib.s2op_w4_gemv_workspace_bytes(2560, 8) > 0
    assert lib.s2op_w4_gemv_workspace_bytes(2560, 9) == lib.s2op_w4_gemv_workspace_bytes(0, 1) == 0


A = 1 << 20      # an aligned address that is never followed: every call below is refused


def refused(lib, name, good, bad):
    call = getattr(lib.LIB, name)
    for at, v in bad:
        args = list(good)
        args[at] = v
        assert call(*args) == lib.S2_EINVAL, (name, at, v)


def test_refusals_pack(lib):
    # W, bf16, N, K, ldw, codes, scale, stream
    good = [A, 0, 8, 64, 64, A, A, None]
    bad = [(0, None), (0, A + 2), (2, -1), (2, (1 << 24) + 1), (3, 0), (3, (1 << 20) + 1), (4, 63), (5, None),
           (5, A + 16), (6, None), (6, A + 8)]
    refused(lib, "s2op_w4_pack", good, bad)
    # codes, scale, N, K, W, bf16, ldw, stream
    refused(lib, "s2op_w4_unpack", [A, A, 8, 64, A, 1, 64, None],
            [(0, None), (0, A + 16), (1, A + 8), (1, None), (2, -1), (3, 0), (4, None), (4, A + 1), (6, 63)])
    assert lib.LIB.s2op_w4_pack(None, 0, 0, 64, 64, None, None, None) == lib.S2_OK
    assert lib.LIB.s2op_w4_unpack(None, None, 0, 64, None, 0, 64, None) == lib.S2_OK


def test_refusals_rows(lib):
    # X, bf16, ldx, T, K, y8, ld8, scale, stream
    refused(lib, "s2op_mx8_pack", [A, 1, 64, 4, 64, A, 64, A, None],
            [(0, None), (0, A + 1), (2, 63), (3, -1), (3, (1 << 24) + 1), (4, 0), (4, (1 << 20) + 1), (5, None),
             (5, A + 8), (6, 48), (6, 72), (7, None), (7, A + 4)])
    assert lib.LIB.s2op_mx8_pack(None, 0, 64, 0, 64, None, 64, None, None) == lib.S2_OK
    # X, bf16, ldx, R, bf16, ldr, T, K, gain, eps, H, ldh, y8, ld8, scale, stream
    good = [A, 0, 64, A, 0, 64, 4, 64, A, 1e-6, A, 64, A, 64, A, None]
    bad = [(0, None), (0, A + 2), (2, 63), (3, A + 2), (5, 63), (6, -1), (7, 0), (8, None), (8, A + 2), (9, -1.0),
           (9, float("nan")), (10, None), (10, A + 2), (11, 63), (11, 65), (12, None), (12, A + 8), (13, 72), (14, None),
           (14, A + 8)]
    refused(lib, "s2op_add_rmsnorm_mx8", good, bad)
    good[6] = 0
    assert lib.LIB.s2op_add_rmsnorm_mx8(*good) == lib.S2_OK


def test_refusals_products(lib):
    # codes, scale, N, K, X, bf16, ldx, B, Y, bf16, ldy, mode, workspace, stream
    good = [A, A, 8, 64, A, 0, 64, 2, A, 0, 8, 0, A, None]
    bad = [(0, None), (0, A + 16), (1, None), (1, A + 8), (2, -1), (3, 0), (4, None), (4, A + 2), (6, 63), (7, 0),
           (7, 9), (8, None), (8, A + 2), (10, 7), (11, -1), (11, 3), (12, None), (12, A + 8)]
    refused(lib, "s2op_w4_gemv", good, bad)
    # codes, scale, N, K, X8, ld8, x_scale, T, Y, bf16, ldy, mode, stream
    good = [A, A, 8, 64, A, 64, A, 2, A, 1, 8, 0, None]
    bad = [(0, None), (0, A + 16), (1, A + 8), (2, (1 << 24) + 1), (3, 0), (4, None), (4, A + 8), (5, 56), (5, 48),
           (6, None), (6, A + 8), (7, -1), (7, (1 << 24) + 1), (8, None), (8, A + 1), (10, 7), (11, 3)]
    refused(lib, "s2op_w4_gemm", good, bad)
    odd = [A, A, 7, 64, A, 64, A, 2, A, 1, 8, 2, None]          # SwiGLU of an odd number of rows
    assert lib.LIB.s2op_w4_gemm(*odd) == lib.S2_EINVAL
    for n, t in ((0, 2), (8, 0)):
        assert lib.LIB.s2op_w4_gemm(None, None, n, 64, None, 64, None, t, None, 0, 8, 0, None) == lib.S2_OK
    with pytest.raises(lib.S2Error):
        lib.s2op_w4_gemm(None, None, 8, 64, None, 64, None, 2, None, False, 8, 0)


def test_refusals_in_place(lib):
    good = [A, 0, 64, 2 * A, 0, 64, 4, 64, A, 1e-6, 2 * A, 64, A, 64, A, None]      # the residual's rows overwritten
    refused(lib, "s2op_add_rmsnorm_mx8", good, [(4, 1), (5, 68), (11, 68), (9, float("inf"))])


def test_a_failed_query_is_not_kept(tmp_path):
    """What a device is asked for once is kept only where it answered."""
    import os
    import shutil
    import subprocess
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    here = os.path.dirname(os.path.abspath(__file__))
    csrc = os.path.join(os.path.dirname(here), "serving_dual_ar_gb300", "csrc")
    exe = str(tmp_path / "kept_count_driver")
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", csrc, os.path.join(here, "kept_count_driver.cpp"),
                    "-o", exe], check=True)
    assert subprocess.run([exe], capture_output=True, text=True, timeout=60).stdout == "ok\n"
