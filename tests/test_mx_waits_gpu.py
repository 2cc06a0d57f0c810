"""Waits inside the products with 4-bit weights that run out (S2_FAULT_W4_POLLS:
each gives up after so many polls; no GPU fault is made).  An output behind such
a wait is NaN; no number made of memory that was not waited for comes out, and
the next process finds nothing changed.  The setting is read once in a process:
each case is a process of its own."""

import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

CHILD = """
import sys
import numpy as np, torch
sys.path[:0] = ["tests", "."]
import mx_util as U
from test_mx_gpu import weights, dev, host, guarded, sum_bound
from serving_dual_ar_gb300 import binding as b

polls = int(sys.argv[1])
# one part and several of K, tiles of every kind, plain rows in the CTAs and ahead
CASES = [(None, 1, 256, 2560), (None, 5, 300, 100), (None, 30, 20000, 512), (None, 50, 640, 2560), (None, 128, 640, 2560),
         (None, 600, 5000, 640), (None, 1000, 19456, 256), ("f32", 1, 640, 2560), ("bf16", 2, 200, 300), ("f32", 8, 640, 2560)]
for i, (kind, T, N, K) in enumerate(CASES):
    for bf16 in (False, True):
        rs = np.random.RandomState(i)
        wv, codes, sc = weights(rs, N, K)
        x = U.rows(rs, T, K)
        Y = torch.full((T + 1, N), 7.0, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
        if kind is None:
            x8, xs = U.pack8(x)
            x = U.unpack8(x8, xs, T, K)
            b.s2op_w4_gemm(codes, sc, N, K, dev(x8), x8.shape[1], dev(xs), T, Y, bf16, N, 0)
        else:
            X = dev(x, kind)
            x = host(X)
            b.s2op_w4_gemv(codes, sc, N, K, X, kind == "bf16", K, T, Y, bf16, N, 0,
                           guarded(b.s2op_w4_gemv_workspace_bytes(K, T)))
        torch.cuda.synchronize()
        got = host(Y)
        assert (got[T] == 7).all()
        got = got[:T]
        nan = np.isnan(got)
        if polls == 0:
            assert nan.all(), (i, "numbers behind waits that ran out", np.argwhere(~nan)[:3])
        want = x @ wv.T
        A = np.abs(x) @ np.abs(wv).T
        tol = sum_bound(K) * A + (2.0 ** -8 if bf16 else 2.0 ** -24) * (np.abs(want) + sum_bound(K) * A)
        bad = ~nan & ~(np.abs(got - want) <= tol)
        assert not bad.any(), (i, bf16, "neither NaN nor right", np.argwhere(bad)[:3])
        print(i, bf16, "outputs that are NaN:", nan.mean())
x = torch.arange(1000, device="cuda").sum().item()
assert x == 499500
print("POLLS_OK", polls)
"""


@pytest.mark.parametrize("polls", [0, 1, 3, 100])
def test_outputs_behind_a_wait_that_ran_out_are_nan(polls):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CHILD, str(polls)], cwd=root, capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, S2_FAULT_W4_POLLS=str(polls)))
    assert "POLLS_OK" in r.stdout, r.stdout[-500:] + r.stderr[-2000:]


LONG = """
import sys
import numpy as np, torch
sys.path[:0] = ["tests", "."]
import mx_util as U
from test_mx_gpu import weights, dev, guarded
from serving_dual_ar_gb300 import binding as b

# a bf16 product of 100 tiles and about 0.3 ms, beside which the calls after it start on the SMs that are left
M, D = 12800, 65536
a, x = torch.zeros(M, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(20, D, dtype=torch.bfloat16, device="cuda")
h = torch.zeros(20, M, device="cuda")
for kind, T, N, K in ((None, 16, 640, 2560), (None, 100, 256, 300), (None, 700, 256, 300), ("f32", 1, 640, 2560),
                      ("bf16", 6, 640, 2560)):
    rs = np.random.RandomState(T)
    _, codes, sc = weights(rs, N, K)
    rows = U.rows(rs, T, K)
    x8, xs = (dev(v) for v in U.pack8(rows))
    X = dev(rows, kind or "f32")
    ws = guarded(b.s2op_w4_gemv_workspace_bytes(K, min(T, 8)))
    Y, Z = torch.zeros(T, N, device="cuda"), torch.zeros(T, N, device="cuda")

    def call(out):
        if kind is None:
            b.s2op_w4_gemm(codes, sc, N, K, x8, x8.shape[1], xs, T, out, False, N, 0)
        else:
            b.s2op_w4_gemv(codes, sc, N, K, X, kind == "bf16", K, T, out, False, N, 0, ws)

    call(Y)
    torch.cuda.synchronize()
    assert not torch.isnan(Y).any(), (kind, T, "too few polls for the product itself")
    b.s2op_tc_gemm(a, M, D, x, 20, D, h, M, split_k=1)
    call(Z)
    torch.cuda.synchronize()
    assert torch.equal(Y, Z), (kind, T)
print("LONG_OK")
"""


def test_waits_do_not_count_the_kernel_ahead():
    """A wait gives up after so much of its own kernel's time: with polls for a tenth of a millisecond or so, products
    behind a kernel that takes longer and lets them start under it come out whole."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", LONG], cwd=root, capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, S2_FAULT_W4_POLLS="1000"))
    assert "LONG_OK" in r.stdout, r.stdout[-500:] + r.stderr[-2000:]


# plain rows whose parts wait for a stage to come free, and tiles of several sums
LONGER = """CASES = [("f32", 1, 19600, 900), ("bf16", 2, 19600, 900), ("f32", 2, 130, 20480), ("bf16", 1, 140, 16500),
         (None, 3, 130, 9000), (None, 200, 20000, 1000), (None, 300, 2000, 2560)]
"""


@pytest.mark.parametrize("polls", [5, 50, 200, 800])
def test_every_lane_of_a_warp_takes_the_same_way_out(polls):
    """A wait that runs out somewhere in the middle of a product: its warps go on whole, so the product ends."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    child = CHILD[:CHILD.index("CASES")] + LONGER + CHILD[CHILD.index("for i, (kind"):]
    r = subprocess.run([sys.executable, "-c", child, str(polls)], cwd=root, capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, S2_FAULT_W4_POLLS=str(polls)))
    assert "POLLS_OK" in r.stdout, r.stdout[-500:] + r.stderr[-2000:]
