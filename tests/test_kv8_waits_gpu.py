"""Waits inside the 8-bit cache's attention kernels that run out
(S2_FAULT_KV8_POLLS: each gives up after so many polls; no GPU fault is made).
A row behind such a wait is NaN; no number made of memory that was not waited for
comes out, and the next process finds nothing changed.  The setting is read once
in a process: each case is a process of its own."""

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
import kv8_util as ref
from test_kv8_gpu import Setup
from serving_dual_ar_gb300 import binding as b

polls = int(sys.argv[1])
CASES = [("decode", [100, 37, -1], [2, 2, 2], 8, 2, 128, False),
         ("decode", [5000], [1], 8, 8, 64, True),
         ("prefill", [150, 0, -1], [300, 33, 4], 8, 2, 128, False),
         ("prefill", [150, 0, -1], [300, 33, 4], 8, 2, 128, True),
         ("prefill", [0, 700], [40, 500], 4, 2, 64, True),
         ("prefill", [2500], [3], 8, 2, 128, False)]          # cut into ranges of keys
for i, (kind, pos, new, H, Hkv, hd, bf16) in enumerate(CASES):
    s = Setup(pos, new, H, Hkv, hd, seed=60 + i)
    s.upload()
    o, _ = s.run(b, kind, bf16)
    torch.cuda.synchronize()
    got = o.float().cpu().numpy()
    assert (got[s.T:] == 7).all() and (got[:, H * hd:] == 7).all()
    got = got[:s.T].reshape(s.T, H, hd).astype(np.float64)
    live = np.repeat(np.asarray(pos) >= 0, new)
    assert (got[~live] == 0).all()
    nan = np.isnan(got).all(-1)
    assert (nan == np.isnan(got).any(-1)).all(), "a row is NaN as a whole"
    if polls == 0:
        assert nan[live].all(), (i, "numbers behind waits that ran out", np.argwhere(~nan & live[:, None])[:3])
    _, want, SV = s.want()
    tol = ref.tolerance(SV, want, bf16, 1 if bf16 and kind == "prefill" else 2)
    bad = ~nan[..., None] & ~(np.abs(got - want) <= tol)
    assert not bad.any(), (i, "neither NaN nor right", np.argwhere(bad)[:3])
    print(kind, i, "rows that are NaN:", nan[live].mean())
x = torch.arange(1000, device="cuda").sum().item()
assert x == 499500
print("POLLS_OK", polls)
"""


@pytest.mark.parametrize("polls", [0, 1, 2, 50])
def test_rows_behind_a_wait_that_ran_out_are_nan(polls):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CHILD, str(polls)], cwd=root, capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, S2_FAULT_KV8_POLLS=str(polls)))
    assert "POLLS_OK" in r.stdout, r.stdout[-500:] + r.stderr[-2000:]
