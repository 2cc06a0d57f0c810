"""Attention over the 8-bit cache at sizes and values that take paths of their
own: more sequences than a CTA has threads, more CTAs than SMs, NaN among cached
and new keys."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_kv8_gpu import Setup, b  # noqa: E402, F401  (b: the fixture)


@pytest.mark.parametrize("B,H,Hkv,hd,m", [
    (300, 4, 2, 64, 1),      # 256 threads a CTA: two sequences for some
    (1024, 2, 1, 64, 1),     # as many as there may be
    (1024, 16, 8, 128, 4),   # with the largest buffers beside them
    (333, 5, 5, 64, 1),      # 160 threads
])
def test_decode_of_many_sequences(b, B, H, Hkv, hd, m):
    rng = np.random.default_rng(B + H)
    pos = rng.integers(0, 70, B)
    pos[::7] = -1
    pos[[3, B // 2, B - 1]] = [400, 333, 511]
    s = Setup(pos, [m] * B, H, Hkv, hd, seed=B)
    s.upload()
    o, ws = s.run(b, "decode", False)
    torch.cuda.synchronize()
    s.check(o, False)
    o2, _ = s.run(b, "decode", False, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(o, o2)


@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,H,Hkv,hd", [(41, 16, 8, 128), (90, 4, 4, 64)])
def test_prompts_of_more_ctas_than_sms(b, B, H, Hkv, hd, bf16):
    """An SM takes a CTA after another: tensor memory and barriers set up anew."""
    rng = np.random.default_rng(B)
    new = rng.integers(1, 40, B)
    new[::9] = 0
    s = Setup(rng.integers(0, 200, B), new, H, Hkv, hd, seed=B)
    s.upload()
    o, ws = s.run(b, "prefill", bf16)
    torch.cuda.synchronize()
    s.check(o, bf16, planes=1 if bf16 else 2)
    o2, _ = s.run(b, "prefill", bf16, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(o, o2)


@pytest.mark.parametrize("kind,bf16", [("decode", False), ("decode", True), ("prefill", False), ("prefill", True)])
def test_nan_key_is_seen_by_its_rows_alone(b, kind, bf16):
    """A NaN among cached keys is seen by every row of its sequence and kv head, one
    among new keys by its row and later ones."""
    s = Setup([50, 40, 30, 33], [4, 4, 4, 4], 4, 2, 64, seed=51)
    s.codes[s.table[0, 1], 0, 1, 5, 9] = 0x7f           # cached, kv head 1 of sequence 0
    s.qkv[6, s.H * s.hd + 3] = np.nan                   # new, kv head 0, row 2 of sequence 1
    s.codes[s.table[2, 2], 0, :, :, :] = 0x7f           # free rows behind position 30 .. 33, and none else
    s.codes[s.table[2, 1], 0, 0, 15, 0] = 0x7f          # position 31 (new): written over
    s.upload()
    o, _ = s.run(b, kind, bf16)
    torch.cuda.synchronize()
    _, want = s.check(o, bf16, planes=1 if bf16 and kind == "prefill" else 2)
    nan = np.isnan(want).all(-1)                        # [rows, heads]
    assert nan[:4, 2:].all() and not nan[:4, :2].any()
    assert nan[6:8, :2].all() and not nan[4:6].any() and not nan[6:8, 2:].any()
    assert not nan[8:].any()


@pytest.mark.parametrize("kind,bf16", [("decode", False), ("decode", True), ("prefill", False), ("prefill", True)])
@pytest.mark.parametrize("gain", [5, 20])
def test_large_gains(b, kind, bf16, gain):
    """Scores of tens and hundreds: few keys have all the weight, and what a rounding
    of the queries does is multiplied by the score."""
    s = Setup([150, 64, 900], [8, 8, 8] if kind == "decode" else [33, 1, 140], 3, 3, 128, seed=52)
    s.qg *= np.float32(gain)
    s.upload()
    o, _ = s.run(b, kind, bf16)
    torch.cuda.synchronize()
    s.check(o, bf16, planes=1 if bf16 and kind == "prefill" else 2)
