"""The 8-bit KV cache: attention for single tokens and prompts, packing and
copying of pages, each through the C ABI against a 64-bit restatement."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import kv8_util as ref  # noqa: E402

EPS = 1e-6


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from serving_dual_ar_gb300 import buildlib
    buildlib.build()
    from serving_dual_ar_gb300 import binding
    return binding


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Setup:
    """Sequences over scattered pages of a pool whose free rows and free pages
    hold NaN codes and wild scales: nothing of them may be looked at."""

    def __init__(self, pos, new, H, Hkv, hd, seed=0, pad=0, cols=None, spread=0.0):
        rng = np.random.default_rng(seed)
        pos, new = np.asarray(pos), np.asarray(new)
        self.pos, self.new, self.H, self.Hkv, self.hd, self.B = pos, new, H, Hkv, hd, len(pos)
        self.T = int(new.sum())
        self.row0 = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        need = [(max(int(p), 0) + int(n) + 15) // 16 for p, n in zip(pos, new)]
        self.cols = cols or max(need) + 1
        self.n_pages = sum(need) + 3
        perm = rng.permutation(self.n_pages)
        self.table = np.full((self.B, self.cols), perm[-1], np.int32)
        at = 0
        codes = np.full((self.n_pages, 2, Hkv, 16, hd), 0x7f, np.uint8)
        exps = rng.integers(-32, 33, (self.n_pages, 2, Hkv))
        for i, k in enumerate(need):
            own = perm[at:at + k]
            at += k
            self.table[i, :min(k, self.cols)] = own[:self.cols]
            x = rng.standard_normal((k, 2, Hkv, 16, hd)) * 2.0 ** rng.uniform(-spread, spread, (k, 2, Hkv, 1, 1))
            e = ref.exponent(x)
            c = ref.encode(x / 2.0 ** e[..., None, None])
            for j, p in enumerate(own):
                rows = min(max(int(pos[i]) - 16 * j, 0), 16)
                codes[p, :, :, :rows] = c[j, :, :, :rows]
                if rows:
                    exps[p] = e[j]
        self.codes, self.exps = codes, exps
        self.ld = (H + 2 * Hkv) * hd + pad
        self.old = H * hd + pad
        self.qkv = rng.standard_normal((self.T + 2, self.ld), dtype=np.float32)
        self.qg = rng.uniform(0.5, 1.5, hd).astype(np.float32)
        self.kg = rng.uniform(0.5, 1.5, hd).astype(np.float32)
        self.n_pos = self.cols * 16
        ang = np.arange(self.n_pos)[:, None] * 1e6 ** (-2.0 * np.arange(hd // 2) / hd)
        self.cos, self.sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)

    def upload(self):
        self.d = dict(codes=dev(self.codes), scale=dev((2.0 ** self.exps).astype(np.float32)), qkv=dev(self.qkv),
                      qg=dev(self.qg), kg=dev(self.kg), cos=dev(self.cos), sin=dev(self.sin),
                      pos=dev(self.pos.astype(np.int32)), row0=dev(self.row0), table=dev(self.table))
        return self.d

    def run(self, b, kind, bf16, stream=None, o=None, ws=None):
        d = self.d
        o = torch.full((self.T + 2, self.old), 7.0, device="cuda",
                       dtype=torch.bfloat16 if bf16 else torch.float32) if o is None else o
        tail = (self.H, self.Hkv, self.hd, d["qg"], d["kg"], EPS, d["cos"], d["sin"], self.n_pos)
        if kind == "decode":
            m = int(self.new[0])
            ws = torch.zeros(b.s2op_attn_decode_kv8_workspace_bytes(self.B, m, self.H, self.Hkv, self.hd),
                             dtype=torch.uint8, device="cuda") if ws is None else ws
            b.s2op_attn_decode_kv8(d["qkv"], self.ld, self.B, m, *tail, d["pos"], d["codes"], d["scale"], self.n_pages,
                                   d["table"], self.cols, o, bf16, self.old, ws, stream=stream)
        else:
            ws = torch.zeros(b.s2op_attn_prefill_kv8_workspace_bytes(self.T, self.B, self.H, self.Hkv, self.hd),
                             dtype=torch.uint8, device="cuda") if ws is None else ws
            b.s2op_attn_prefill_kv8(d["qkv"], self.ld, self.T, self.B, d["row0"], d["pos"], *tail, d["codes"],
                                    d["scale"], self.n_pages, d["table"], self.cols, o, bf16, self.old, ws,
                                    stream=stream)
        return o, ws

    def want(self):
        cache = ref.Cache(self.codes, self.exps)
        o = np.full((self.T, self.H, self.hd), 7.0)
        SV = ref.attention(cache, self.qkv[:self.T, :(self.H + 2 * self.Hkv) * self.hd].astype(np.float64), self.H,
                           self.Hkv, self.hd, self.row0, self.pos, self.table, self.qg, self.kg, EPS, self.cos,
                           self.sin, self.n_pos, o)
        return cache, o, SV

    def check(self, o, bf16, planes=2):
        cache, want, SV = self.want()
        got = o.float().cpu().numpy()
        assert (got[self.T:] == 7).all() and (got[:, self.H * self.hd:] == 7).all()   # nothing behind the rows
        got = got[:self.T, :self.H * self.hd].reshape(self.T, self.H, self.hd).astype(np.float64)
        np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
        tol = ref.tolerance(SV, want, bf16, planes)
        err = np.where(np.isnan(want), 0, np.abs(got - want))
        assert (err <= tol).all(), (float((err / tol).max()), np.argwhere(err > tol)[:5].tolist())
        codes, scale = self.d["codes"].cpu().numpy(), self.d["scale"].cpu().numpy()
        np.testing.assert_array_equal(scale, (2.0 ** cache.exps).astype(np.float32))
        assert ref.same_codes(codes, cache.codes).all()
        return cache, want


DECODE = [
    # positions, m, H, Hkv, hd
    ([0], 1, 32, 8, 128),                              # the first token of all
    ([41], 1, 32, 8, 128),
    ([15, 16, 17, 31, 0, 1], 1, 8, 2, 128),            # page borders
    ([-1, 5, -1, 200], 1, 8, 2, 128),                  # rows of a padded batch
    ([-1, -1], 1, 8, 2, 128),                          # nothing to do at all
    ([15, 14, 31, 100], 2, 8, 2, 128),                 # new rows on both sides of a border
    ([13, 15, 0, 77], 4, 4, 2, 64),
    ([9, 15, 40, 3], 8, 3, 3, 128),                    # one query head a kv head, eight rows
    ([63, 500], 1, 8, 1, 128),                         # eight query heads on one kv head
    ([33, 7, 129], 1, 21, 3, 64),                      # seven a kv head
    ([33, 7, 129], 2, 9, 3, 128),                      # three a kv head
    ([1090, 900, 1003], 1, 32, 8, 128),
    ([5000, 12, 0, 777], 2, 4, 2, 64),
    ([9000], 1, 4, 1, 128),                            # one long sequence, one kv head
]


@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
@pytest.mark.parametrize("pos,m,H,Hkv,hd", DECODE)
def test_decode_matches_the_definition(b, pos, m, H, Hkv, hd, bf16):
    s = Setup(pos, [m] * len(pos), H, Hkv, hd, seed=len(pos) + m, pad=3 if m == 2 else 0)
    s.upload()
    o, ws = s.run(b, "decode", bf16)
    torch.cuda.synchronize()
    s.check(o, bf16)
    # again on the same state: the same tokens in the same places
    o2, _ = s.run(b, "decode", bf16, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(o.nan_to_num(), o2.nan_to_num())
    s.check(o2, bf16)


def test_decode_batch_of_ragged_lengths(b):
    rng = np.random.default_rng(3)
    pos = rng.integers(0, 700, 96)
    pos[::17] = -1
    s = Setup(pos, [1] * 96, 8, 2, 128, seed=3, spread=6)
    s.upload()
    o, _ = s.run(b, "decode", False)
    torch.cuda.synchronize()
    s.check(o, False)


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_block_scales_far_apart(b, kind):
    """Blocks of one sequence whose scales differ by up to 2^40."""
    s = Setup([150, 60], [2, 2], 8, 2, 128, seed=5, spread=20)
    s.qkv[:, :(s.H + s.Hkv) * s.hd] *= np.float32(1e-4)     # keys and queries of any size: the norm takes it
    s.upload()
    o, _ = s.run(b, kind, False)
    torch.cuda.synchronize()
    s.check(o, False)


@pytest.mark.parametrize("hd", [64, 128])
def test_block_scales_far_apart_in_a_bf16_prompt(b, hd):
    s = Setup([150, 60, 0], [140, 2, 33], 8, 2, hd, seed=25, spread=20)
    s.qkv[150:, (s.H + s.Hkv) * s.hd:] *= np.float32(2.0 ** -18)
    s.upload()
    o, ws = s.run(b, "prefill", True)
    torch.cuda.synchronize()
    s.check(o, True, planes=1)
    o2, _ = s.run(b, "prefill", True, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(o, o2)


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_scales_a_bit_beside_a_power_of_two(b, kind):
    s = Setup([150, 61], [1, 1], 8, 2, 128, seed=17)
    d = s.upload()
    d["scale"].mul_(torch.tensor([1 - 2.0 ** -23, 1 + 2.0 ** -22], device="cuda").repeat(s.n_pages)[:s.n_pages, None, None])
    touched = {int(s.table[0, 9]), int(s.table[1, 3])}
    o, _ = s.run(b, kind, False)
    torch.cuda.synchronize()
    got = d["scale"].clone()
    exact = torch.from_numpy((2.0 ** s.exps).astype(np.float32)).cuda()
    rest = [p for p in range(s.n_pages) if p not in touched]
    assert ((got[rest] / exact[rest] - 1).abs() < 1e-6).all()      # left as they were
    d["scale"][rest] = exact[rest]
    s.check(o, False)


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_scale_grows_and_old_rows_move(b, kind):
    s = Setup([5, 12, 30], [2, 2, 2], 8, 2, 128, seed=6)
    s.qkv[:, (s.H + s.Hkv) * s.hd:] *= np.float32(300)
    s.kg[::5] *= 50
    s.upload()
    o, _ = s.run(b, kind, False)
    torch.cuda.synchronize()
    cache, _ = s.check(o, False)
    p = s.table[0, 0]
    assert (cache.exps[p, 1] > s.exps[p, 1]).all()


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_values_out_of_range_saturate(b, kind):
    s = Setup([20], [2], 8, 2, 128, seed=7)
    v0 = (s.H + s.Hkv) * s.hd
    s.qkv[0, v0] = np.inf
    s.qkv[0, v0 + 1] = -np.inf
    s.qkv[1, v0 + s.hd] = 1e20
    s.qkv[1, v0 + s.hd + 3] = 0.0
    s.upload()
    o, _ = s.run(b, kind, False)
    torch.cuda.synchronize()
    s.check(o, False)


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_nan_value_is_seen_by_its_row_and_later_ones_alone(b, kind):
    s = Setup([20, 14, 40], [4, 4, 4], 4, 2, 64, seed=8)
    v0 = (s.H + s.Hkv) * s.hd
    s.qkv[2, v0 + 5] = np.nan          # row 2 of sequence 0: rows 0 and 1 must not see it
    s.qkv[8, v0 + s.hd + 63] = np.nan  # row 0 of sequence 2
    s.upload()
    o, _ = s.run(b, kind, False)
    torch.cuda.synchronize()
    _, want = s.check(o, False)
    assert np.isnan(want).any() and not np.isnan(want[:2]).any()


def test_nan_in_the_cache_is_seen(b):
    s = Setup([50, 50], [1, 1], 4, 2, 64, seed=9)
    s.codes[s.table[0, 1], 1, 0, 3, 7] = 0xff
    s.upload()
    o, _ = s.run(b, "decode", False)
    torch.cuda.synchronize()
    _, want = s.check(o, False)
    assert np.isnan(want[0, :2, 7]).all() and not np.isnan(want[1]).any()


def test_few_rows_behind_a_long_context(b):
    """The keys are cut into ranges: a NaN, a missing page and a page of large
    values in different ones, rows that see all of them."""
    for bf16 in (False, True):
        s = Setup([3000, 1700, 90], [3, 20, 1], 4, 2, 64, seed=19, spread=3)
        s.codes[s.table[0, 11], 1, 0, 3, 7] = 0xff
        s.table[1, 60] = -1
        s.exps[s.table[1, 3]] += 20
        s.upload()
        o, ws = s.run(b, "prefill", bf16)
        torch.cuda.synchronize()
        _, want = s.check(o, bf16, planes=1 if bf16 else 2)
        assert np.isnan(want[:3, :2, 7]).all()
        o2, _ = s.run(b, "prefill", bf16, ws=ws)
        torch.cuda.synchronize()
        assert torch.equal(o.nan_to_num(), o2.nan_to_num())


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_bad_pages_are_not_followed(b, kind):
    s = Setup([40, 33, 10, 5], [2, 2, 2, 2], 8, 2, 128, seed=10)
    s.table[0, 1] = -1                  # a page in the middle
    s.table[1, 2] = s.n_pages           # the page of the new rows
    s.table[2, 0] = 2 ** 31 - 1         # the only page: rows without a key
    s.upload()
    o, _ = s.run(b, kind, False)
    torch.cuda.synchronize()
    _, want = s.check(o, False)
    assert (want[4:6] == 0).all()


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_positions_outside_the_table_are_left_out(b, kind):
    s = Setup([10, 30, 20, 20], [2, 2, 2, 2], 8, 2, 128, seed=11, cols=3)
    s.pos = np.array([10, 47, 2 ** 31 - 2, -5])
    s.upload()
    o, _ = s.run(b, kind, True)
    torch.cuda.synchronize()
    _, want = s.check(o, True, planes=1)
    assert (want[2:] == 0).all() and (want[:2] != 0).any()


PREFILL = [
    # positions, new rows, H, Hkv, hd
    ([0], [1], 32, 8, 128),
    ([0], [41], 32, 8, 128),
    ([0], [16], 8, 2, 128),
    ([0, 0, 0], [17, 1, 15], 8, 2, 128),
    ([5, 16, 31, 0], [40, 0, 70, 3], 8, 2, 128),       # a sequence without rows
    ([900, 640], [33, 150], 8, 2, 128),                # behind cached pages
    ([0, 130], [300, 77], 4, 2, 64),
    ([3, 0], [129, 64], 7, 7, 128),
    ([0, 20], [100, 260], 16, 2, 64),
    ([0, 50], [100, 31], 21, 3, 128),
    ([0, 17], [130, 259], 6, 1, 64),
    ([0], [513], 8, 2, 128),
    ([2000], [3], 8, 1, 128),                          # few rows behind a long context
    ([-1, 8], [20, 20], 8, 2, 128),
]


@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
@pytest.mark.parametrize("pos,new,H,Hkv,hd", PREFILL)
def test_prefill_matches_the_definition(b, pos, new, H, Hkv, hd, bf16):
    s = Setup(pos, new, H, Hkv, hd, seed=len(pos) + sum(new), pad=5 if H == 7 else 0)
    s.upload()
    o, ws = s.run(b, "prefill", bf16)
    torch.cuda.synchronize()
    s.check(o, bf16, planes=1 if bf16 else 2)
    o2, _ = s.run(b, "prefill", bf16, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(o, o2)


def test_prefill_of_many_sequences(b):
    rng = np.random.default_rng(12)
    new = rng.integers(0, 30, 70)
    s = Setup(rng.integers(0, 100, 70), new, 8, 2, 128, seed=12)
    s.upload()
    o, _ = s.run(b, "prefill", False)
    torch.cuda.synchronize()
    s.check(o, False)


def test_prompt_and_single_steps_write_the_same_bytes(b):
    """A sequence appended at once, and the same rows one or two at a time."""
    n = 45
    s = Setup([0], [n], 8, 2, 128, seed=13)
    s.kg[:] = 1.0
    d = s.upload()
    s.run(b, "prefill", False)
    torch.cuda.synchronize()
    at_once, scale = d["codes"].clone(), d["scale"].clone()
    d["codes"].fill_(0x7f)
    d["scale"].fill_(2.0 ** 20)
    at = 0
    while at < n:
        m = 2 if at % 3 == 0 and at + 2 <= n else 1
        ws = torch.zeros(b.s2op_attn_decode_kv8_workspace_bytes(1, m, 8, 2, 128), dtype=torch.uint8, device="cuda")
        o = torch.zeros((m, 1024), device="cuda")
        b.s2op_attn_decode_kv8(d["qkv"][at:], s.ld, 1, m, 8, 2, 128, d["qg"], d["kg"], EPS, d["cos"], d["sin"], s.n_pos,
                               torch.tensor([at], dtype=torch.int32, device="cuda"), d["codes"], d["scale"],
                               s.n_pages, d["table"], s.cols, o, False, 1024, ws)
        at += m
    torch.cuda.synchronize()
    for j in range((n + 15) // 16):
        p, rows = s.table[0, j], min(16, n - 16 * j)
        assert torch.equal(scale[p], d["scale"][p])
        x, y = at_once[p, :, :, :rows].cpu().numpy(), d["codes"][p, :, :, :rows].cpu().numpy()
        same = ref.same_codes(x, y)
        # a value may differ only where it became an e4m3 subnormal when a
        # block's scale grew later: it then was rounded twice
        assert (np.abs(ref.VALUE[x][~same]) <= 2.0 ** -6).all() and (~same).mean() < 1e-2


# --------------------------------------------------------------------- the calls together

def test_prompt_fork_and_decode(b):
    """A prompt, two forks of it (shared full pages, the last one copied), and
    decode steps of all three in one batch: as three sequences computed alone."""
    H, Hkv, hd, n = 8, 2, 128, 37
    s = Setup([0], [n], H, Hkv, hd, seed=14, cols=6)
    n_pages = 16
    rng = np.random.default_rng(14)
    codes, exps = np.full((n_pages, 2, Hkv, 16, hd), 0x7f, np.uint8), np.zeros((n_pages, 2, Hkv), np.int64)
    s.codes, s.exps, s.n_pages = codes, exps, n_pages
    table = np.full((3, 6), 15, np.int32)
    table[0, :4] = [4, 9, 2, 7]
    table[1, :4] = [4, 9, 11, 0]
    table[2, :4] = [4, 9, 13, 5]
    s.table = table[:1].copy()
    d = s.upload()
    s.run(b, "prefill", False)
    b.s2op_kv_copy_pages(d["codes"], 2 * Hkv * 16 * hd, d["scale"], 2 * Hkv * 4, n_pages, 1, [2, 2], [11, 13], 2)
    cache = ref.Cache(codes, exps)
    x = s.qkv[:n].reshape(n, H + 2 * Hkv, hd).astype(np.float64)
    cache.append(table[0], 0, ref.norm_rope(x[:, H:H + Hkv], s.kg, s.cos[:n], s.sin[:n], EPS), x[:, H + Hkv:])
    for page in (11, 13):
        cache.codes[page], cache.exps[page] = cache.codes[2], cache.exps[2]
    ws = torch.zeros(b.s2op_attn_decode_kv8_workspace_bytes(3, 1, H, Hkv, hd), dtype=torch.uint8, device="cuda")
    tab, o = dev(table), torch.zeros((3, H * hd), device="cuda")
    for step in range(14):
        qkv = rng.standard_normal((3, s.ld), dtype=np.float32)
        pos = np.full(3, n + step, np.int32)
        b.s2op_attn_decode_kv8(dev(qkv), s.ld, 3, 1, H, Hkv, hd, d["qg"], d["kg"], EPS, d["cos"], d["sin"], s.n_pos,
                               dev(pos), d["codes"], d["scale"], n_pages, tab, 6, o, False, H * hd, ws)
        want = np.zeros((3, H, hd))
        SV = ref.attention(cache, qkv.astype(np.float64), H, Hkv, hd, np.arange(4), pos, table, s.qg, s.kg, EPS,
                           s.cos, s.sin, s.n_pos, want)
        err = np.abs(o.cpu().numpy().reshape(3, H, hd) - want)
        assert (err <= ref.tolerance(SV, want, False)).all(), step
    # compaction: pages 9.. to free ones in front, tables rewritten; then one more step
    src, dst = [9, 11, 13, 7], [1, 3, 6, 8]
    b.s2op_kv_copy_pages(d["codes"], 2 * Hkv * 16 * hd, d["scale"], 2 * Hkv * 4, n_pages, 1, src, dst, 4)
    b.s2op_kv_remap_pages(tab, 3, 6, 6, src, dst, 4)
    moved = dict(zip(src, dst))
    np.testing.assert_array_equal(tab.cpu().numpy(), np.vectorize(lambda p: moved.get(p, p))(table))
    qkv = rng.standard_normal((3, s.ld), dtype=np.float32)
    pos = np.full(3, n + 14, np.int32)
    b.s2op_attn_decode_kv8(dev(qkv), s.ld, 3, 1, H, Hkv, hd, d["qg"], d["kg"], EPS, d["cos"], d["sin"], s.n_pos,
                           dev(pos), d["codes"], d["scale"], n_pages, tab, 6, o, False, H * hd, ws)
    want = np.zeros((3, H, hd))
    SV = ref.attention(cache, qkv.astype(np.float64), H, Hkv, hd, np.arange(4), pos, table, s.qg, s.kg, EPS, s.cos,
                       s.sin, s.n_pos, want)
    assert (np.abs(o.cpu().numpy().reshape(3, H, hd) - want) <= ref.tolerance(SV, want, False)).all()


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_captured_and_replayed(b, kind):
    """One call captured into a graph: replayed on new inputs and positions."""
    s = Setup([100, 37, 5], [2, 2, 2], 8, 2, 128, seed=15)
    d = s.upload()
    first = {k: v.clone() for k, v in d.items()}
    o, ws = s.run(b, kind, False)
    torch.cuda.synchronize()
    for k in d:
        d[k].copy_(first[k])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        s.run(b, kind, False, stream=torch.cuda.current_stream(), o=o, ws=ws)
    for seed in (1, 2):
        rng = np.random.default_rng(seed)
        s.qkv = rng.standard_normal(s.qkv.shape, dtype=np.float32)
        s.pos = np.array([100 - seed, 37 - 2 * seed, 5 - seed])
        for k in ("codes", "scale"):
            d[k].copy_(first[k])
        d["qkv"].copy_(dev(s.qkv))
        d["pos"].copy_(dev(s.pos.astype(np.int32)))
        o.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        s.check(o, False)


def test_two_streams_with_a_workspace_each(b):
    runs = []
    for seed in (1, 2):
        s = Setup([400 + seed, 30], [1, 1], 8, 2, 128, seed=seed)
        s.upload()
        runs.append((s, torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = []
    for s, st in runs:
        with torch.cuda.stream(st):
            for _ in range(20):
                r = s.run(b, "decode", False, stream=st, **(dict(o=r[0], ws=r[1]) if _ else {}))
            outs.append(r[0])
    torch.cuda.synchronize()
    for (s, _), o in zip(runs, outs):
        s.check(o, False)


def test_one_workspace_for_calls_of_all_sizes(b):
    """Prompts of other sizes and kv heads, single tokens and prompts in turn
    over one workspace: what a call leaves in it is no ticket to the next."""
    sizes = [b.s2op_attn_decode_kv8_workspace_bytes(4, m, H, Hkv, hd) for m, H, Hkv, hd in
             ((1, 32, 8, 128), (2, 9, 3, 128), (1, 20, 20, 64))]
    sizes += [b.s2op_attn_prefill_kv8_workspace_bytes(T, B, 8, 2, hd) for T, B in ((8000, 1), (3, 2)) for hd in (64, 128)]
    ws = torch.zeros(max(sizes), dtype=torch.uint8, device="cuda")
    calls = [
        ("prefill", [2500], [3], 32, 8, 128),
        ("prefill", [1500, 900], [150, 3], 22, 11, 64),     # 66 CTAs a range
        ("decode", [1090, 900, 1003], [1] * 3, 32, 8, 128),
        ("prefill", [1100] * 8, [2] * 8, 18, 9, 128),       # 72 CTAs a range
        ("decode", [2000, 77], [2] * 2, 9, 3, 128),
        ("decode", [2000, 1000], [1] * 2, 20, 20, 64),      # three groups of kv heads
        ("prefill", [2500], [3], 32, 8, 128),
        ("decode", [41], [1], 32, 8, 128),
    ]
    for i, (kind, pos, new, H, Hkv, hd) in enumerate(calls):
        s = Setup(pos, new, H, Hkv, hd, seed=40 + i)
        s.upload()
        o, _ = s.run(b, kind, False, ws=ws)
        torch.cuda.synchronize()
        s.check(o, False)


@pytest.mark.parametrize("hd,bf16", [(128, False), (128, True), (64, False)])
def test_prompt_whose_table_has_the_longest_row(b, hd, bf16):
    """A table and RoPE rows for 2^20 positions: the call takes the sizes that its
    documentation gives."""
    s = Setup([50, 0], [3, 20], 4, 2, hd, seed=23)
    d = s.upload()
    wide = torch.full((2, 65536), -1, dtype=torch.int32, device="cuda")
    wide[:, :s.cols] = d["table"]
    for k in ("cos", "sin"):
        x = torch.zeros((2 ** 20, hd // 2), device="cuda")
        x[:s.n_pos] = d[k]
        d[k] = x
    d["table"] = wide
    cols, n_pos = s.cols, s.n_pos
    s.cols, s.n_pos = 65536, 2 ** 20
    o, _ = s.run(b, "prefill", bf16)
    torch.cuda.synchronize()
    s.cols, s.n_pos = cols, n_pos
    s.check(o, bf16, planes=1 if bf16 else 2)


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_pool_of_more_than_four_gigabytes(b, kind):
    """Pages whose bytes lie beyond 2^32."""
    s = Setup([70, 33], [2, 2], 16, 8, 128, seed=24)
    small = s.upload()
    n = 2 ** 32 // (2 * 8 * 16 * 128) + s.n_pages
    off = n - s.n_pages
    codes = torch.zeros((n, 2, 8, 16, 128), dtype=torch.uint8, device="cuda")
    scale = torch.ones((n, 2, 8), device="cuda")
    codes[off:] = small["codes"]
    scale[off:] = small["scale"]
    s.d = dict(small, codes=codes, scale=scale, table=small["table"] + off)
    few, s.n_pages = s.n_pages, n
    o, _ = s.run(b, kind, False)
    torch.cuda.synchronize()
    s.n_pages = few
    s.d["codes"], s.d["scale"] = codes[off:], scale[off:]
    assert not codes[:off].any()
    s.check(o, False)


# --------------------------------------------------------------------- packing

@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,Hkv,hd", [(1, 1, 64), (5, 8, 128), (37, 2, 64), (9, 7, 128)])
def test_pack_and_unpack(b, n, Hkv, hd, dt):
    rng = np.random.default_rng(n)
    n_src, n_dst = n + 2, n + 3
    x = rng.standard_normal((n_src, 2, Hkv, 16, hd)) * 2.0 ** rng.uniform(-50, 50, (n_src, 2, Hkv, 1, 1))
    x[0, 0, 0, 0, :5] = [np.inf, -np.inf, np.nan, 0.0, -0.0]
    x[1, 1] = 0.0
    xt = torch.from_numpy(x).to(torch.float32 if dt == "f32" else torch.bfloat16)
    x = xt.double().numpy()
    src, dst = rng.permutation(n_src)[:n].astype(np.int32), rng.permutation(n_dst)[:n].astype(np.int32)
    fill = rng.integers(0, 17, n).astype(np.int32)
    fill[0] = 16
    if n > 4:
        src[2], dst[3], fill[4] = -1, n_dst, 99          # left out; clamped
    codes = torch.full((n_dst, 2, Hkv, 16, hd), 0x55, dtype=torch.uint8, device="cuda")
    scale = torch.full((n_dst, 2, Hkv), 5.0, device="cuda")
    b.s2op_kv8_pack_pages(xt.cuda(), dt == "bf16", n_src, dev(src), dev(fill), codes, scale, n_dst, dev(dst), n, Hkv, hd)
    torch.cuda.synchronize()
    want, wscale = np.full((n_dst, 2, Hkv, 16, hd), 0x55, np.uint8), np.full((n_dst, 2, Hkv), 5.0)
    for i in range(n):
        if not (0 <= src[i] < n_src and 0 <= dst[i] < n_dst):
            continue
        y = x[src[i]].copy()
        y[:, :, min(fill[i], 16):] = 0
        e = ref.exponent(y)
        with np.errstate(invalid="ignore"):
            want[dst[i]] = ref.encode(y / 2.0 ** e[..., None, None])
        wscale[dst[i]] = 2.0 ** e
    np.testing.assert_array_equal(scale.cpu().numpy(), wscale.astype(np.float32))
    assert ref.same_codes(codes.cpu().numpy(), want).all()

    back = torch.full((n_src, 2, Hkv, 16, hd), 3.0, device="cuda", dtype=xt.dtype)
    ok = [i for i in range(n) if 0 <= src[i] < n_src and 0 <= dst[i] < n_dst]
    b.s2op_kv8_unpack_pages(codes, scale, n_dst, dev(dst), back, dt == "bf16", n_src, dev(src), n, Hkv, hd)
    torch.cuda.synchronize()
    got = back.double().cpu().numpy()
    rest = np.ones(n_src, bool)
    for i in ok:
        v = ref.VALUE[want[dst[i]]] * wscale[dst[i]][..., None, None]
        np.testing.assert_array_equal(got[src[i]], v)     # exact in fp32 and in bf16
        rest[src[i]] = False
    assert (got[rest] == 3.0).all()


def test_packed_prefix_is_what_decode_reads(b):
    """fp32 pages packed with every row in use give decode the blocks that the
    definition gives."""
    s = Setup([64], [1], 8, 2, 128, seed=16)
    rng = np.random.default_rng(16)
    x = rng.standard_normal((4, 2, 2, 16, 128), dtype=np.float32)
    s.codes[s.table[0, :4]] = 0
    d = s.upload()
    b.s2op_kv8_pack_pages(dev(x), False, 4, dev(np.arange(4, dtype=np.int32)), None, d["codes"], d["scale"], s.n_pages,
                          dev(s.table[0, :4]), 4, 2, 128)
    e = ref.exponent(x)
    s.codes[s.table[0, :4]], s.exps[s.table[0, :4]] = ref.encode(x / 2.0 ** e[..., None, None]), e
    o, _ = s.run(b, "decode", False)
    torch.cuda.synchronize()
    s.check(o, False)


# --------------------------------------------------------------------- page copies

@pytest.mark.parametrize("page_bytes,scale_bytes,layers,n_pages,n", [
    (16, 0, 1, 4, 2), (48, 4, 3, 9, 4), (4096, 16, 5, 40, 20), (32768, 64, 36, 30, 7), (131072, 0, 2, 12, 5),
    (16, 8, 2, 9001, 4500), (1040, 12, 4, 33, 1), (32768, 64, 1, 8, 0)])
def test_copy_pages(b, page_bytes, scale_bytes, layers, n_pages, n):
    rng = np.random.default_rng(page_bytes + n)
    kv = rng.integers(0, 256, (layers, n_pages, page_bytes), dtype=np.uint8)
    sc = rng.integers(0, 256, (layers, n_pages, scale_bytes), dtype=np.uint8) if scale_bytes else None
    perm = rng.permutation(n_pages)
    dst, src = perm[:n], rng.choice(perm[n:], n)
    kvd, scd = dev(kv), None if sc is None else dev(sc)
    b.s2op_kv_copy_pages(kvd, page_bytes, scd, scale_bytes, n_pages, layers, src, dst, n)
    torch.cuda.synchronize()
    kv[:, dst] = kv[:, src]
    np.testing.assert_array_equal(kvd.cpu().numpy(), kv)
    if sc is not None:
        sc[:, dst] = sc[:, src]
        np.testing.assert_array_equal(scd.cpu().numpy(), sc)


@pytest.mark.parametrize("rows,cols,ld,n", [(1, 1, 1, 1), (7, 13, 20, 5), (128, 107, 107, 4500), (3, 0, 4, 2)])
def test_remap_pages(b, rows, cols, ld, n):
    rng = np.random.default_rng(rows + n)
    perm = rng.permutation(max(2 * n + 4, 10)).astype(np.int32)
    src, dst = perm[:n], np.concatenate([perm[n:2 * n - 1], perm[n:n + 1]])    # two pages may become one
    table = rng.integers(-1, len(perm), (rows, ld)).astype(np.int32)
    d = dev(table)
    b.s2op_kv_remap_pages(d, rows, cols, ld, src, dst, n)
    torch.cuda.synchronize()
    to = dict(zip(src.tolist(), dst.tolist()))
    want = table.copy()
    want[:, :cols] = np.array([to.get(int(p), int(p)) for p in table[:, :cols].ravel()],
                              np.int32).reshape(rows, cols)
    np.testing.assert_array_equal(d.cpu().numpy(), want)
