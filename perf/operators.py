"""Cases of the 8-bit KV cache operators: decode and prompt attention over a
paged e4m3 cache with one scale per page, kv head and tensor, the packing of
fp32 / bf16 pages into that cache and back, and the copying of pages.

A page holds 16 tokens of every kv head: bytes [2 (K, V)][Hkv][16][hd] in
e4m3, and scales [2][Hkv], each a power of two, such that a cached value is
byte value x scale.  The scale of a block (16 tokens of one head) is the
smallest 2^e, -32 <= e <= 32, whose 448 * 2^e covers the block's largest
magnitude; a block that gets new tokens keeps the larger of its old scale and
the new tokens' one, its old values rescaled (exact but for e4m3's subnormals).

``own`` selects the framework's calls; otherwise the operators are computed
in their plain form from elementary torch operations.
"""

import numpy as np
import torch

own = False

PAGE = 16
EMIN, EMAX = -32, 32
EPS = float(np.float32(1e-6))
DEV = "cuda"


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one new frame of one sequence behind a 41-token prompt: the
        # interactive case, a single sequence where only latency counts
        dict(name="decode_1x41", op="decode", B=1, m=1, H=32, Hkv=8, hd=128, lo=41, hi=41, out="f32"),
        # a batch of 32 with about a thousand tokens each (a voice prompt of
        # 900 positions and up to 190 generated frames)
        dict(name="decode_32x1090", op="decode", B=32, m=1, H=32, Hkv=8, hd=128, lo=900, hi=1090, out="f32"),
        # the throughput batch: 128 sequences anywhere between prompt and end
        dict(name="decode_128x1700", op="decode", B=128, m=1, H=32, Hkv=8, hd=128, lo=200, hi=1700, out="bf16"),
        # few long contexts, two new tokens each (a drafted token checked with
        # the one before it): the keys have to be split over the machine
        dict(name="decode_2x32k_m2", op="decode", B=2, m=2, H=32, Hkv=8, hd=128, lo=31000, hi=32768, out="f32"),
        # the 41-token prompt itself
        dict(name="prefill_1x41", op="prefill", B=1, T=41, lo=0, hi=0, H=32, Hkv=8, hd=128, out="f32"),
        # the 1,024-token voice-clone prompt
        dict(name="prefill_1x1024", op="prefill", B=1, T=1024, lo=0, hi=0, H=32, Hkv=8, hd=128, out="f32"),
        # 16 requests, ragged, each behind cached pages of a voice prompt
        dict(name="prefill_16_cached", op="prefill", B=16, T=1500, lo=600, hi=900, H=32, Hkv=8, hd=128, out="bf16"),
        # one long prompt: bound by the tensor cores
        dict(name="prefill_1x8000", op="prefill", B=1, T=8000, lo=0, hi=0, H=32, Hkv=8, hd=128, out="bf16"),
        # a prefix of the fp32 cache packed into the 8-bit one, 36 layers of
        # 57 pages, the last page of each not full
        dict(name="pack_f32_2052", op="pack", n=2052, kv="f32", Hkv=8, hd=128),
        # one sequence's pages of one layer, brought back for a bf16 reader
        dict(name="unpack_bf16_69", op="unpack", n=69, kv="bf16", Hkv=8, hd=128),
        # 32 sequences forked: the last, partly filled page of each copied in
        # 36 layers
        dict(name="fork_32", op="copy", layers=36, pages=256, n=32, rows=0, cols=0, Hkv=8, hd=128, elem=1, scaled=True),
        # a pool compacted: 400 pages of 36 layers moved to the front, and the
        # page tables of 128 sequences rewritten
        dict(name="compact_400", op="copy", layers=36, pages=1000, n=400, rows=128, cols=107, Hkv=8, hd=128, elem=1,
             scaled=True),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "pack", "unpack", "copy"])
    H, Hkv, hd = rng.choice([(32, 8, 128), (32, 8, 128), (32, 8, 128), (8, 2, 128), (4, 2, 64), (24, 8, 128),
                             (16, 2, 64), (7, 7, 128)])
    out = rng.choice(["f32", "bf16"])
    if op == "decode":
        B = _log(rng, 1, 128)
        hi = _log(rng, 1, min(32768, 200000 // B))
        lo = rng.randint(max(0, hi // 4 - 1), hi)
        m = rng.randint(1, min(4, 8 // (H // Hkv)))
        return dict(op=op, B=B, m=m, H=H, Hkv=Hkv, hd=hd, lo=lo, hi=hi, out=out)
    if op == "prefill":
        B = _log(rng, 1, 24)
        T = _log(rng, B, 5000 if B == 1 else 1800)
        hi = rng.choice([0, _log(rng, 1, 4000 if B == 1 else 1200)])
        return dict(op=op, B=B, T=T, lo=hi // 2, hi=hi, H=H, Hkv=Hkv, hd=hd, out=out)
    if op in ("pack", "unpack"):
        return dict(op=op, n=_log(rng, 1, 2000), kv=rng.choice(["f32", "bf16"]), Hkv=Hkv, hd=hd)
    layers = _log(rng, 1, 36)
    pages = _log(rng, 8, 800)
    n = _log(rng, 1, pages // 2)
    rows = rng.choice([0, _log(rng, 1, 128)])
    elem = rng.choice([1, 1, 2, 4]) if pages < 300 else 1
    return dict(op=op, layers=layers, pages=pages, n=n, rows=rows, cols=rng.randint(1, 130) if rows else 0, Hkv=Hkv,
                hd=hd, elem=elem, scaled=elem == 1)


def _spread(case):
    """The lengths of a case, a fixed function of its numbers: cached tokens
    per sequence, and new tokens per sequence."""
    B = case["B"]
    rs = np.random.RandomState(B * 7919 + case["lo"] * 31 + case["hi"] + case.get("T", 0))
    cached = rs.randint(case["lo"], case["hi"] + 1, B)
    if case["op"] == "decode":
        return cached, np.full(B, case["m"])
    # T rows over B sequences, each at least one
    cuts = np.sort(rs.choice(np.arange(1, case["T"]), B - 1, replace=False)) if B > 1 else np.zeros(0, int)
    return cached, np.diff(np.concatenate([[0], cuts, [case["T"]]]))


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed * 2 + 1)
    rs = np.random.RandomState(seed % (1 << 31))
    s = dict(case=case)
    Hkv, hd = case["Hkv"], case["hd"]
    randn = lambda *n: torch.randn(*n, device=DEV, generator=g)  # noqa: E731
    ints = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)  # noqa: E731

    def cache(n):
        """n pages of a cache in use: values of the size that normed keys and
        projected values have, heads of unlike size."""
        size = torch.exp2(2 * torch.rand(2, Hkv, 1, 1, device=DEV, generator=g) - 1)
        x = randn(n, 2, Hkv, PAGE, hd).mul_(size)
        e = _exponent(x.abs().amax((-1, -2)))
        x.mul_(torch.exp2(-e.float())[..., None, None])
        return x.to(torch.float8_e4m3fn).view(torch.uint8), torch.exp2(e.float())

    if case["op"] in ("decode", "prefill"):
        cached, new = _spread(case)
        order = rs.permutation(case["B"])
        cached, new = cached[order], new[order]
        need = (cached + new + PAGE - 1) // PAGE
        cols = int(need.max()) + 1
        n_pages = int(need.sum()) + 3
        free = rs.permutation(n_pages)
        table = np.full((case["B"], cols), free[-1])
        at = 0
        for b, k in enumerate(need):
            table[b, :k] = free[at:at + k]
            at += k
        T = int(new.sum())
        n_pos = cols * PAGE
        ang = torch.arange(n_pos, device=DEV, dtype=torch.float64)[:, None] * torch.pow(
            torch.tensor(1e6, device=DEV, dtype=torch.float64), -2.0 * torch.arange(hd // 2, device=DEV) / hd)
        s.update(qkv=randn(T, (case["H"] + 2 * Hkv) * hd), table=ints(table), cols=cols, n_pages=n_pages, n_pos=n_pos,
                 pos=ints(cached), row0=ints(np.concatenate([[0], np.cumsum(new)])), T=T,
                 most_new=int(new.max()), most_keys=int((cached + new).max()),
                 q_gain=torch.rand(hd, device=DEV, generator=g) + 0.5,
                 k_gain=torch.rand(hd, device=DEV, generator=g) + 0.5,
                 cos=ang.cos().float().bfloat16().float(), sin=ang.sin().float().bfloat16().float(),
                 o=torch.zeros(T, case["H"] * hd, device=DEV,
                               dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16))
        s["kv8"], s["scale"] = cache(n_pages)
    elif case["op"] in ("pack", "unpack"):
        n = case["n"]
        dt = torch.float32 if case["kv"] == "f32" else torch.bfloat16
        s["src"], s["dst"] = ints(rs.permutation(n)), ints(rs.permutation(n))
        if case["op"] == "pack":
            fill = np.full(n, PAGE)
            fill[rs.rand(n) < 1 / 57] = rs.randint(0, PAGE)
            s["fill"] = ints(fill)
            s["kv"] = randn(n, 2, Hkv, PAGE, hd).to(dt)
            s["kv8"] = torch.zeros(n, 2, Hkv, PAGE, hd, device=DEV, dtype=torch.uint8)
            s["scale"] = torch.zeros(n, 2, Hkv, device=DEV)
        else:
            s["kv8"], s["scale"] = cache(n)
            s["kv"] = torch.zeros(n, 2, Hkv, PAGE, hd, device=DEV, dtype=dt)
    else:
        L, P, n = case["layers"], case["pages"], case["n"]
        size = 2 * Hkv * PAGE * hd * case["elem"]
        s["kv"] = torch.randint(0, 256, (L, P, size), device=DEV, generator=g, dtype=torch.uint8)
        s["scale"] = torch.exp2(torch.randint(-8, 8, (L, P, 2, Hkv), device=DEV, generator=g).float()) \
            if case["scaled"] else None
        if case["rows"]:      # compaction: pages from the back to free ones in front
            half = P // 2
            s["dst"] = np.sort(rs.permutation(half)[:n]).astype(np.int32)
            s["src"] = (half + np.sort(rs.permutation(P - half)[:n])).astype(np.int32)
            s["table"] = ints(rs.randint(0, P, (case["rows"], case["cols"])))
        else:                 # fork: a page may be the source of several
            free = rs.permutation(P).astype(np.int32)
            s["dst"] = np.ascontiguousarray(free[:n])
            s["src"] = np.ascontiguousarray(rs.choice(free[n:], n).astype(np.int32))
            s["table"] = None
        s["src_dev"], s["dst_dev"] = ints(s["src"]), ints(s["dst"])
    return s


# ---------------------------------------------------------------- the plain forms

def _exponent(amax):
    """The smallest e of [EMIN, EMAX] with amax <= 448 * 2^e."""
    f, x = torch.frexp(amax)
    e = torch.where(f <= 0.875, x - 9, x - 8)
    return torch.where(amax == 0, EMIN, e.clamp(EMIN, EMAX))


def _pow2(e):
    """2^e, exactly (float64)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(x):
    """x (float64) rounded to the nearest e4m3 value, ties to even."""
    a = x.abs()
    _, p = torch.frexp(a)
    step = _pow2((p - 1).clamp(min=-6) - 3)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=448.0)


def _bytes(v):
    return v.float().to(torch.float8_e4m3fn).view(torch.uint8)


def _values(u8):
    return u8.view(torch.float8_e4m3fn).float()


def _norm_rope(x, gain, cos, sin):
    """RMSNorm per head, then the rotation of (i, i + hd/2); x [T, heads, hd],
    cos / sin [T, hd/2]; in x's type."""
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain.to(x.dtype)
    a, b = x.chunk(2, -1)
    c, s = cos[:, None].to(x.dtype), sin[:, None].to(x.dtype)
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _plain_attention(s):
    c = s["case"]
    H, Hkv, hd, B, T = c["H"], c["Hkv"], c["hd"], c["B"], s["T"]
    kv8, scale, table = s["kv8"], s["scale"], s["table"].long()
    pos, row0 = s["pos"].long(), s["row0"].long()
    new = row0[1:] - row0[:-1]
    seq = torch.repeat_interleave(torch.arange(B, device=DEV), new, output_size=T)
    at = pos[seq] + torch.arange(T, device=DEV) - row0[seq]
    x = s["qkv"].view(T, H + 2 * Hkv, hd)
    q = _norm_rope(x[:, :H], s["q_gain"], s["cos"][at], s["sin"][at]) / hd ** 0.5
    # rounding to 8 bits is taken on keys in 64 bits: next to the middle of
    # two e4m3 values the last bits of 32 decide
    k = _norm_rope(x[:, H:H + Hkv].double(), s["k_gain"], s["cos"][at], s["sin"][at])
    v = x[:, H + Hkv:].double()

    # the new tokens into their pages [B, J pages, 2, Hkv, 16, hd]
    J = (s["most_new"] + PAGE - 2) // PAGE + 1
    pj = pos[:, None] // PAGE + torch.arange(J, device=DEV)
    live = pj * PAGE < (pos + new)[:, None]
    page = table.gather(1, pj.clamp(max=s["cols"] - 1))
    slot = pj[..., None] * PAGE + torch.arange(PAGE, device=DEV)
    is_old = (slot < pos[:, None, None])[:, :, None, None, :, None]
    is_new = ((slot >= pos[:, None, None]) & (slot < (pos + new)[:, None, None]))[:, :, None, None, :, None]
    r = (row0[:-1, None, None] + slot - pos[:, None, None]).clamp(0, T - 1)
    x = torch.stack([k, v], 1)[r].permute(0, 1, 3, 4, 2, 5) * is_new
    e_new = _exponent(x.abs().amax((-1, -2)))
    e_old = torch.where(is_old.any(-2)[..., 0], torch.log2(scale[page]).round().int(), EMIN)
    e = torch.maximum(e_new, e_old)
    old = kv8[page]
    kept = _e4m3(_values(old).double() * _pow2(e_old - e)[..., None, None])
    q8 = torch.where(is_new, _bytes(_e4m3(x * _pow2(-e)[..., None, None])),
                     torch.where(is_old, _bytes(kept), old))
    kv8[page[live]] = q8[live]
    scale[page[live]] = torch.exp2(e.float())[live]

    # attention over the cache as it now stands
    L = (s["most_keys"] + PAGE - 1) // PAGE
    pages = table[:, :L]
    kv = _values(kv8[pages]) * scale[pages][..., None, None]
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, B, Hkv, L * PAGE, hd)
    M = s["most_new"]
    rows = (row0[:-1, None] + torch.arange(M, device=DEV)).clamp(max=T - 1)
    qs = q[rows].view(B, M, Hkv, H // Hkv, hd).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, hd)
    sc = (qs @ kv[0].transpose(-1, -2)).view(B, Hkv, H // Hkv, M, L * PAGE)
    last = pos[:, None] + torch.arange(M, device=DEV)
    sc.masked_fill_((torch.arange(L * PAGE, device=DEV) > last[..., None])[:, None, None], float("-inf"))
    sc.sub_(sc.amax(-1, keepdim=True)).exp_()
    sc.div_(sc.sum(-1, keepdim=True))
    o = (sc.view(B, Hkv, -1, L * PAGE) @ kv[1]).view(B, H, M, hd)
    o = o[seq, :, torch.arange(T, device=DEV) - row0[seq]].reshape(T, H * hd)
    return dict(o=o.to(s["o"].dtype), cache=kv8.view(torch.float8_e4m3fn), scale=scale)


def _plain_pack(s):
    src, dst = s["src"].long(), s["dst"].long()
    if s["case"]["op"] == "unpack":
        s["kv"][dst] = (_values(s["kv8"][src]) * s["scale"][src][..., None, None]).to(s["kv"].dtype)
        return dict(kv=s["kv"])
    x = s["kv"][src].float()
    x = x * (torch.arange(PAGE, device=DEV) < s["fill"].long()[:, None])[:, None, None, :, None]
    e = _exponent(x.abs().amax((-1, -2)))
    s["kv8"][dst] = (x * torch.exp2(-e.float())[..., None, None]).clamp(-448, 448).to(
        torch.float8_e4m3fn).view(torch.uint8)
    s["scale"][dst] = torch.exp2(e.float())
    return dict(cache=s["kv8"].view(torch.float8_e4m3fn), scale=s["scale"])


def _plain_copy(s):
    src, dst = s["src_dev"].long(), s["dst_dev"].long()
    s["kv"][:, dst] = s["kv"][:, src]
    if s["scale"] is not None:
        s["scale"][:, dst] = s["scale"][:, src]
    if s["table"] is not None:
        to = torch.arange(s["case"]["pages"], device=DEV, dtype=torch.int32)
        to[src] = s["dst_dev"]
        s["table"] = to[s["table"].long()]
    return dict(kv=s["kv"], scale=s["scale"], table=s["table"])


# ---------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    if own:
        return _own(s)
    if c["op"] in ("decode", "prefill"):
        return _plain_attention(s)
    if c["op"] == "copy":
        return _plain_copy(s)
    return _plain_pack(s)


def _own(s):
    from serving_dual_ar_gb300 import binding as s2
    c = s["case"]
    Hkv, hd = c["Hkv"], c["hd"]
    if c["op"] in ("decode", "prefill"):
        H = c["H"]
        if "workspace" not in s:      # a server allocates it once for its largest batch
            size = s2.s2op_attn_decode_kv8_workspace_bytes(c["B"], c["m"], H, Hkv, hd) if c["op"] == "decode" else \
                s2.s2op_attn_prefill_kv8_workspace_bytes(s["T"], c["B"], H, Hkv, hd)
            s["workspace"] = torch.zeros(size, dtype=torch.uint8, device=DEV)
        ld = (H + 2 * Hkv) * hd
        tail = (H, Hkv, hd, s["q_gain"], s["k_gain"], EPS, s["cos"], s["sin"], s["n_pos"])
        cache = (s["kv8"], s["scale"], s["n_pages"], s["table"], s["cols"], s["o"], c["out"] == "bf16", H * hd,
                 s["workspace"])
        if c["op"] == "decode":
            s2.s2op_attn_decode_kv8(s["qkv"], ld, c["B"], c["m"], *tail, s["pos"], *cache)
        else:
            s2.s2op_attn_prefill_kv8(s["qkv"], ld, s["T"], c["B"], s["row0"], s["pos"], *tail, *cache)
        return dict(o=s["o"], cache=s["kv8"].view(torch.float8_e4m3fn), scale=s["scale"])
    if c["op"] == "pack":
        s2.s2op_kv8_pack_pages(s["kv"], c["kv"] == "bf16", c["n"], s["src"], s["fill"], s["kv8"], s["scale"], c["n"],
                               s["dst"], c["n"], Hkv, hd)
        return dict(cache=s["kv8"].view(torch.float8_e4m3fn), scale=s["scale"])
    if c["op"] == "unpack":
        s2.s2op_kv8_unpack_pages(s["kv8"], s["scale"], c["n"], s["src"], s["kv"], c["kv"] == "bf16", c["n"], s["dst"],
                                 c["n"], Hkv, hd)
        return dict(kv=s["kv"])
    s2.s2op_kv_copy_pages(s["kv"], 2 * Hkv * PAGE * hd * c["elem"], s["scale"], 2 * Hkv * 4 if c["scaled"] else 0,
                          c["pages"], c["layers"], s["src"], s["dst"], c["n"])
    if c["rows"]:
        s2.s2op_kv_remap_pages(s["table"], c["rows"], c["cols"], c["cols"], s["src"], s["dst"], c["n"])
    return dict(kv=s["kv"], scale=s["scale"], table=s["table"])


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    Hkv, hd = case["Hkv"], case["hd"]
    if case["op"] in ("decode", "prefill"):
        cached, new = _spread(case)
        H, T = case["H"], int(new.sum())
        pairs = int((new * cached + new * (new + 1) // 2).sum())
        block = 2 * Hkv * hd
        moved = (int(cached.sum()) + T) * block + int(((cached + new + PAGE - 1) // PAGE).sum()) * 2 * Hkv * 4
        return dict(bytes=moved + T * ((H + 2 * Hkv) * hd * 4 + H * hd * (4 if case["out"] == "f32" else 2)),
                    flops=4 * pairs * H * hd)
    if case["op"] in ("pack", "unpack"):
        elems = case["n"] * 2 * Hkv * PAGE * hd
        return dict(bytes=elems * (5 if case["kv"] == "f32" else 3) + case["n"] * 2 * Hkv * 4, flops=elems)
    page = 2 * Hkv * PAGE * hd * case["elem"] + (2 * Hkv * 4 if case["scaled"] else 0)
    return dict(bytes=2 * case["layers"] * case["n"] * page + 8 * case["rows"] * case["cols"], flops=0)


# ---------------------------------------------------------------- the definition in 64 bits

def _grid64():
    """Every non-negative finite e4m3 value, in order: 2^(e-7) (1 + m/8), or
    2^-6 m/8 where e is 0."""
    code = torch.arange(127, device=DEV)
    e, m = code // 8, (code % 8).double()
    return torch.where(e == 0, m / 512, (1 + m / 8) * torch.pow(torch.tensor(2.0, device=DEV, dtype=torch.float64),
                                                                (e - 7).double()))


def _nearest64(x, grid):
    """The value of the grid next to each x, the even code on a tie."""
    a = x.abs().clamp(max=448.0).contiguous()
    hi = torch.searchsorted(grid, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    down, up = a - grid[lo], grid[hi] - a
    code = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return torch.where(x < 0, -grid[code], grid[code])


def _scale64(x):
    """2^e of each block over its last two dimensions, by counting powers."""
    powers = torch.pow(torch.tensor(2.0, device=DEV, dtype=torch.float64),
                       torch.arange(EMIN, EMAX + 1, device=DEV).double())
    amax = x.abs().flatten(-2).max(-1).values
    i = torch.searchsorted(448.0 * powers, amax.contiguous()).clamp(max=EMAX - EMIN)
    return powers[i]


def exact(case, seed):
    s = prepare(case, seed)
    grid = _grid64()
    Hkv, hd = case["Hkv"], case["hd"]
    if case["op"] == "copy":
        return None
    if case["op"] == "unpack":
        kv = torch.zeros(s["kv"].shape, dtype=torch.float64, device=DEV)
        kv[s["dst"].long()] = (s["kv8"].view(torch.float8_e4m3fn).double() * s["scale"].double()[..., None, None])[
            s["src"].long()]
        return dict(kv=kv)
    if case["op"] == "pack":
        x = s["kv"].double()[s["src"].long()]
        for t in range(PAGE):
            x[:, :, :, t] *= (s["fill"] > t).double()[:, None, None, None]
        sc = _scale64(x)
        cache, scale = torch.empty_like(x), torch.empty_like(sc)
        cache[s["dst"].long()] = _nearest64(x / sc[..., None, None], grid)
        scale[s["dst"].long()] = sc
        return dict(cache=cache, scale=scale)
    H, G = case["H"], case["H"] // Hkv
    cache, scale = s["kv8"].view(torch.float8_e4m3fn).double(), s["scale"].double()
    row0, pos, table = s["row0"].tolist(), s["pos"].tolist(), s["table"].tolist()
    o = torch.empty(s["T"], H, hd, dtype=torch.float64, device=DEV)
    x = s["qkv"].double().view(s["T"], H + 2 * Hkv, hd)
    half = hd // 2
    for b in range(case["B"]):
        r0, n, p0 = row0[b], row0[b + 1] - row0[b], pos[b]
        c, d = s["cos"][p0:p0 + n].double()[:, None], s["sin"][p0:p0 + n].double()[:, None]
        y = x[r0:r0 + n].clone()
        for heads, gain in ((slice(0, H), s["q_gain"]), (slice(H, H + Hkv), s["k_gain"])):
            z = y[:, heads]
            z = z / torch.sqrt(z.pow(2).sum(-1, keepdim=True) / hd + EPS) * gain.double()
            y[:, heads] = torch.cat([z[..., :half] * c - z[..., half:] * d, z[..., half:] * c + z[..., :half] * d], -1)
        for j in range(p0 // PAGE, (p0 + n - 1) // PAGE + 1):
            page = table[b][j]
            first, end = max(p0, j * PAGE), min(p0 + n, (j + 1) * PAGE)
            z = y[first - p0:end - p0, H:].reshape(end - first, 2, Hkv, hd).permute(1, 2, 0, 3)
            had = first - j * PAGE
            sc = _scale64(z)
            if had:
                sc = torch.maximum(sc, scale[page])
                cache[page, :, :, :had] = _nearest64(
                    cache[page, :, :, :had] * (scale[page] / sc)[..., None, None], grid)
            cache[page, :, :, had:had + end - first] = _nearest64(z / sc[..., None, None], grid)
            scale[page] = sc
        used = torch.tensor(table[b][:(p0 + n + PAGE - 1) // PAGE], device=DEV)
        kv = (cache[used] * scale[used][..., None, None]).permute(1, 2, 0, 3, 4).reshape(2, Hkv, -1, hd)
        hide = torch.arange(kv.shape[2], device=DEV) > (p0 + torch.arange(n, device=DEV))[:, None]
        for h in range(H):
            w = y[:, h] @ kv[0, h // G].T * hd ** -0.5
            o[r0:r0 + n, h] = torch.softmax(w.masked_fill(hide, float("-inf")), -1) @ kv[1, h // G]
    return dict(o=o.reshape(s["T"], H * hd), cache=cache, scale=scale)
