"""Norm, rotation + cache append and attention on the GPU against their
definitions in 64 bits (layer_ref.py), at the sizes, types and masks where
they can go wrong."""
import math

import pytest
import torch

import bit_weight_only_g128_gb300 as w4
import layer_ref as ref

pytestmark = pytest.mark.gpu

FP16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ------------------------------------------------------------------ norm

NORM_SHAPES = [(1, 1), (3, 7), (1, 8), (5, 64), (2, 100), (33, 128), (7, 1000), (1, 4096), (16, 5120), (305, 8192),
               (2, 11008), (400, 2056), (3, 28672), (2, 65536), (2, 65535)]


@pytest.mark.parametrize("M,K", NORM_SHAPES)
@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_norm(M, K, dtype):
    g = gen(M * 7 + K)
    x, r, w = normal(g, M, K, dtype=dtype), normal(g, M, K, std=4, dtype=dtype), normal(g, K, dtype=dtype)
    want, _ = ref.rms_norm(x, w, r)
    y, h = w4.rms_norm(x, w, residual=r)
    assert same(h, (x.float() + r.float()).to(dtype))
    ref.within(y, want, want.abs() * ref.norm_rel(K))
    assert same(w4.rms_norm(x, w, residual=r)[0], y)
    want, _ = ref.rms_norm(x, w, eps=1e-3)
    ref.within(w4.rms_norm(x, w, eps=1e-3), want, want.abs() * ref.norm_rel(K))


@pytest.mark.parametrize("M,K", NORM_SHAPES)
@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_norm_codes(M, K, dtype):
    g = gen(M * 5 + K)
    x, r, w = normal(g, M, K, dtype=dtype), normal(g, M, K, std=4, dtype=dtype), normal(g, K, dtype=dtype)
    if M > 2:
        x[1], r[1] = 0, 0
    want, _ = ref.rms_norm(x, w, r)
    top = want.abs().amax(1)
    s = torch.where(top > 0, top / 127, 1.0)
    rel = 2 * ref.norm_rel(K)
    aq, sa, h = w4.rms_norm(x, w, residual=r, quant="int8")
    assert aq.dtype == torch.int8 and same(h, (x.float() + r.float()).to(dtype))
    assert ((sa.double() - s).abs() <= rel * s).all()
    # the code is the nearest integer to a quotient within `rel` of y / s
    assert ((aq.double() - want / s[:, None]).abs() <= 0.5 + 127 * (rel + ref.E32)).all()
    assert int(aq.abs().amax()) <= 127
    codes, sc, _ = w4.rms_norm(x, w, residual=r, quant="codes")
    assert codes.dtype == dtype and torch.equal(codes.float(), aq.float()) and torch.equal(sc, sa)
    if M > 2:
        assert float(sa[1]) == 1.0 and not aq[1].any()


def test_norm_strides_alignment_and_in_place():
    g = gen(3)
    for dtype in (FP16, BF16):
        wide = normal(g, 9, 700, dtype=dtype)
        w = normal(g, 257, dtype=dtype)
        for lo, K in ((0, 256), (8, 256), (1, 256), (3, 255), (100, 104)):  # aligned, shifted, odd
            x, r = wide[:, lo:lo + K], wide[:, 300 + lo:300 + lo + K]
            wk = w[1:K + 1] if lo == 1 else w[:K]
            want, h64 = ref.rms_norm(x, wk, r)
            buf = torch.full((9, K + 24), 7.0, dtype=dtype, device="cuda")
            y, h = w4.rms_norm(x, wk, residual=r, residual_out=buf[:, 8:K + 8])
            ref.within(y, want, want.abs() * ref.norm_rel(K))
            assert torch.equal(h, (x.float() + r.float()).to(dtype))
            assert (buf[:, :8] == 7).all() and (buf[:, K + 8:] == 7).all()
            # the residual stream updated in place
            r2 = r.clone()
            y2, h2 = w4.rms_norm(x, wk, residual=r2, residual_out=r2)
            assert h2 is r2 and torch.equal(r2, h) and torch.equal(y2, y)
            q1 = w4.rms_norm(x, wk, residual=r, quant="int8")
            r2 = r.clone()
            q2 = w4.rms_norm(x, wk, residual=r2, residual_out=r2, quant="int8")
            assert torch.equal(q1[0], q2[0]) and torch.equal(q1[1], q2[1]) and torch.equal(r2, h)
    assert w4.rms_norm(torch.empty((0, 64), dtype=FP16, device="cuda"), w[:64].half()).shape == (0, 64)


def test_norm_extremes():
    # the largest fp16 values: the sum of squares stays far inside fp32
    x = torch.full((2, 4096), 65504.0, dtype=FP16, device="cuda")
    w = torch.ones(4096, dtype=FP16, device="cuda")
    y, h = w4.rms_norm(x, w, residual=x)
    assert (y == 1).all() and torch.isinf(h).all()  # h beyond fp16, y from the fp32 sum
    # subnormal rows: eps decides
    x = torch.full((1, 512), 2.0 ** -24, dtype=FP16, device="cuda")
    want, _ = ref.rms_norm(x, w[:512])
    ref.within(w4.rms_norm(x, w[:512]), want, want.abs() * ref.norm_rel(512))


def test_codes_through_the_gemm():
    """rms_norm's codes multiplied by gemm_scaled are s_a * sum a_q deq, on
    every path, with the fused gate/up epilogue too."""
    g = gen(11)
    K, N, group = 1024, 256, 128
    pw = w4.quantize_pack(normal(g, K, N, std=0.02), group)
    for dtype in (FP16, BF16):
        deq = w4.dequantize(pw, dtype=dtype).double()
        for M, path in ((3, "decode"), (16, "auto"), (40, "tensor"), (300, "tensor-pair")):
            x, w = normal(g, M, K, dtype=dtype), normal(g, K, dtype=dtype)
            codes, s = w4.rms_norm(x, w, quant="codes")
            y = w4.gemm_scaled(codes, s, pw, path=path)
            a = codes.double() * s.double()[:, None]
            want, mag = a @ deq, a.abs() @ deq.abs()
            # one weight rounding (none on the decode path), K additions, one rounding of y
            ref.within(y, want, (ref.U[dtype] + (K + 8) * ref.E32) * mag)
            gate, up = want[:, :N // 2], want[:, N // 2:]
            tol = (ref.U[dtype] + (K + 8) * ref.E32) * mag + ref.U[dtype] * want.abs()
            silu = gate * torch.sigmoid(gate)
            # |silu'| <= 1.1 carries the gate's error, and the exponential's few ulps
            t = (1.1 * tol[:, :N // 2]) * (up.abs() + tol[:, N // 2:]) + silu.abs() * (tol[:, N // 2:] + 16 * ref.E32 * up.abs())
            ref.within(w4.gemm_scaled(codes, s, pw, path=path, silu_mul=True), silu * up, t)


# ------------------------------------------------------------------ rotation and append


def table(n, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    angle = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def new_cache(g, pages, hk, page, D, dtype, fill=None):
    scales = [None, None]
    if dtype == E4M3:
        scales = [0.01 + 0.02 * torch.rand((hk,), generator=g, device="cuda") for _ in "kv"]
    cache = w4.new_kv_cache(pages, hk, page, D, dtype, *scales)
    if fill == "nan":
        for t in (cache.k, cache.v):
            t.view(torch.uint8).fill_(0xFF)  # NaN in all three types
    return cache


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,cache_dtype", [(FP16, FP16), (BF16, BF16), (FP16, E4M3), (BF16, E4M3)])
@pytest.mark.parametrize("T,heads,hk,D,rot,page", [
    (1, 32, 32, 128, 128, 16), (1, 1, 1, 64, 64, 16), (17, 8, 1, 128, 64, 32), (130, 5, 5, 64, 32, 64),
    (3, 64, 8, 128, 128, 256), (9, 10, 2, 128, 30, 128), (6, 4, 2, 64, 2, 16), (1001, 16, 2, 128, 128, 16)])
def test_rope_append(T, heads, hk, D, rot, page, dtype, cache_dtype, interleaved):
    g = gen(T + heads * 3 + rot)
    pages = -(-T // page) + 3
    cache = new_cache(g, pages, hk, page, D, cache_dtype, fill="nan")
    qkv = normal(g, T, (heads + 2 * hk) * D, std=2, dtype=dtype)
    cs = table(2000, rot)
    pos = torch.randint(0, 2000, (T,), generator=g, device="cuda", dtype=torch.int32)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
    if T > 4:
        slots[2] = -1
        slots[4] = -7
    q = w4.rope_append(qkv, cs, pos, slots, cache, interleaved=interleaved)
    x = qkv.view(T, heads + 2 * hk, D)
    want = ref.rope(x[:, :heads + hk], cs, pos, interleaved)
    mag = x[:, :heads + hk].double().abs().amax(2, keepdim=True) * 4 * ref.E32  # two products and a sum
    ref.within(q, want[:, :heads], mag[:, :heads].expand(-1, -1, D))
    keep = slots >= 0
    used = torch.zeros(pages * page, dtype=torch.bool, device="cuda")
    used[slots[keep]] = True
    for t, scale, new, m in ((cache.k, cache.k_scale, want[:, heads:], mag[:, heads:]),
                             (cache.v, cache.v_scale, x[:, heads + hk:].double(), None)):
        flat = t.view(torch.uint8).view(pages, hk, page, -1).transpose(1, 2).reshape(pages * page, hk, -1)
        assert (flat[~used] == 0xFF).all(), "a slot that was not named was written"
        got = flat[slots[keep]].contiguous().view(t.dtype)
        new = new[keep]
        if scale is None:
            ref.within(got, new, torch.zeros_like(new) if m is None else m[keep].expand_as(new))
        else:
            z = new / scale.double()[:, None]
            near = z.clamp(-448, 448).float().to(E4M3).double()
            # the nearest code; next to a midpoint of two codes either of them
            err, best = (got.double() - z.clamp(-448, 448)).abs(), (near - z.clamp(-448, 448)).abs()
            slack = 8 * ref.E32 * (z.abs() + (0 if m is None else m[keep] / scale.double()[:, None] / ref.E32))
            assert (err <= best + slack).all()
    w4.device_status()


def test_rope_append_strided_and_saturating():
    g = gen(5)
    T, heads, hk, D, page = 7, 4, 2, 128, 16
    cols = (heads + 2 * hk) * D
    wide = normal(g, T, cols + 40, std=3000, dtype=FP16)
    cs, pos = table(50, D), torch.arange(T, device="cuda", dtype=torch.int32)
    slots = torch.arange(T, device="cuda")
    for lo in (0, 8, 3):  # aligned rows, and rows that take the element path
        qkv = wide[:, lo:lo + cols]
        a, b = new_cache(g, 2, hk, page, D, FP16), new_cache(g, 2, hk, page, D, FP16)
        qa = w4.rope_append(qkv, cs, pos, slots, a)
        qb = w4.rope_append(qkv.contiguous(), cs, pos, slots, b)
        assert torch.equal(qa, qb) and torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
        e = new_cache(g, 2, hk, page, D, E4M3)
        w4.rope_append(qkv, cs, pos, slots, e)
        assert e.k.float().abs().amax() == 448 and torch.isfinite(e.v.float()).all()
    w4.device_status()


def test_rope_append_out_of_range_data_is_recorded_and_skipped():
    g = gen(6)
    cache = new_cache(g, 3, 2, 16, 64, FP16, fill="nan")
    qkv = normal(g, 3, 6 * 64, dtype=FP16)
    cs = table(10, 64)
    ok = torch.arange(3, device="cuda", dtype=torch.int32)
    for slots, pos in (([0, 48, 2], ok), ([0, 1 << 40, 2], ok),
                       ([-1, -1, -1], torch.tensor([0, 10, -1], device="cuda", dtype=torch.int32))):
        w4.rope_append(qkv, cs, pos, torch.tensor(slots, device="cuda"), cache)
        with pytest.raises(w4.W4A16Error) as e:
            w4.device_status()
        assert e.value.code == -6 and "0x80" in str(e.value)
    assert (cache.k[1:].view(torch.uint8) == 0xFF).all()
    w4.device_status()


# ------------------------------------------------------------------ attention


def scattered(g, lens, hk, page, D, dtype, spare=2, std=1.0):
    """A cache with sequences of the given lengths on pages in mixed order;
    every place that is no sequence's token is NaN, and so is every table
    entry beyond a sequence's pages out of range."""
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + spare
    cache = new_cache(g, pages, hk, page, D, dtype, fill="nan")
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    tab = torch.full((len(lens), max(counts + [1]) + 1), -123456, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        tab[b, :counts[b]] = order[at:at + counts[b]]
        at += counts[b]
        if n == 0:
            continue
        slot = torch.arange(n, device="cuda")
        pg = tab[b].long()[slot // page]
        for t in (cache.k, cache.v):
            x = normal(g, n, hk, D, std=std if dtype != E4M3 else 40 * std)
            x = x.clamp(-448, 448).to(dtype) if dtype == E4M3 else x.to(dtype)
            t.view(torch.uint8).view(pages, hk, page, -1)[pg, :, slot % page] = x.contiguous().view(torch.uint8).view(n, hk, -1)
    return cache, tab


def check_attention(q, cache, tab, starts, lens, got, lse, scale):
    """Each sequence's rows against the definition; starts and lens as lists."""
    for b, n in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        if lo == hi:
            continue
        out, l, tol, tol_l = ref.attention(q[lo:hi], cache, tab[b], n, scale, n - (hi - lo))
        ref.within(got[lo:hi], out, tol)
        if lse is not None:
            finite = torch.isfinite(l)
            assert torch.equal(torch.isneginf(lse[lo:hi]), ~finite)
            ref.within(lse[lo:hi][finite], l[finite], tol_l[finite])


DECODE = [
    # lens, heads, kv heads, D, page
    ([1], 1, 1, 64, 16),
    ([777], 64, 8, 128, 16),
    ([0, 1, 2, 15, 16, 17, 31, 33], 8, 8, 128, 16),
    ([63, 64, 65, 0, 127, 128, 129], 8, 2, 64, 32),
    ([5000, 1], 8, 1, 128, 64),
    ([257, 0, 4100], 10, 2, 128, 128),        # groups of 5
    ([300, 90], 32, 2, 128, 16),              # groups of 16
    ([300, 90, 1000], 40, 1, 64, 16),         # groups of 40: three tiles of rows
    ([40 + 13 * i for i in range(40)], 4, 4, 128, 16),
    ([0, 0], 4, 2, 128, 256),
    ([20000], 2, 1, 128, 256),
    ([513] * 5, 5, 5, 64, 64),
]


@pytest.mark.parametrize("lens,heads,hk,D,page", DECODE)
@pytest.mark.parametrize("dtype,cache_dtype", [(FP16, FP16), (BF16, BF16), (FP16, E4M3), (BF16, E4M3)])
def test_decode(lens, heads, hk, D, page, dtype, cache_dtype):
    g = gen(sum(lens) + heads)
    cache, tab = scattered(g, lens, hk, page, D, cache_dtype)
    B = len(lens)
    q = normal(g, B, heads, D, std=2, dtype=dtype)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got, lse = w4.attn_decode(q, cache, tab, n, return_lse=True)
    w4.device_status()
    check_attention(q, cache, tab, list(range(B + 1)), lens, got, lse, D ** -0.5)
    again, l2 = w4.attn_decode(q, cache, tab, n, return_lse=True)
    assert same(again, got) and same(l2, lse)
    assert same(w4.attn_decode(q, cache, tab, n), got)


PROMPT = [
    # (new, cached) per sequence, heads, kv heads, D, page
    ([(1, 1)], 1, 1, 64, 16),
    ([(37, 37)], 32, 32, 128, 16),
    ([(128, 128), (129, 129), (127, 127)], 4, 4, 128, 16),
    ([(256, 256), (257, 300), (1, 500), (0, 40), (3, 3)], 8, 2, 128, 32),
    ([(700, 2000), (33, 1000)], 5, 1, 128, 64),     # groups of 5 behind a prefix
    ([(300, 300)], 16, 1, 64, 128),
    ([(64, 1000), (65, 65), (200, 713)], 4, 2, 64, 256),
    ([(10, 4), (5, 0), (6, 6)], 2, 2, 128, 16),      # rows that see no key
    ([(1500, 1500)], 2, 2, 128, 16),
    ([(7, 4000), (1, 1)], 40, 1, 128, 16),
]


@pytest.mark.parametrize("seqs,heads,hk,D,page", PROMPT)
@pytest.mark.parametrize("dtype,cache_dtype", [(FP16, FP16), (BF16, BF16), (FP16, E4M3), (BF16, E4M3)])
def test_prompt(seqs, heads, hk, D, page, dtype, cache_dtype):
    new, lens = [a for a, _ in seqs], [n for _, n in seqs]
    g = gen(sum(new) + sum(lens))
    cache, tab = scattered(g, lens, hk, page, D, cache_dtype)
    lead, trail = 3, 2  # rows that belong to no sequence
    starts = [lead]
    for a in new:
        starts.append(starts[-1] + a)
    T = starts[-1] + trail
    q = normal(g, T, heads, D, std=2, dtype=dtype)
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.full((T, heads, D), 3.0, dtype=dtype, device="cuda")
    got, lse = w4.attn_prompt(q, cache, tab, st, n, out=out, return_lse=True)
    w4.device_status()
    check_attention(q, cache, tab, starts, lens, got, lse, D ** -0.5)
    assert (out[:lead] == 3).all() and (out[T - trail:] == 3).all()
    again = w4.attn_prompt(q, cache, tab, st, n)
    assert same(again[lead:T - trail].contiguous(), got[lead:T - trail].contiguous())


@pytest.mark.parametrize("seqs,heads,hk,D,page", [
    ([(16, 9000)], 16, 2, 128, 64),                  # few rows behind a long cache: split over it
    ([(1, 5000), (3, 700), (40, 41)], 8, 1, 128, 16),  # sequences too short for every part among them
    ([(300, 4000), (2, 0)], 2, 2, 64, 128),          # two row tiles with other last keys; rows that see none
    ([(9, 3001)], 40, 1, 128, 32),
])
@pytest.mark.parametrize("dtype,cache_dtype", [(FP16, FP16), (BF16, BF16), (FP16, E4M3), (BF16, E4M3)])
def test_prompt_split_over_a_long_cache(seqs, heads, hk, D, page, dtype, cache_dtype):
    new, lens = [a for a, _ in seqs], [n for _, n in seqs]
    g = gen(sum(new) + sum(lens))
    cache, tab = scattered(g, lens, hk, page, D, cache_dtype)
    starts = [sum(new[:b]) for b in range(len(new) + 1)]
    q = normal(g, starts[-1], heads, D, std=2, dtype=dtype)
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = w4.new_workspace(w4.attn_workspace_size(starts[-1], len(lens), heads, hk, D) + 4096)
    ws[-4096:] = 0x5A
    for _ in range(3):  # the same bits whichever part comes last, and the flags zero for the next call
        got, lse = w4.attn_prompt(q, cache, tab, st, n, return_lse=True, workspace=ws)
        w4.device_status()
        assert not ws[:32768].any() and (ws[-4096:] == 0x5A).all()
        check_attention(q, cache, tab, starts, lens, got, lse, D ** -0.5)
        again, l2 = w4.attn_prompt(q, cache, tab, st, n, return_lse=True, workspace=ws)
        assert same(again, got) and same(l2, lse)


def test_attention_workspaces():
    """A workspace too small or misaligned is refused; one serves decode,
    prompt and GEMM calls in turn."""
    g = gen(23)
    lens, heads, hk, D = [300, 70], 8, 2, 128
    cache, tab = scattered(g, lens, hk, 16, D, FP16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st = torch.tensor([0, 5, 7], dtype=torch.int32, device="cuda")
    qd, qp = normal(g, 2, heads, D, dtype=FP16), normal(g, 7, heads, D, dtype=FP16)
    calls = [lambda ws: w4.attn_decode(qd, cache, tab, n, workspace=ws),
             lambda ws: w4.attn_prompt(qp, cache, tab, st, n, workspace=ws)]
    pw = w4.quantize_pack(normal(g, 1024, 512, std=0.02), 128)
    x = normal(g, 40, 1024, dtype=FP16)
    calls.append(lambda ws: w4.gemm(x, pw, path="tensor", parts=4, workspace=ws))
    calls.append(lambda ws: w4.gemm(x[:3], pw, path="decode-streamk", workspace=ws))
    for call in calls[:2]:
        for ws, code in ((w4.new_workspace(4096), -4), (w4.new_workspace(64 << 20)[8:], -3)):
            with pytest.raises(w4.W4A16Error) as e:
                call(ws)
            assert e.value.code == code
    ws = w4.new_workspace(64 << 20)
    want = [call(None) for call in calls]
    for _ in range(3):
        for call, y in zip(calls, want):
            assert same(call(ws), y)
            assert not ws[:32768].any()
    w4.device_status()


@pytest.mark.parametrize("cache_dtype", [FP16, E4M3])
@pytest.mark.parametrize("std,scale", [(0.0, None), (30.0, None), (1.0, -0.3), (1.0, 0.0), (200.0, 1.0)])
def test_attention_of_extreme_scores(std, scale, cache_dtype):
    """Uniform rows (zero queries or scale), one-hot rows, a negative scale."""
    g = gen(17)
    lens, heads, hk, D, page = [300, 1, 130], 8, 2, 128, 16
    cache, tab = scattered(g, lens, hk, page, D, cache_dtype)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = normal(g, 3, heads, D, std=std, dtype=FP16)
    got, lse = w4.attn_decode(q, cache, tab, n, scale=scale, return_lse=True)
    check_attention(q, cache, tab, [0, 1, 2, 3], lens, got, lse, D ** -0.5 if scale is None else scale)
    new = [100, 1, 130]
    starts = [0, 100, 101, 231]
    q = normal(g, 231, heads, D, std=std, dtype=FP16)
    got, lse = w4.attn_prompt(q, cache, tab, torch.tensor(starts, dtype=torch.int32, device="cuda"), n, scale=scale,
                              return_lse=True)
    check_attention(q, cache, tab, starts, lens, got, lse, D ** -0.5 if scale is None else scale)
    w4.device_status()


def test_attention_of_large_bf16_queries_over_an_e4m3_cache():
    """bf16 queries beyond fp16's range, over 8-bit keys."""
    g = gen(18)
    lens, heads, hk, D, page = [100, 33], 4, 2, 64, 16
    cache, tab = scattered(g, lens, hk, page, D, E4M3)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for std, scale in ((1e6, 1e-7), (1e-9, 1e8)):
        q = normal(g, 2, heads, D, std=std, dtype=BF16)
        got, lse = w4.attn_decode(q, cache, tab, n, scale=scale, return_lse=True)
        check_attention(q, cache, tab, [0, 1, 2], lens, got, lse, scale)
        q = normal(g, 60, heads, D, std=std, dtype=BF16)
        starts = [0, 40, 60]
        got, lse = w4.attn_prompt(q, cache, tab, torch.tensor(starts, dtype=torch.int32, device="cuda"), n,
                                  scale=scale, return_lse=True)
        check_attention(q, cache, tab, starts, lens, got, lse, scale)
    w4.device_status()


def test_attention_strided_queries_and_tables():
    g = gen(19)
    lens, heads, hk, D, page = [50, 200], 8, 2, 128, 16
    cache, tab = scattered(g, lens, hk, page, D, BF16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    wide = normal(g, 2, heads + 4, D, dtype=BF16)
    big = torch.full((2, tab.shape[1] + 9), -1, dtype=torch.int32, device="cuda")
    big[:, 4:4 + tab.shape[1]] = tab
    view = big[:, 4:4 + tab.shape[1]]
    a = w4.attn_decode(wide[:, 2:2 + heads], cache, view, n)
    assert same(a, w4.attn_decode(wide[:, 2:2 + heads].contiguous(), cache, tab, n))
    wide = normal(g, 70, heads + 4, D, dtype=BF16)
    st = torch.tensor([0, 20, 70], dtype=torch.int32, device="cuda")
    a = w4.attn_prompt(wide[:, 2:2 + heads], cache, view, st, n)
    assert same(a, w4.attn_prompt(wide[:, 2:2 + heads].contiguous(), cache, tab, st, n))
    w4.device_status()


def test_attention_out_of_range_data_is_recorded():
    g = gen(20)
    cache, tab = scattered(g, [40, 40], 2, 16, 64, FP16)
    cache.k.zero_(), cache.v.zero_()
    q = normal(g, 2, 4, 64, dtype=FP16)
    st = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    bad = tab.clone()
    bad[1, 0] = cache.k.shape[0]
    for t, lens in ((bad, [40, 40]), (tab, [40, -1]), (tab[:, :2], [20, 40])):
        n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for call in (lambda: w4.attn_decode(q, cache, t, n), lambda: w4.attn_prompt(q, cache, t, st, n)):
            call()
            with pytest.raises(w4.W4A16Error) as e:
                w4.device_status()
            assert e.value.code == -6 and "0x80" in str(e.value)
    w4.device_status()


@pytest.mark.parametrize("dtype", [FP16, E4M3])
def test_offsets_beyond_32_bits(dtype):
    """Pages behind more than 2^32 elements of the cache: appended, then read
    by both attentions."""
    D, hk, page = 128, 8, 128
    pages = (1 << 32) // (D * hk * page) + 4
    g = gen(21)
    scales = [torch.full((hk,), 0.02, device="cuda") for _ in "kv"] if dtype == E4M3 else [None, None]
    k, v = (torch.empty((pages, hk, page, D), dtype=dtype, device="cuda") for _ in "kv")
    cache = w4.KVCache(k, v, *scales)
    n, heads = 200, 16
    tab = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device="cuda")
    at = torch.arange(n, device="cuda")
    slots = tab[0].long()[at // page] * page + at % page
    qkv = normal(g, n, (heads + 2 * hk) * D, dtype=FP16)
    q = w4.rope_append(qkv, table(n, D), at.int(), slots, cache)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    small = w4.KVCache(k[-4:], v[-4:], *scales)
    tab_small = tab - (pages - 4)
    got = w4.attn_prompt(q, cache, tab, torch.tensor([0, n], dtype=torch.int32, device="cuda"), lens)
    check_attention(q, small, tab_small, [0, n], [n], got, None, D ** -0.5)
    got = w4.attn_decode(q[-1:], cache, tab, lens)
    check_attention(q[-1:], small, tab_small, [0, 1], [n], got, None, D ** -0.5)
    w4.device_status()


def test_other_streams():
    """Each operator on a stream that is not the default one, behind slow work
    of the same stream, and given as `stream`."""
    g = gen(22)
    lens, heads, hk, D, page = [400, 65], 8, 2, 128, 16
    cache, tab = scattered(g, lens, hk, page, D, FP16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    src = normal(g, 2, heads, D, dtype=FP16)
    want = w4.attn_decode(src, cache, tab, n)
    w = normal(g, 1024, dtype=FP16)
    want_norm = w4.rms_norm(src.view(2, 1024), w)
    big = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    q = torch.zeros_like(src)
    with torch.cuda.stream(side):
        for _ in range(10):
            big = big @ big * 1e-3
        q.copy_(src)
        got, norm = w4.attn_decode(q, cache, tab, n), w4.rms_norm(q.view(2, 1024), w)
    side.synchronize()
    assert same(got, want) and same(norm, want_norm)
    out = torch.empty_like(src)
    w4.attn_decode(src, cache, tab, n, out=out, stream=side)
    side.synchronize()
    assert same(out, want)
    # results and workspace of a stream that has none yet, behind slow work on
    # the current one (which their zeros must not wait for)
    fresh = torch.cuda.Stream()
    for _ in range(10):
        big = big @ big * 1e-3
    got = w4.attn_decode(src, cache, tab, n, stream=fresh)
    norm = w4.rms_norm(src.view(2, 1024), w, stream=fresh)
    fresh.synchronize()
    assert same(got.clone(), want) and same(norm.clone(), want_norm)
