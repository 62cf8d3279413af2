"""Attention with NaN and infinities inside a sequence, against the
definition in 64 bits: a row that sees a NaN or +inf score is NaN, a key of
score -inf has no weight, a non-finite value reaches the rows that see it."""
import math

import pytest
import torch

import bit_weight_only_g128_gb300 as w4
import layer_ref as ref
from test_gpu_layer import BF16, E4M3, FP16, gen, normal, scattered

pytestmark = pytest.mark.gpu

TYPES = [(FP16, FP16), (BF16, BF16), (FP16, E4M3), (BF16, E4M3)]


def definition(q, k, v, first, scale, u):
    """q [rows, D], k and v [n, D] in 64 bits, row i seeing keys 0 .. first + i.
    Returns out and lse of the finite part of v with the rows of a NaN or +inf
    score NaN, `touched` [rows, D] (a seen key has a non-finite value there),
    and the error bounds of layer_ref.attention."""
    n = len(k)
    seen = torch.arange(n, device=q.device)[None] <= first + torch.arange(len(q), device=q.device)[:, None]
    s = q @ k.T * scale
    bad = ((s.isnan() | (s == math.inf)) & seen).any(1)
    s = s.masked_fill(~seen | ~torch.isfinite(s), -math.inf)
    top = s.amax(1, keepdim=True)
    p = (s - torch.where(top > -math.inf, top, 0)).exp()
    total = p.sum(1, keepdim=True)
    w = p / torch.where(total > 0, total, 1)
    whole = torch.where(torch.isfinite(v), v, 0)
    out, lse = w @ whole, torch.where(total > 0, top + total.log(), -math.inf)[:, 0]
    touched = (w > 0).double() @ (~torch.isfinite(v)).double() > 0
    fq, fk = torch.where(torch.isfinite(q), q, 0), torch.where(torch.isfinite(k), k, 0)
    delta = (q.shape[1] + 16) * ref.E32 * (fq.abs() @ fk.abs().T * abs(scale)).masked_fill(~seen, 0).amax(1, keepdim=True)
    rel = 2 * delta + 2.0 ** -20 + n * ref.E32
    tol = (rel + u) * (w @ whole.abs()) + seen.sum(1, keepdim=True) * 2.0 ** -24 * whole.abs().amax()
    out[bad], lse[bad] = math.nan, math.nan
    return out, lse, touched, tol, (rel + 4 * ref.E32 * lse[:, None].abs().nan_to_num(0, 0, 0))[:, 0]


def check(q, cache, tab, starts, lens, got, lse, values):
    """Every row against the definition; with `values` (non-finite values in
    the cache) only rows that see one, and rows of other key/value heads."""
    D, heads, hk = q.shape[2], q.shape[1], cache.k.shape[1]
    counts = dict(nan=0, finite=0, touched=0)
    for b, n in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        k = ref.cached(cache.k, cache.k_scale, tab[b], n)
        v = ref.cached(cache.v, cache.v_scale, tab[b], n)
        u = ref.U[q.dtype] if cache.k.dtype != E4M3 else ref.U[FP16]
        for h in range(heads):
            kv = h * hk // heads
            out, l, touched, tol, tol_l = definition(q[lo:hi, h].double(), k[kv], v[kv], n - (hi - lo), D ** -0.5, u)
            y, z = got[lo:hi, h], lse[lo:hi, h]
            nan = l.isnan()
            assert y[nan].isnan().all() and not (torch.isfinite(z[nan]) | z[nan].isneginf()).any(), (b, h)
            assert not torch.isfinite(y[touched]).any(), (b, h)
            clean = ~nan & ~touched.any(1)
            if values and not torch.isfinite(v[kv]).all():
                clean &= False
            ref.within(y[clean], out[clean], tol[clean])
            some = torch.isfinite(l)
            assert torch.equal(z.isneginf(), l.isneginf())
            ref.within(z[some], l[some], tol_l[some])
            counts["nan"] += int(nan.sum())
            counts["finite"] += int(clean.sum())
            counts["touched"] += int(touched.any(1).sum())
    return counts


def place(cache, tab, b, token):
    return tab[b].long()[token // cache.k.shape[2]], token % cache.k.shape[2]


def put(cache, tab, b, token, head, dim, keys, value):
    t = cache.k if keys else cache.v
    page, at = place(cache, tab, b, token)
    if t.dtype == E4M3:
        t.view(torch.uint8)[page, head, at, dim] = 0x7F  # its only non-finite code: NaN
    else:
        t[page, head, at, dim] = value


SEQS = {
    "whole": [(100, 300), (1, 1), (150, 150)],
    "split": [(16, 9000), (3, 1500)],
    "group": [(40, 500), (129, 129)],
}


@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
@pytest.mark.parametrize("seqs,heads,hk,D", [("whole", 8, 2, 128), ("split", 16, 2, 128), ("group", 5, 1, 64)])
@pytest.mark.parametrize("where", ["query", "key", "value"])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_prompt(seqs, heads, hk, D, where, value, dtype, cache_dtype):
    seqs = SEQS[seqs]
    new, lens = [a for a, _ in seqs], [n for _, n in seqs]
    g = gen(sum(lens) + heads)
    cache, tab = scattered(g, lens, hk, 16, D, cache_dtype)
    starts = [sum(new[:b]) for b in range(len(new) + 1)]
    q = normal(g, starts[-1], heads, D, std=2, dtype=dtype)
    if where == "query":
        q[starts[0] + 3, 1, 5] = value
        q[starts[-1] - 1, heads - 1, 0] = value
    else:  # a cached key, and one among the new ones
        put(cache, tab, 0, 7, 0, 3, where == "key", value)
        put(cache, tab, len(lens) - 1, lens[-1] - 2, hk - 1, D - 1, where == "key", value)
    got, lse = w4.attn_prompt(q, cache, tab, torch.tensor(starts, dtype=torch.int32, device="cuda"),
                              torch.tensor(lens, dtype=torch.int32, device="cuda"), return_lse=True)
    w4.device_status()
    counts = check(q, cache, tab, starts, lens, got, lse, where == "value")
    assert counts["touched" if where == "value" else "nan"] > 0 and (counts["finite"] > 0 or hk == 1)


@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
@pytest.mark.parametrize("heads,hk,D", [(8, 2, 128), (32, 2, 64), (1, 1, 128)])
@pytest.mark.parametrize("where,value", [("query", math.nan), ("query", math.inf), ("key", math.nan),
                                         ("key", math.inf), ("value", math.nan), ("value", math.inf)])
def test_decode(heads, hk, D, where, value, dtype, cache_dtype):
    lens = [300, 1, 9000, 33]
    g = gen(sum(lens) + heads)
    cache, tab = scattered(g, lens, hk, 16, D, cache_dtype)
    q = normal(g, len(lens), heads, D, std=2, dtype=dtype)
    if where == "query":
        q[0, 0, 5] = value
        q[2, heads - 1, 0] = value
    else:
        put(cache, tab, 0, 299, 0, 3, where == "key", value)
        put(cache, tab, 1, 0, hk - 1, 0, where == "key", value)
        put(cache, tab, 2, 5000, 0, D - 1, where == "key", value)
    got, lse = w4.attn_decode(q, cache, tab, torch.tensor(lens, dtype=torch.int32, device="cuda"), return_lse=True)
    w4.device_status()
    counts = check(q, cache, tab, list(range(len(lens) + 1)), lens, got, lse, where == "value")
    assert counts["touched" if where == "value" else "nan"] > 0 and counts["finite"] > 0


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("decode", [True, False])
def test_tiles_of_scores_without_weight(decode, D, dtype):
    """The first 256 keys all score -inf, as do all keys of a short sequence:
    the others decide, and a row of nothing else is as an empty one."""
    lens, heads, hk = [300, 20, 2000], 8, 2
    new = [1, 1, 1] if decode else [9, 3, 40]
    g = gen(D)
    cache, tab = scattered(g, lens, hk, 16, D, dtype)
    for b, n in enumerate(lens):
        for t in range(min(n, 256)):
            page, at = place(cache, tab, b, t)
            cache.k[page, :, at, 2] = math.inf
    starts = [sum(new[:b]) for b in range(4)]
    q = normal(g, starts[-1], heads, D, std=2, dtype=dtype)
    q[:, :, 2] = -q[:, :, 2].abs() - 0.5
    q[0, 0, 2] = 1.0  # and a head that those keys score +inf for
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if decode:
        got, lse = w4.attn_decode(q, cache, tab, n, return_lse=True)
    else:
        got, lse = w4.attn_prompt(q, cache, tab, torch.tensor(starts, dtype=torch.int32, device="cuda"), n,
                                  return_lse=True)
    w4.device_status()
    counts = check(q, cache, tab, starts, lens, got, lse, False)
    assert counts["nan"] == 1 and counts["finite"] == starts[-1] * heads - 1
    rows = slice(starts[1], starts[2])
    assert not got[rows].any() and lse[rows].isneginf().all()
