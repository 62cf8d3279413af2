"""The decoder layer's other operators from their definitions in 64 bits
(norm, rotation and cache append, attention over a paged cache), and bounds on
how far 32-bit kernels with 16-bit products may be from them."""
import math

import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}   # half a unit in the last place
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -130}  # half the smallest subnormal
E32 = 2.0 ** -24
E4M3 = torch.float8_e4m3fn


def rms_norm(x, weight, residual=None, eps=1e-5):
    h = x.double() if residual is None else x.double() + residual.double()
    return h * (h.square().mean(1, keepdim=True) + eps).rsqrt() * weight.double(), h


def norm_rel(K):
    """Relative error of the fp32 y: the sum of squares adds at most K/256
    terms one after another and then a tree; a few roundings follow."""
    return (K / 256 + 40) * E32


def rope(x, cos_sin, positions, interleaved):
    """x [T, heads, D] in 64 bits with its first rotary dimensions turned."""
    x = x.double().clone()
    rot = cos_sin.shape[1]
    half = rot // 2
    turn = cos_sin.double()[positions.long()]
    for i in range(half):
        i0, i1 = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        a, b = x[:, :, i0].clone(), x[:, :, i1].clone()
        c, s = turn[:, i, None], turn[:, half + i, None]
        x[:, :, i0], x[:, :, i1] = a * c - b * s, b * c + a * s
    return x


def cached(cache, scale, table_row, n):
    """[kv heads, n, D] of a sequence's cached values in 64 bits."""
    page = cache.shape[2]
    pages = table_row[: -(-n // page)].long()
    x = cache.view(torch.uint8)[pages].view(E4M3) if cache.dtype == E4M3 else cache[pages]
    x = x.double().transpose(0, 1).reshape(cache.shape[1], -1, cache.shape[3])[:, :n]
    return x if scale is None else x * scale.double()[:, None, None]


def attention(q, cache, table_row, n, scale, first):
    """q [rows, heads, D] of one sequence with n cached tokens, row i seeing
    the keys 0 .. first + i. Returns out, lse and the bounds of their errors
    (before the 16-bit rounding of out)."""
    rows, heads, D = q.shape
    hk = cache.k.shape[1]
    out = torch.zeros((rows, heads, D), dtype=torch.float64, device=q.device)
    lse = torch.full((rows, heads), -math.inf, dtype=torch.float64, device=q.device)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    if n <= 0:
        return out, lse, tol, tol_lse
    k, v = cached(cache.k, cache.k_scale, table_row, n), cached(cache.v, cache.v_scale, table_row, n)
    seen = torch.arange(n, device=q.device)[None] <= first + torch.arange(rows, device=q.device)[:, None]
    u = U[q.dtype] if cache.k.dtype != E4M3 else U[torch.float16]
    for h in range(heads):
        kh, vh, qh = k[h // (heads // hk)], v[h // (heads // hk)], q[:, h].double()
        s = (qh @ kh.T * scale).masked_fill(~seen, -math.inf)
        top = s.amax(1, keepdim=True)
        p = torch.where(seen, (s - torch.where(top > -math.inf, top, 0)).exp(), 0)
        total = p.sum(1, keepdim=True)
        some = total > 0
        w = torch.where(some, p / torch.where(some, total, 1), 0)
        out[:, h] = w @ vh
        lse[:, h] = torch.where(some, top + total.log(), -math.inf)[:, 0]
        # the scores' error: D products added in fp32, and a few roundings of
        # the exponent; then the exponential (2 ulps) and its 16-bit rounding
        # (relative, or half the smallest subnormal against a maximum of 1),
        # and n additions in fp32
        delta = (D + 16) * E32 * (qh.abs() @ kh.abs().T * abs(scale)).masked_fill(~seen, 0).amax(1, keepdim=True)
        rel = 2 * delta + 2.0 ** -20 + n * E32
        tol[:, h] = (rel + u) * (w @ vh.abs()) + (seen.sum(1, keepdim=True) * 2.0 ** -24) * vh.abs().amax()
        tol_lse[:, h] = (rel + 4 * E32 * lse[:, h:h + 1].abs().nan_to_num(0, 0, 0))[:, 0]
    return out, lse, tol, tol_lse


def within(got, want, tol):
    """got (16-bit or fp32) is within tol of want, and its own rounding."""
    u, tiny = (U[got.dtype], TINY[got.dtype]) if got.dtype in U else (E32, 0.0)
    err = (got.double() - want).abs()
    bound = tol + u * (want.abs() + tol) + tiny
    bad = ~(err <= bound)
    if want.numel() and bad.any():
        i = int(torch.where(bad, (err / bound).nan_to_num(1e30), torch.zeros_like(err)).argmax())
        raise AssertionError(f"{int(bad.sum())} of {want.numel()} outside the bound; worst at {i}: got "
                             f"{float(got.reshape(-1)[i])}, want {float(want.reshape(-1)[i])}, "
                             f"bound {float(bound.reshape(-1)[i])}")
