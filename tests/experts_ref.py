"""A layer of experts from its definitions in 64 bits (router, products
grouped by expert), and bounds on how far 32-bit kernels may be from them."""
import math

import torch

import bit_weight_only_g128_gb300 as w4
from layer_ref import E32, U


def route(logits, top, scoring, renormalize):
    """experts, weights (64 bits), rows and offsets, and the bound of the
    weights' errors."""
    x = logits.double()
    T, E = x.shape
    best, experts = torch.sort(x, dim=1, descending=True, stable=True)  # equal ones: the lower index first
    best, experts = best[:, :top], experts[:, :top].clone()
    none = best == -math.inf
    if scoring == "softmax":
        m = best[:, :1].masked_fill(none[:, :1], 0)
        score, all_ = (best - m).exp(), (x - m).exp().sum(1, keepdim=True)
        far = (m - best).masked_fill(none, 0)
    else:
        score, all_ = torch.sigmoid(best), torch.ones_like(best[:, :1])
        far = torch.zeros_like(best)
    total = score.sum(1, keepdim=True) if renormalize else all_
    weights = (score / torch.where(total == 0, 1.0, total)).masked_fill(none, 0)
    experts[none] = -1
    flat = experts.flatten()
    rows = torch.sort(torch.where(flat < 0, E, flat), stable=True)[1]
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=x.device)
    offsets[1:] = (flat[:, None] == torch.arange(E, device=x.device)).sum(0).cumsum(0)
    # the argument's rounding (far, in fp32), 2 ulps of the exponential, at
    # most E additions, sums of terms as far off (t e^-t is below 1), a division
    rel = (far + E + 12) * E32
    # fp32 underflow: an exponential below the smallest normal number
    return experts.int(), weights, rows.int(), offsets.int(), rel * weights.abs() + 2.0 ** -126


def weights_of(pe):
    """[experts, K, N] of (q - z) s in 64 bits."""
    out = []
    for e in range(pe.experts):
        q, s, z = w4.unpack(pe.expert(e))
        rep = lambda t: t.double().repeat_interleave(pe.group, 0)  # noqa: E731
        out.append((q.double() - rep(z)) * rep(s))
    return torch.stack(out)


def terms_of(pe, dtype):
    """[experts, K, N]: what the path for few rows adds up for a weight, in
    magnitude. Where an expert has up to 8 rows it does not subtract the zero
    point from the code but its product from the code's: (c + q) s and (c + z) s
    with c = 0, in bf16 128 (the form that the codes have there)."""
    c = 128 if dtype == torch.bfloat16 else 0
    out = []
    for e in range(pe.experts):
        q, s, z = w4.unpack(pe.expert(e))
        rep = lambda t: t.double().repeat_interleave(pe.group, 0)  # noqa: E731
        out.append((2 * c + q.double() + rep(z)) * rep(s))
    return torch.stack(out)


def products(A, W, experts, weight_error=0.0, terms=None):
    """y [T, top, N] in 64 bits with zeros for choices of no expert, and the
    bound of its error before the result's rounding: K additions in fp32 of
    `terms` (default: the weights, in magnitude), and `weight_error` relative in
    each weight."""
    T, top = experts.shape
    E, K, N = W.shape
    a = (A if A.dim() == 3 else A[:, None].expand(T, top, K)).double()
    y = torch.zeros((T, top, N), dtype=torch.float64, device=A.device)
    tol = torch.zeros_like(y)
    for e in range(E):
        t, j = torch.nonzero(experts == e, as_tuple=True)
        if len(t):
            y[t, j] = a[t, j] @ W[e]
            mag = a[t, j].abs() @ W[e].abs()
            added = mag if terms is None else a[t, j].abs() @ terms[e]
            tol[t, j] = (K + 8) * E32 * added + weight_error * mag
    return y, tol


def silu_mul(y, tol):
    n = y.shape[-1] // 2
    g, u, tg, tu = y[..., :n], y[..., n:], tol[..., :n], tol[..., n:]
    silu = g * torch.sigmoid(g)
    # |silu'| <= 1.1 carries the gate's error; the exponential is off by
    # 2 + |g| ulps, and a few roundings follow
    return silu * u, 1.1 * tg * (u.abs() + tu) + silu.abs() * (tu + (16 + 2 * g.abs()) * E32 * u.abs())


def combine(y, tol, weights, experts, each=0.0):
    """The weighted sums and their bound; `each`: a relative rounding of every
    weighted product."""
    w = torch.where(experts < 0, 0.0, weights.double())[..., None]
    top = experts.shape[1]
    return (w * y).sum(1), (w.abs() * (tol + (each + (top + 2) * E32) * (y.abs() + tol))).sum(1)


WEIGHT_ERROR = U  # of a weight rounded to the activations' type
