"""Norms of query and key heads in the pass that rotates and appends them,
against the definition in 64 bits."""
import math

import pytest
import torch

import bit_weight_only_g128_gb300 as w4
import layer_ref as ref
from test_gpu_layer import BF16, E4M3, FP16, gen, new_cache, normal, table

pytestmark = pytest.mark.gpu


def normed(x, heads, hk, q_norm, k_norm, eps):
    """x [T, heads + 2 hk, D] in 64 bits with its query and key heads normed."""
    x = x.double().clone()
    for at, w in ((slice(0, heads), q_norm), (slice(heads, heads + hk), k_norm)):
        if w is not None:
            x[:, at] = x[:, at] * (x[:, at].square().mean(2, keepdim=True) + eps).rsqrt() * w.double()
    return x


def check(qkv, cs, pos, slots, cache, heads, hk, q_norm, k_norm, eps, interleaved):
    T, D = len(qkv), cache.k.shape[3]
    q = w4.rope_append(qkv, cs, pos, slots, cache, interleaved=interleaved, q_norm=q_norm, k_norm=k_norm, eps=eps)
    x = normed(qkv.reshape(T, heads + 2 * hk, D), heads, hk, q_norm, k_norm, eps)
    want = ref.rope(x[:, :heads + hk], cs, pos, interleaved)
    # D squares added, the root, two products; then two products and a sum
    mag = x[:, :heads + hk].abs().amax(2, keepdim=True) * 2 * (D + 16) * ref.E32
    ref.within(q, want[:, :heads], mag[:, :heads].expand(-1, -1, D))
    pages, page = cache.k.shape[0], cache.k.shape[2]
    keep = slots >= 0
    used = torch.zeros(pages * page, dtype=torch.bool, device="cuda")
    used[slots[keep]] = True
    for t, scale, new, m in ((cache.k, cache.k_scale, want[:, heads:], mag[:, heads:]),
                             (cache.v, cache.v_scale, x[:, heads + hk:], None)):
        flat = t.view(torch.uint8).view(pages, hk, page, -1).transpose(1, 2).reshape(pages * page, hk, -1)
        assert (flat[~used] == 0xFF).all(), "a slot that was not named was written"
        got = flat[slots[keep]].contiguous().view(t.dtype)
        new = new[keep]
        m = torch.zeros_like(new) if m is None else m[keep].expand_as(new)
        if scale is None:
            ref.within(got, new, m)
        else:
            z = (new / scale.double()[:, None]).clamp(-448, 448)
            near = z.float().to(E4M3).double()
            # the nearest code; next to a midpoint of two codes either of them
            slack = 8 * ref.E32 * z.abs() + 2 * m / scale.double()[:, None]
            assert ((got.double() - z).abs() <= (near - z).abs() + slack).all()
    w4.device_status()
    return q


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,cache_dtype", [(FP16, FP16), (BF16, BF16), (FP16, E4M3), (BF16, E4M3)])
@pytest.mark.parametrize("T,heads,hk,D,rot,page", [
    (1, 32, 32, 128, 128, 16), (1, 1, 1, 64, 64, 16), (17, 8, 1, 128, 64, 32), (130, 5, 5, 64, 32, 64),
    (3, 64, 8, 128, 128, 256), (9, 10, 2, 128, 30, 128), (6, 4, 2, 64, 2, 16), (301, 16, 2, 128, 128, 16)])
def test_rope_append_with_norms(T, heads, hk, D, rot, page, dtype, cache_dtype, interleaved):
    g = gen(T + heads * 3 + rot)
    pages = -(-T // page) + 3
    qkv = normal(g, T, (heads + 2 * hk) * D, std=2, dtype=dtype)
    qkv[:, ::50] *= 20
    qn, kn = ((1 + normal(g, D, std=0.2)).to(dtype) for _ in "qk")
    cs = table(2000, rot)
    pos = torch.randint(0, 2000, (T,), generator=g, device="cuda", dtype=torch.int32)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
    if T > 4:
        slots[2] = -1
        slots[4] = -7
    for a, b, eps in ((qn, kn, 1e-6), (qn, None, 1e-5), (None, kn, 0.0)):
        check(qkv, cs, pos, slots, new_cache(g, pages, hk, page, D, cache_dtype, fill="nan"), heads, hk, a, b, eps, interleaved)


def test_alignment_strides_and_streams():
    g = gen(5)
    T, heads, hk, D, page = 7, 4, 2, 128, 16
    cols = (heads + 2 * hk) * D
    wide = normal(g, T, cols + 40, dtype=FP16)
    weights = normal(g, D + 8, dtype=FP16)
    cs, pos = table(50, D), torch.arange(T, device="cuda", dtype=torch.int32)
    slots = torch.arange(T, device="cuda")
    for lo in (0, 8, 3):      # rows
        for w in (0, 1):      # weights
            check(wide[:, lo:lo + cols], cs, pos, slots, new_cache(g, 2, hk, page, D, FP16, fill="nan"), heads, hk,
                  weights[w:w + D], weights[8 - w:8 - w + D], 1e-5, False)
    side = torch.cuda.Stream()
    a, b = new_cache(g, 2, hk, page, D, FP16), new_cache(g, 2, hk, page, D, FP16)
    side.wait_stream(torch.cuda.current_stream())
    one = w4.rope_append(wide[:, :cols], cs, pos, slots, a, q_norm=weights[:D], k_norm=weights[8:], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    two = w4.rope_append(wide[:, :cols], cs, pos, slots, b, q_norm=weights[:D], k_norm=weights[8:])
    assert torch.equal(one, two) and torch.equal(a.k, b.k) and torch.equal(a.v, b.v)


def test_rows_of_zeros_and_extremes():
    g = gen(8)
    heads, hk, D = 2, 1, 64
    cs, pos = table(50, D), torch.zeros(4, device="cuda", dtype=torch.int32)
    slots = torch.arange(4, device="cuda")
    w = torch.ones(D, dtype=FP16, device="cuda")
    qkv = normal(g, 4, 4 * D, dtype=FP16)
    qkv[0] = 0
    qkv[1] = 65504.0
    qkv[2] = 2.0 ** -24
    cache = new_cache(g, 1, hk, 16, D, FP16)
    q = w4.rope_append(qkv, cs, pos, slots, cache, q_norm=w, k_norm=w, eps=1e-6)
    assert not q[0].any() and not cache.k[0, :, 0].any()
    assert (q[1] == 1).all() and (cache.k[0, :, 1] == 1).all() and (cache.v[0, :, 1] == 65504).all()
    want = 2.0 ** -24 / math.sqrt(2.0 ** -48 + 1e-6)
    assert (q[2].double() - want).abs().max() <= want * 2.0 ** -11 + 2.0 ** -25
    qkv[3, D + 3] = math.nan  # one head's NaN stays in it
    q = w4.rope_append(qkv, cs, pos, slots, cache, q_norm=w, k_norm=w)
    assert q[3, 0].isfinite().all() and q[3, 1].isnan().all() and cache.k[0, :, 3].isfinite().all()
