"""Cases of the decoder layer's other operators beyond test_gpu_layer.py's:
batches of more sequences than one pass over them takes, tiny scales, empty
tables."""
import pytest
import torch

import bit_weight_only_g128_gb300 as w4
from test_gpu_layer import BF16, E4M3, FP16, check_attention, gen, normal, same, scattered

pytestmark = pytest.mark.gpu

TYPES = [(FP16, FP16), (BF16, BF16), (FP16, E4M3), (BF16, E4M3)]


@pytest.mark.parametrize("batch", [129, 300])
@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
def test_decode_of_many_sequences(batch, dtype, cache_dtype):
    g = gen(batch)
    lens = [(37 * b) % 211 for b in range(batch)]
    lens[-1] = 3000
    cache, tab = scattered(g, lens, 2, 16, 128, cache_dtype)
    q = normal(g, batch, 4, 128, std=2, dtype=dtype)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got, lse = w4.attn_decode(q, cache, tab, n, return_lse=True)
    w4.device_status()
    check_attention(q, cache, tab, list(range(batch + 1)), lens, got, lse, 128 ** -0.5)
    assert same(w4.attn_decode(q, cache, tab, n), got)


@pytest.mark.parametrize("batch", [33, 70])
@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
def test_prompts_of_many_sequences(batch, dtype, cache_dtype):
    g = gen(batch)
    new = [(13 * b) % 41 for b in range(batch)]
    lens = [a + (29 * b) % 97 for b, a in enumerate(new)]
    new[batch // 2], lens[batch // 2] = 200, 2500
    cache, tab = scattered(g, lens, 2, 16, 64, cache_dtype)
    starts = [sum(new[:b]) for b in range(batch + 1)]
    q = normal(g, starts[-1], 8, 64, std=2, dtype=dtype)
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for t in (tab, tab[:, : -(-2500 // 16)].contiguous()):
        got, lse = w4.attn_prompt(q, cache, t, st, n, return_lse=True)
        w4.device_status()
        check_attention(q, cache, t, starts, lens, got, lse, 64 ** -0.5)


@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_norm_of_no_rows_answers_as_of_some(dtype):
    w = torch.ones(64, dtype=dtype, device="cuda")
    for rows in (0, 2):
        x, r = (torch.ones((rows, 64), dtype=dtype, device="cuda") for _ in range(2))
        y, h = w4.rms_norm(x, w, residual=r)
        assert y.shape == h.shape == (rows, 64)
        for quant, code in (("int8", torch.int8), ("codes", dtype)):
            q, s = w4.rms_norm(x, w, quant=quant)
            assert q.shape == (rows, 64) and q.dtype == code and s.shape == (rows,)
            q, s, h = w4.rms_norm(x, w, residual=r, quant=quant)
            assert q.shape == h.shape == (rows, 64) and s.shape == (rows,)


def nearest_codes(v):
    """Codes and scales of rows v (float32) by the rule, in IEEE fp32 on the
    host: s = max / 127 (1 where that is zero), clamp(round(v / s))."""
    v = v.cpu()
    s = v.abs().amax(1) / 127
    s = torch.where(s > 0, s, torch.ones_like(s))
    return (v / s[:, None]).round().clamp(-127, 127), s


# 1 over the scale leaves fp32 below 3.7e-37, the scale has few bits below 1e-36, bf16 ends at 9.2e-41
TINY = [1e-30, 4e-37, 3.7e-37, 1e-37, 1e-38, 1e-39, 1e-43, 1e-45]


@pytest.mark.parametrize("size", TINY)
def test_codes_of_tiny_activations(size):
    x = (torch.randn((5, 96), generator=gen(1), device="cuda").double() * size).to(BF16)
    x[:, ::3] = 0
    x[4] = 0
    aq, s = w4.quantize_act(x)
    want, scale = nearest_codes(x.float())
    assert torch.equal(s.cpu(), scale) and torch.equal(aq.cpu().float(), want)


@pytest.mark.parametrize("K", [96, 97, 4096])
@pytest.mark.parametrize("size", TINY)
def test_norm_codes_of_tiny_results(size, K):
    """Powers of two and rows of one magnitude: y is exact, so the codes are
    those of the rule."""
    x = torch.zeros((3, K), dtype=BF16, device="cuda")
    x[0, ::2], x[1, 1::2] = 1, -1
    w = torch.full((K,), size, dtype=BF16, device="cuda")
    y = w4.rms_norm(x, w, eps=0.5 - 0.25 * (K % 2)).float()
    codes, s = w4.rms_norm(x, w, eps=0.5 - 0.25 * (K % 2), quant="codes")
    aq, s2 = w4.rms_norm(x, w, eps=0.5 - 0.25 * (K % 2), quant="int8")
    assert torch.equal(codes.float(), aq.float()) and torch.equal(s, s2)
    assert not aq[x == 0].any() and float(s[2]) == 1.0
    if y.abs().amax() / 127 > 2.0 ** -140:  # (the scale has bits enough to tell)
        assert (aq[0, ::2] == 127).all() and (aq[1, 1::2] == -127).all()


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("k_scale", [0.02, 1e-20])
@pytest.mark.parametrize("scale", [0.0, 1e-30, 1e-7, 0.125])
def test_scores_too_small_for_their_factor(scale, k_scale, dtype):
    """Queries of zero, or of ordinary size under tiny scales, over e4m3 keys:
    the mean of the values, whatever the masked places held."""
    lens, heads, hk = [300, 1, 33, 700], 8, 2
    g = gen(35)
    cache, tab = scattered(g, lens, hk, 16, 64, E4M3)
    cache.k_scale.fill_(k_scale)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for std in (0.0, 1.0):
        q = normal(g, 4, heads, 64, std=std, dtype=dtype)
        q[0] = 0
        got, lse = w4.attn_decode(q, cache, tab, n, scale=scale, return_lse=True)
        check_attention(q, cache, tab, [0, 1, 2, 3, 4], lens, got, lse, scale)
        starts = [0, 100, 101, 134, 150]
        q = normal(g, 150, heads, 64, std=std, dtype=dtype)
        got, lse = w4.attn_prompt(q, cache, tab, torch.tensor(starts, dtype=torch.int32, device="cuda"), n,
                                  scale=scale, return_lse=True)
        check_attention(q, cache, tab, starts, lens, got, lse, scale)
    w4.device_status()


def test_sequences_of_no_pages():
    """Tables of no columns, as a server's first step of empty slots has them,
    and a prompt call of no sequences."""
    g = gen(36)
    cache, _ = scattered(g, [20], 2, 16, 64, FP16)
    n = torch.zeros(3, dtype=torch.int32, device="cuda")
    tab = torch.empty((3, 0), dtype=torch.int32, device="cuda")
    got, lse = w4.attn_decode(normal(g, 3, 8, 64, dtype=FP16), cache, tab, n, return_lse=True)
    assert not got.any() and lse.isneginf().all()
    st = torch.tensor([0, 2, 2, 5], dtype=torch.int32, device="cuda")
    q = normal(g, 5, 8, 64, dtype=FP16)
    got, lse = w4.attn_prompt(q, cache, tab, st, n, return_lse=True)
    assert not got.any() and lse.isneginf().all()
    out = torch.full_like(q, 3.0)
    assert w4.attn_prompt(q, cache, tab[:0], st[:1], n[:0], out=out) is out
    assert (out == 3).all()
    assert w4.attn_decode(q[:0], cache, tab[:0], n[:0]).shape == (0, 8, 64)
    w4.device_status()
