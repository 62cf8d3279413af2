"""Refusals of the decoder layer's other operators, decided on the host (no
GPU needed): the C ABI's codes and the binding's checks."""
import ctypes
import math

import pytest
import torch

import bit_weight_only_g128_gb300 as w4
from bit_weight_only_g128_gb300 import build as wbuild

# fake device addresses, never dereferenced: each call is refused on the host
P = 0x10000


@pytest.fixture(scope="module")
def lib():
    wbuild.build()
    return w4.lib()


def norm(lib, x=P, ldx=64, r=None, ldr=0, w=P, M=1, K=64, eps=1e-5, flags=0, y=P, codes=None, aq=None, sa=None,
         h=None, ldh=0):
    return lib.w4a16_rms_norm(x, ldx, r, ldr, w, M, K, eps, flags, y, codes, aq, sa, h, ldh, None)


def test_norm_refusals(lib):
    assert norm(lib, M=0) == 0
    for code, bad in [(-1, dict(M=-1)), (-1, dict(K=0)), (-2, dict(K=65537, ldx=65537)), (-2, dict(M=(1 << 20) + 1)),
                      (-1, dict(x=None)), (-1, dict(w=None)), (-1, dict(y=None)), (-1, dict(flags=1)),
                      (-1, dict(flags=0x800)), (-1, dict(eps=-1.0)), (-1, dict(eps=math.nan)),
                      (-1, dict(eps=math.inf)), (-1, dict(ldx=63)), (-1, dict(r=P, ldr=63)),
                      (-1, dict(h=P, ldh=1)), (-1, dict(codes=P)), (-1, dict(aq=P)), (-1, dict(sa=P)),
                      (-3, dict(x=P + 1)), (-3, dict(w=P + 1)), (-3, dict(y=P + 1)), (-3, dict(h=P + 1, ldh=64)),
                      (-3, dict(codes=P, sa=P + 2)), (-3, dict(r=P + 1, ldr=64))]:
        assert norm(lib, **bad) == code, bad
        assert lib.w4a16_last_error()


def rope(lib, qkv=P, ld=768, cs=P, n=10, rot=128, pos=P, slots=P, T=1, heads=4, hk=1, D=128, q=P, k=P, v=P, ks=None,
         vs=None, pages=2, page=16, flags=0):
    return lib.w4a16_rope_append(qkv, ld, cs, n, rot, pos, slots, T, heads, hk, D, q, k, v, ks, vs, pages, page, flags,
                                 None)


CACHE_BAD = [(-1, dict(heads=0)), (-1, dict(hk=0)), (-2, dict(heads=5, hk=2, ld=9 * 128)), (-2, dict(D=96)),
             (-2, dict(D=256)), (-2, dict(page=8)), (-2, dict(page=48)), (-2, dict(page=512)), (-1, dict(page=0)),
             (-1, dict(pages=0)), (-1, dict(k=None)), (-1, dict(v=None)), (-3, dict(k=P + 8)), (-3, dict(v=P + 2)),
             (-1, dict(flags=0x1000)), (-1, dict(flags=0x1000, ks=P)), (-1, dict(ks=P)), (-1, dict(vs=P)),
             (-3, dict(flags=0x1000, ks=P + 2, vs=P)), (-1, dict(flags=0x4000)), (-1, dict(flags=0x100)),
             (-2, dict(heads=2048, hk=2048, ld=6144 * 128))]


def test_rope_append_refusals(lib):
    assert rope(lib, T=0) == 0
    for code, bad in CACHE_BAD + [
            (-1, dict(T=-1)), (-2, dict(T=(1 << 20) + 1)), (-2, dict(rot=0)), (-2, dict(rot=127)), (-2, dict(rot=130)),
            (-1, dict(n=0)), (-1, dict(ld=767)), (-1, dict(qkv=None)), (-1, dict(cs=None)), (-1, dict(pos=None)),
            (-1, dict(slots=None)), (-1, dict(q=None)), (-3, dict(qkv=P + 1)), (-3, dict(q=P + 1)),
            (-3, dict(cs=P + 2)), (-3, dict(pos=P + 2)), (-3, dict(slots=P + 4))]:
        assert rope(lib, **bad) == code, bad
        assert lib.w4a16_last_error()


def decode(lib, q=P, ldq=512, k=P, v=P, ks=None, vs=None, pages=2, page=16, tab=P, ldt=4, most=4, lens=P, B=1, heads=4,
           hk=1, D=128, scale=0.1, out=P, lse=None, flags=0, ld=None):
    return lib.w4a16_attn_decode(q, ldq if ld is None else ld, k, v, ks, vs, pages, page, tab, ldt, most, lens, B, heads,
                                 hk, D, scale, out, lse, None, 0, flags, None)


def prompt(lib, q=P, ldq=512, k=P, v=P, ks=None, vs=None, pages=2, page=16, tab=P, ldt=4, most=4, starts=P, lens=P, T=1,
           B=1, heads=4, hk=1, D=128, scale=0.1, out=P, lse=None, flags=0, ld=None):
    return lib.w4a16_attn_prompt(q, ldq if ld is None else ld, k, v, ks, vs, pages, page, tab, ldt, most, starts, lens, T,
                                 B, heads, hk, D, scale, out, lse, None, 0, flags, None)


@pytest.mark.parametrize("call", [decode, prompt])
def test_attention_refusals(lib, call):
    assert call(lib, B=0) == 0
    for code, bad in CACHE_BAD + [
            (-1, dict(B=-1)), (-2, dict(B=(1 << 20) + 1)), (-1, dict(ldq=511)), (-3, dict(ldq=513)),
            (-1, dict(ldt=3)), (-1, dict(most=-1)), (-2, dict(most=1 << 27, ldt=1 << 27)), (-1, dict(q=None)),
            (-1, dict(tab=None)), (-1, dict(lens=None)), (-1, dict(out=None)), (-3, dict(q=P + 8)),
            (-3, dict(out=P + 2)), (-3, dict(tab=P + 2)), (-3, dict(lens=P + 1)), (-3, dict(lse=P + 2)),
            (-1, dict(scale=math.nan)), (-1, dict(scale=math.inf)), (-1, dict(flags=0x2000))]:
        assert call(lib, **bad) == code, bad
        assert lib.w4a16_last_error()
    if call is prompt:
        assert prompt(lib, T=0) == 0
        assert prompt(lib, T=-1) == -1
        assert prompt(lib, starts=None) == -1
        assert prompt(lib, starts=P + 2) == -3


def test_attention_workspace_size(lib):
    b = ctypes.c_size_t()
    assert lib.w4a16_attn_workspace_size(1, 1, 8, 8, 128, None) == -1
    assert lib.w4a16_attn_workspace_size(-1, 1, 8, 8, 128, ctypes.byref(b)) == -1
    assert lib.w4a16_attn_workspace_size(1, 1, 0, 8, 128, ctypes.byref(b)) == -1
    assert lib.w4a16_attn_workspace_size(0, 0, 8, 8, 128, ctypes.byref(b)) == 0 and b.value == 0


def test_gemm_scaled_refusals(lib):
    def call(A=P, rs=P, M=1, K=128, path=0, ws=None):
        return lib.w4a16_gemm_scaled(A, rs, P, P, P, M, 64, K, 128, P, ws, 0, path, 0, None)
    assert call(rs=None) == -1
    assert call(rs=P + 2) == -3
    assert call(A=None) == -1
    assert call(path=0x800) == -1   # W4A16_ACT_A8 quantizes itself
    assert call(K=100) == -2
    assert call(path=4) == -4       # the stream-K variant's workspace
    assert call(M=0, rs=None) == 0


def test_binding_checks():
    x = torch.zeros((2, 64), dtype=torch.float16)
    w = torch.zeros(64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        w4.rms_norm(x, w)
    with pytest.raises(ValueError, match="float16 or bfloat16"):
        w4.rms_norm(x.float(), w)
    with pytest.raises(ValueError, match=r"\[M, K\]"):
        w4.rms_norm(x[0], w)
    cache = w4.KVCache(torch.zeros((2, 1, 16, 64), dtype=torch.float16), torch.zeros((2, 1, 16, 64), dtype=torch.float16))
    assert cache.nbytes == 2 * 2 * 16 * 64 * 2
    pos, slots = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA tensors"):
        w4.rope_append(torch.zeros((2, 256), dtype=torch.float16), torch.zeros((4, 64)), pos, slots, cache)
    q, tab = torch.zeros((2, 2, 64), dtype=torch.float16), torch.zeros((2, 3), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensors"):
        w4.attn_decode(q, cache, tab, pos)
    cache.k = cache.k.float()
    with pytest.raises(ValueError, match="must be torch.float16 or float8_e4m3fn"):
        w4.attn_decode(q, cache, tab, pos)
    cache.k = cache.k.to(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="needs k_scale"):
        w4.attn_prompt(q, cache, tab, pos, pos)
    cache.k = torch.zeros((2, 1, 32, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="alike"):
        w4.attn_decode(q, cache, tab, pos)
