"""Refusals of the router, the products grouped by expert and the norms of
query and key heads, decided on the host (no GPU needed)."""
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


def route(lib, x=P, ld=8, T=4, E=8, k=2, e=P, w=P, r=P, o=P, ws=None, n=0, flags=0):
    return lib.w4a16_route(x, ld, T, E, k, e, w, r, o, ws, n, flags, None)


def test_route_refusals(lib):
    for code, bad in [(-1, dict(T=-1)), (-1, dict(E=0)), (-1, dict(k=0)), (-2, dict(T=(1 << 20) + 1)), (-2, dict(E=513, ld=513)),
                      (-2, dict(k=9)), (-2, dict(k=33, E=64, ld=64)), (-1, dict(ld=7)), (-1, dict(x=None)), (-1, dict(e=None)),
                      (-1, dict(w=None)), (-1, dict(r=None)), (-1, dict(o=None)), (-1, dict(T=0, o=None)), (-1, dict(flags=1)),
                      (-1, dict(flags=0x4400)), (-1, dict(flags=0x200)), (-3, dict(x=P + 1)), (-3, dict(x=P + 2, flags=0x4000)),
                      (-3, dict(e=P + 2)), (-3, dict(w=P + 1)), (-3, dict(r=P + 2)), (-3, dict(o=P + 2)),
                      (-4, dict(T=1000)), (-4, dict(T=1000, ws=P, n=100)), (-3, dict(T=1000, ws=P + 16, n=1 << 20))]:
        assert route(lib, **bad) == code, bad
        assert lib.w4a16_last_error()
    b = ctypes.c_size_t()
    assert lib.w4a16_route_workspace_size(4, 8, 2, None) == -1
    assert lib.w4a16_route_workspace_size(4, 8, 9, ctypes.byref(b)) == -2
    assert lib.w4a16_route_workspace_size(64, 8, 2, ctypes.byref(b)) == 0 and b.value == 0
    assert lib.w4a16_route_workspace_size(1000, 8, 2, ctypes.byref(b)) == 0 and b.value > w4.FLAG_BYTES


def product(lib, A=P, q=P, s=P, z=P, T=4, k=2, E=8, N=64, K=128, group=128, e=P, w=P, r=P, o=P, Y=P, ws=None, n=0, flags=0):
    return lib.w4a16_gemm_experts(A, q, s, z, T, k, E, N, K, group, e, w, r, o, Y, ws, n, flags, None)


def test_gemm_experts_refusals(lib):
    assert product(lib, T=0) == 0
    combine, silu = w4.EXPERTS_COMBINE, w4.SILU_MUL
    for code, bad in [(-1, dict(T=-1)), (-2, dict(E=513)), (-2, dict(k=9)), (-2, dict(T=(1 << 20) + 1)), (-1, dict(N=0)),
                      (-1, dict(K=0)), (-1, dict(group=0)), (-2, dict(N=8)), (-2, dict(K=96)), (-2, dict(group=32)),
                      (-2, dict(K=192)), (-2, dict(N=1 << 21)), (-2, dict(K=1 << 21)), (-2, dict(N=16, flags=silu)),
                      (-2, dict(E=512, N=1 << 20, K=64, group=64, k=1) | dict(N=(1 << 20) + 16)),
                      (-1, dict(flags=silu | combine)), (-1, dict(flags=0x800)), (-1, dict(flags=0x100)), (-1, dict(flags=2)),
                      (-1, dict(flags=9)), (-1, dict(A=None)), (-1, dict(q=None)), (-1, dict(s=None)), (-1, dict(z=None)),
                      (-1, dict(e=None)), (-1, dict(r=None)), (-1, dict(o=None)), (-1, dict(Y=None)),
                      (-1, dict(w=None, flags=combine)), (-3, dict(A=P + 8)), (-3, dict(q=P + 8)), (-3, dict(s=P + 2)),
                      (-3, dict(z=P + 4)), (-3, dict(Y=P + 2)), (-3, dict(e=P + 2)), (-3, dict(w=P + 2)), (-3, dict(r=P + 2)),
                      (-3, dict(o=P + 2)), (-4, dict(flags=combine)), (-4, dict(flags=combine, ws=P, n=32768)),
                      (-3, dict(flags=combine, ws=P + 16, n=1 << 20))]:
        assert product(lib, **bad) == code, bad
        assert lib.w4a16_last_error()
    b = ctypes.c_size_t()
    assert lib.w4a16_experts_workspace_size(4, 2, 8, 64, 128, 128, combine, None) == -1
    assert lib.w4a16_experts_workspace_size(4, 2, 8, 60, 128, 128, 0, ctypes.byref(b)) == -2
    assert lib.w4a16_experts_workspace_size(0, 2, 8, 64, 128, 128, combine, ctypes.byref(b)) == 0 and b.value == 0


def test_rope_append_norm_refusals(lib):
    def rope(qn=P, kn=P, eps=1e-5, T=1, flags=0):
        return lib.w4a16_rope_append_norm(P, 768, P, 10, 128, P, P, T, 4, 1, 128, P, P, P, None, None, 2, 16, qn, kn, eps, flags, None)
    assert rope(T=0) == 0
    for code, bad in [(-1, dict(eps=-1.0)), (-1, dict(eps=math.nan)), (-1, dict(eps=math.inf)), (-3, dict(qn=P + 1)),
                      (-3, dict(kn=P + 1)), (-1, dict(flags=0x4000))]:
        assert rope(**bad) == code, bad


def test_binding_refusals(lib):
    x = torch.zeros((4, 8))
    with pytest.raises(ValueError, match="CUDA tensor"):
        w4.route(x, 2)
    with pytest.raises(ValueError, match="float32"):
        w4.route(x.double(), 2)
    with pytest.raises(ValueError, match="tensor"):
        w4.route([1.0], 2)
    pe = w4.PackedExperts(*(torch.zeros(n, dtype=t) for n, t in ((8 * 1024, torch.int32), (512, torch.float16), (64, torch.int32))),
                          8, 128, 64, 128)
    assert pe.nbytes == 8 * 1024 * 4 + 512 * 2 + 64 * 4
    assert pe.expert(3).Wq.data_ptr() == pe.Wq.data_ptr() + 3 * 4096 and pe.expert(7).nbytes * 8 == pe.nbytes
    with pytest.raises(IndexError):
        pe.expert(8)
    none = w4.Routing(*(torch.zeros(s, dtype=t) for s, t in (((4, 2), torch.int32), ((4, 2), torch.float32), (8, torch.int32), (9, torch.int32))))
    with pytest.raises(ValueError, match="CUDA tensor"):
        w4.gemm_experts(torch.zeros((4, 128), dtype=torch.float16), pe, none)
    with pytest.raises(ValueError, match="float16 or bfloat16"):
        w4.gemm_experts(torch.zeros((4, 128)), pe, none)
    with pytest.raises(KeyError):
        w4.gemm_experts(torch.zeros((4, 128), dtype=torch.float16), pe, none, path="nowhere")


def test_stack_experts():
    def weight(K, N, group, fill):
        return w4.PackedWeight(torch.full((K * N // 8,), fill, dtype=torch.int32), torch.full((K // group * N,), fill, dtype=torch.float16),
                               torch.full((K // group * N // 8,), fill, dtype=torch.int32), K, N, group)
    pe = w4.stack_experts(weight(256, 32, 128, i) for i in range(3))
    assert (pe.experts, pe.K, pe.N, pe.group) == (3, 256, 32, 128)
    assert all((pe.expert(e).Wq == e).all() and (pe.expert(e).Sp == e).all() and (pe.expert(e).Zp == e).all() for e in range(3))
    with pytest.raises(ValueError, match="differ"):
        w4.stack_experts([weight(256, 32, 128, 0), weight(256, 32, 64, 0)])
    with pytest.raises(ValueError, match="no experts"):
        w4.stack_experts([])


def test_flag_values():
    import os
    import re
    header = open(os.path.join(wbuild.INCLUDE, "w4a16.h")).read()
    for name in ("ROUTE_FP32", "ROUTE_SIGMOID", "ROUTE_RENORMALIZE", "EXPERTS_PER_CHOICE", "EXPERTS_COMBINE"):
        assert int(re.search(rf"#define W4A16_{name} (0x[0-9a-f]+)", header).group(1), 16) == getattr(w4, name)
