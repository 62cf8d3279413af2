"""The products grouped by expert held to the narrow bounds that
test_experts_bounds.py finds mistakes with: (q - z) s in 64 bits, K additions in
fp32 of the terms a (q - z) s themselves, and the result's rounding; on the
tensor cores' path the weights' rounding, and combined the products'."""
import pytest
import torch

import bit_weight_only_g128_gb300 as w4
import experts_close
import experts_ref as ref
from test_gpu_experts import BF16, FP16, PATHS, SHAPES, experts, gen, normal

pytestmark = pytest.mark.gpu


def check_all(g, pe, routing, dtype, path):
    T, top = routing.experts.shape
    W = ref.weights_of(pe)

    def call(A, **more):
        return w4.gemm_experts(A, pe, routing, path=path, **more)

    for A in (normal(g, T, pe.K, dtype=dtype), normal(g, T, top, pe.K, dtype=dtype)):
        experts_close.check(call, A, W, routing, path, dtype)
        experts_close.check(call, A, W, routing, path, dtype, combine=True)
        if pe.N % 32 == 0:
            experts_close.check(call, A, W, routing, path, dtype, silu=True)
    w4.device_status()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("E,K,N,group", SHAPES)
@pytest.mark.parametrize("T", [1, 2, 7, 9, 15, 40])
@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_products(E, K, N, group, T, dtype, path):
    g = gen(E * 2 + K + N + T)
    check_all(g, experts(g, E, K, N, group), w4.route(normal(g, T, E), min(2, E)), dtype, path)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("K,group", [(11008, 128), (4096, 4096), (8192, 64)])
@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_long_k(K, group, dtype, path):
    g = gen(K)
    check_all(g, experts(g, 3, K, 64, group), w4.route(normal(g, 20, 3), 2), dtype, path)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("T,E,top", [(24, 8, 4), (100, 16, 4), (300, 16, 8), (700, 12, 4)])
def test_ten_to_three_hundred_rows_per_expert(T, E, top, path):
    """Between the two paths' usual numbers of rows."""
    g = gen(T)
    check_all(g, experts(g, E, 384, 96, 128), w4.route(normal(g, T, E), top), BF16, path)
