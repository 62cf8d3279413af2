"""Activations, weights and products at the ends of their types' ranges through
the products grouped by expert, on both paths, against the definition in 64
bits."""
import pytest
import torch

import bit_weight_only_g128_gb300 as w4
import experts_ref as ref
from layer_ref import within
from test_gpu_experts import BF16, FP16, PATHS, experts, gen, normal, rounding

pytestmark = pytest.mark.gpu


def agree(got, want, tol):
    """NaN and infinities where the definition has them, the rest within tol."""
    assert torch.equal(got.isnan(), want.isnan())
    far = want.isinf()
    assert torch.equal(got[far].double(), want[far])
    fine = want.isfinite()
    within(got[fine], want[fine], tol[fine])


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("group", [64, 128, 256])
@pytest.mark.parametrize("T", [1, 2, 8, 9, 40])
@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_infinite_activations(dtype, T, group, path):
    """Whatever the rows of an expert: plus or minus infinity by the sign of q -
    z, NaN where it is zero."""
    g = gen(T + group)
    pe = experts(g, 2, 256, 96, group)
    routing = w4.route(normal(g, T, 2), 2)
    A = normal(g, T, 256, dtype=dtype)
    A[0, 17] = float("inf")
    A[T // 2, 200] = -float("inf")
    u = rounding(path, dtype)
    y, tol = ref.products(A, ref.weights_of(pe), routing.experts, u)
    assert y.isinf().any() and y.isnan().any()
    agree(w4.gemm_experts(A, pe, routing, path=path), y, tol)
    agree(w4.gemm_experts(A, pe, routing, silu_mul=True, path=path), *ref.silu_mul(y, tol))
    agree(w4.gemm_experts(A, pe, routing, combine=True, path=path),
          *ref.combine(y, tol, routing.weights, routing.experts, ref.U[dtype]))
    w4.device_status()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("group", [64, 128, 256])
@pytest.mark.parametrize("T", [1, 8, 9, 40])
def test_large_bf16_activations(T, group, path):
    """Finite results of activations next to the type's largest: neither the
    codes' form nor a group's sum before its scale may overflow."""
    g = gen(T + group)
    pe = experts(g, 2, 256, 96, group)
    routing = w4.route(normal(g, T, 2), 2)
    W = ref.weights_of(pe)
    one = normal(g, T, 256, dtype=BF16)
    one[:, 5] = 2.0 ** 124
    for A in (one, torch.full((T, 256), 2.0 ** 124, dtype=BF16, device="cuda")):
        y, tol = ref.products(A, W, routing.experts, rounding(path, BF16))
        assert y.abs().max() < torch.finfo(BF16).max
        within(w4.gemm_experts(A, pe, routing, path=path), y, tol)
        within(w4.gemm_experts(A, pe, routing, combine=True, path=path),
               *ref.combine(y, tol, routing.weights, routing.experts, ref.U[BF16]))
    w4.device_status()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("per_choice", [False, True])
@pytest.mark.parametrize("T", [1, 5, 40, 300])
@pytest.mark.parametrize("N,K,group", [(96, 256, 128), (272, 192, 64)])
def test_products_beyond_fp16_whose_sum_is_not(N, K, group, T, per_choice, path):
    """Single products beyond 65504, some by far, beside ordinary ones in the
    same rows: their weighted sum is finite, on both paths."""
    g = gen(T + N)
    pe = w4.stack_experts([w4.quantize_pack(normal(g, K, N, std=std), group) for std in (0.5, 0.5, 0.02, 0.5)])
    routing = w4.route(normal(g, T, 4), 3)
    routing.weights.mul_(0.01)
    routing.weights[::2, 1] *= -1
    A = (normal(g, T, 3, K) if per_choice else normal(g, T, K)).mul_(15000).clamp_(-60000, 60000).to(FP16)
    A[-1] = normal(g, *A[-1].shape, dtype=FP16)  # a token with none
    y, tol = ref.products(A, ref.weights_of(pe), routing.experts, rounding(path, FP16))
    want, tol = ref.combine(y, tol, routing.weights, routing.experts, ref.U[FP16])
    assert want.abs().max() < 60000 and (T == 1 or 0.1 < (y.abs() > 65520).double().mean() < 0.9)
    ws = w4.new_workspace(w4.experts_workspace_size(T, 3, pe, combine=True, path=path))
    for fill in (0xFF, 0):  # whatever it held
        ws[w4.FLAG_BYTES:] = fill
        within(w4.gemm_experts(A, pe, routing, combine=True, path=path, workspace=ws), want, tol)
    routing.weights.mul_(1e5)  # sums beyond the range are infinite
    assert not w4.gemm_experts(A, pe, routing, combine=True, path=path).isnan().any()
    w4.device_status()
