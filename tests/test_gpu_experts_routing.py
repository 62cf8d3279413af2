"""Routings that no router answers through the products grouped by expert: what
is recorded, what is left out, and the values of everything else."""
import pytest
import torch

import bit_weight_only_g128_gb300 as w4
import experts_ref as ref
from layer_ref import within
from test_gpu_experts import BF16, FP16, PATHS, experts, gen, normal, rounding

pytestmark = pytest.mark.gpu


def recorded():
    """The device's error is the one of data outside its range, once."""
    with pytest.raises(w4.W4A16Error) as e:
        w4.device_status()
    assert e.value.code == -6 and "0x80" in str(e.value)
    w4.device_status()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("T", [1, 5])
@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("value", [4, 5, (1 << 31) - 1])
def test_an_expert_beyond_the_last_counts_as_none_in_the_sum(value, dtype, T, path):
    """Whatever the workspace held: the sum of the token's other choices."""
    g = gen(T)
    pe = experts(g, 4, 256, 96, 128)
    good = w4.route(normal(g, T, 4), 3)
    A = normal(g, T, 256, dtype=dtype)
    bad = w4.Routing(*(t.clone() for t in good))
    bad.experts[T // 2, 1] = value
    ws = w4.new_workspace(w4.experts_workspace_size(T, 3, pe, combine=True, path=path))
    ws[w4.FLAG_BYTES:] = 0xFF  # NaN in fp32 and in 16 bits
    got = w4.gemm_experts(A, pe, bad, combine=True, path=path, workspace=ws)
    recorded()
    left = good.experts.clone()
    left[T // 2, 1] = -1
    y, tol = ref.products(A, ref.weights_of(pe), left, rounding(path, dtype))
    within(got, *ref.combine(y, tol, good.weights, left, ref.U[dtype]))
    if T == 1 and path == "decode":  # the products go by the experts too
        assert not w4.gemm_experts(A, pe, bad, path=path)[0, 1].any()
        recorded()


def listed(experts, E, weights):
    """The Routing of these experts [T, top], whichever they are."""
    flat = experts.flatten()
    rows = torch.sort(torch.where(flat < 0, E, flat), stable=True)[1]
    counts = (flat[:, None] == torch.arange(E, device="cuda")).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return w4.Routing(experts.int(), weights, rows.int(), offsets.int())


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("T", [1, 3, 10, 20, 300])
@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_offsets_that_give_an_expert_everything(dtype, T, path):
    """Products go by rows and offsets alone: all of them expert 1's. (One token
    on the path for few rows: by the experts.)"""
    g = gen(T)
    pe = experts(g, 4, 256, 96, 128)
    good = w4.route(normal(g, T, 4), 3)
    bad = w4.Routing(good.experts, good.weights, good.rows, torch.tensor([0, 0, 3 * T, 3 * T, 3 * T], dtype=torch.int32, device="cuda"))
    A = normal(g, T, 256, dtype=dtype)
    of = good.experts if T == 1 and path == "decode" else torch.ones_like(good.experts)
    y, tol = ref.products(A, ref.weights_of(pe), of, rounding(path, dtype))
    within(w4.gemm_experts(A, pe, bad, path=path), y, tol)
    within(w4.gemm_experts(A, pe, bad, combine=True, path=path), *ref.combine(y, tol, good.weights, of, ref.U[dtype]))
    w4.device_status()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("T", [1, 2, 3, 8, 9, 17, 40])
@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_a_token_may_have_an_expert_several_times(dtype, T, path):
    g = gen(T)
    pe = experts(g, 7, 256, 96, 64 if T % 2 else 128)
    W = ref.weights_of(pe)
    A = normal(g, T, 6, 256, dtype=dtype)
    weights = torch.rand((T, 6), generator=g, device="cuda")
    for of in (torch.full((T, 6), 2, device="cuda"), torch.randint(0, 2, (T, 6), generator=g, device="cuda") * 4,
               torch.randint(-1, 5, (T, 6), generator=g, device="cuda")):
        routing = listed(of, 7, weights)
        y, tol = ref.products(A, W, of, rounding(path, dtype))
        within(w4.gemm_experts(A, pe, routing, path=path), y, tol)
        within(w4.gemm_experts(A, pe, routing, silu_mul=True, path=path), *ref.silu_mul(y, tol))
        within(w4.gemm_experts(A, pe, routing, combine=True, path=path), *ref.combine(y, tol, weights, of, ref.U[dtype]))
    w4.device_status()
