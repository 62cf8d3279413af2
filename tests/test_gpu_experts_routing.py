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
