"""The bounds that hold the products grouped by expert are narrow enough to find
mistakes at every K: on the CPU, mistakes planted in the weights of a definition
in 64 bits fall outside them (no GPU needed)."""
import pytest
import torch

import experts_close
import experts_ref as ref
from test_gpu_experts import BF16, FP16, SHAPES, rounding


def weights(E, K, N, group, seed):
    """Codes, zero points (spread over K) and scales, as the quantizer gives them for normal weights."""
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn((E, K, N), generator=g) * 0.02).view(E, K // group, group, N)
    lo, hi = w.amin(2, keepdim=True), w.amax(2, keepdim=True)
    s = ((hi - lo) / 15).half().double()
    z = (-lo / s).round().clamp(0, 15)
    q = ((w / s).round() + z).clamp(0, 15)
    return q, z, s


def dropped(q, z, s):
    q, last = q.clone(), q.shape[1] - 1
    q[:, last] = z[:, last]
    return q, z, s


MISTAKES = {
    "a group dropped": dropped,
    "zero points off by one": lambda q, z, s: (q, z + 1, s),
    "the next group's scales": lambda q, z, s: (q, z, s.roll(1, 1)),
    "the next column's zero points": lambda q, z, s: (q, z.roll(1, 3), s),
    "codes of two octets swapped": lambda q, z, s: (torch.cat([q[:, :, 8:16], q[:, :, :8], q[:, :, 16:]], 2), z, s),
}


@pytest.mark.parametrize("path", ["decode", "tensor-pair"])
@pytest.mark.parametrize("mistake", MISTAKES)
@pytest.mark.parametrize("E,K,N,group", SHAPES)
@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_planted_mistakes_are_outside_the_bounds(dtype, E, K, N, group, mistake, path):
    q, z, s = weights(E, K, N, group, K + N)
    if mistake == "the next group's scales" and K == group:
        pytest.skip("one group")
    g = torch.Generator().manual_seed(E)
    T = 3
    A = torch.randn((T, K), generator=g).to(dtype)
    experts = torch.randint(0, E, (T, 1), generator=g)
    y, tol = ref.products(A, ((q - z) * s).view(E, K, N), experts, rounding(path, dtype))
    q, z, s = MISTAKES[mistake](q, z, s)
    wrong, _ = ref.products(A, ((q - z) * s).view(E, K, N), experts)
    most = experts_close.roundings(path) * ref.U[dtype]
    assert experts_close.off(wrong.to(dtype), y) > 3 * most
    assert experts_close.off(y.to(dtype), y) <= most
    bound = tol + ref.U[dtype] * (y.abs() + tol)
    outside = ((wrong.to(dtype).double() - y).abs() > bound).double().mean()
    # (one element of a result would do. The bound of the weights' rounding takes
    # all of them against the result: it may be wide where K is long.)
    assert outside > (0.5 if path == "decode" else 0), float(outside)
    assert ((y.to(dtype).double() - y).abs() <= bound).all()
