"""The router and the products grouped by expert at the largest sizes, beyond
32 bits of bytes and of elements, and on two streams at once."""
import pytest
import torch

import bit_weight_only_g128_gb300 as w4
import experts_close
import experts_ref as ref
from test_gpu_experts import BF16, FP16, PATHS, check_route, experts, gen, normal
from test_gpu_experts_routing import listed

pytestmark = pytest.mark.gpu


def random_experts(g, E, K, N, group):
    """Packed weights of random codes and zero points."""
    def words(n):
        return torch.randint(-2 ** 31, 2 ** 31, (n,), generator=g, device="cuda", dtype=torch.int64).int()
    Wq = torch.cat([words(K * N // 8) for _ in range(E)])
    Sp = (torch.rand((E * (K // group) * N,), generator=g, device="cuda") * 0.01 + 0.001).half()
    return w4.PackedExperts(Wq, Sp, words(E * (K // group) * N // 8), E, K, N, group)


def columns(pe, e, cols):
    """[K, cols] of expert e's (q - z) s in 64 bits."""
    q, s, z = (t[:, cols].double() for t in w4.unpack(pe.expert(e)))
    rep = lambda t: t.repeat_interleave(pe.group, 0)  # noqa: E731
    return (q - rep(z)) * rep(s)


@pytest.mark.parametrize("path", PATHS)
def test_weights_beyond_32_bits(path):
    g = gen(1)
    E, K, N = 40, 8192, 28672
    pe = random_experts(g, E, K, N, 128)
    assert pe.Wq.numel() * 4 > 1 << 32
    T = 3
    of = torch.tensor([[0, 39], [38, 37], [39, 20]], device="cuda")
    routing = listed(of, E, torch.rand((T, 2), generator=g, device="cuda"))
    A = normal(g, T, K, dtype=FP16)
    plain = w4.gemm_experts(A, pe, routing, path=path)
    silu = w4.gemm_experts(A, pe, routing, silu_mul=True, path=path)
    both = w4.gemm_experts(A, pe, routing, combine=True, path=path)
    w4.device_status()
    u = 0.0 if path == "decode" else ref.WEIGHT_ERROR[FP16]
    half = N // 2
    near = torch.cat([torch.arange(a, a + 32, device="cuda") for a in (0, half - 32, half, N - 32)])
    W = torch.zeros((E, K, 128), dtype=torch.float64, device="cuda")
    for e in set(of.flatten().tolist()):
        W[e] = columns(pe, e, near)
    y, tol = ref.products(A, W, of, u)
    experts_close.close(plain[:, :, near], y, tol, path)
    total, bound = ref.combine(y, tol, routing.weights, of, ref.U[FP16])
    experts_close.close(both[:, near], total, bound, path, combine=True)
    gate_up = torch.cat([torch.arange(0, 64), torch.arange(64, 128)]).cuda()  # 32 first and 32 last columns of gate, and of up
    act, bound = ref.silu_mul(y[:, :, gate_up], tol[:, :, gate_up])
    experts_close.close(silu[:, :, torch.cat([near[:32], near[32:64]])], act, bound, path, silu=True)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("T,K,N", [(33000, 8192, 64), (17000, 64, 16384)])
def test_activations_and_results_beyond_31_bits(T, K, N, path):
    g = gen(2)
    E, top = 8, 8
    pe = random_experts(g, E, K, N, 64)
    routing = w4.route(normal(g, T, E), top)
    A = torch.empty((T, top, K), dtype=BF16, device="cuda").normal_(generator=g)
    assert max(A.numel(), T * top * N) > 1 << 31
    W = ref.weights_of(pe)
    some = torch.cat([torch.arange(20), torch.randint(0, T, (40,)), torch.arange(T - 20, T)]).cuda()
    y, tol = ref.products(A[some], W, routing.experts[some], 0.0 if path == "decode" else ref.WEIGHT_ERROR[BF16])
    got = w4.gemm_experts(A, pe, routing, path=path)
    experts_close.close(got[some], y, tol, path)
    del got
    got = w4.gemm_experts(A, pe, routing, combine=True, path=path)
    experts_close.close(got[some], *ref.combine(y, tol, routing.weights[some], routing.experts[some], ref.U[BF16]), path, combine=True)
    w4.device_status()


@pytest.mark.parametrize("T,E,top", [(1 << 20, 8, 2), ((1 << 20) - 1, 64, 8), (1 << 18, 512, 4)])
def test_route_of_the_most_tokens(T, E, top):
    x = normal(gen(T), T, E, dtype=BF16)
    x[::9] = -float("inf")
    check_route(x, top)


def test_one_row_of_any_stride_and_rows_that_overlap():
    x = normal(gen(3), 70, 64)
    want = w4.route(x[21:22].clone(), 4)
    for row in (x[21::60][:1], x.t().contiguous().t()[21:22].clone(), x[21:22].expand(1, 64)):
        assert all(torch.equal(a, b) for a, b in zip(w4.route(row, 4), want))
    with pytest.raises(w4.W4A16Error, match="row stride"):
        w4.route(x[:1].expand(5, 64), 4)


@pytest.mark.parametrize("path", PATHS)
def test_two_streams_at_once(path):
    """Each with the cached workspace of its own."""
    g = gen(4)
    pe = experts(g, 8, 256, 512, 128)
    calls = []
    for T in (700, 650):
        routing = w4.route(normal(g, T, 8), 4)
        A = normal(g, T, 4, 256, dtype=FP16)
        calls.append((A, routing, w4.gemm_experts(A, pe, routing, combine=True, path=path)))
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[] for _ in calls]
    for _ in range(20):
        for (A, routing, _), stream, results in zip(calls, streams, got):
            with torch.cuda.stream(stream):
                results.append(w4.gemm_experts(A, pe, routing, combine=True, path=path))
    torch.cuda.synchronize()
    for (_, _, want), results in zip(calls, got):
        assert all(torch.equal(r, want) for r in results)
    w4.device_status()
