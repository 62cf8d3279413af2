"""The router and the products grouped by expert on the GPU against their
definitions in 64 bits (experts_ref.py)."""
import math

import pytest
import torch

import bit_weight_only_g128_gb300 as w4
import experts_ref as ref
from layer_ref import within

pytestmark = pytest.mark.gpu

FP16, BF16, FP32 = torch.float16, torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def check_route(logits, top, scoring="softmax", renormalize=True, **more):
    got = w4.route(logits, top, scoring=scoring, renormalize=renormalize, **more)
    experts, weights, rows, offsets, tol = ref.route(logits, top, scoring, renormalize)
    assert torch.equal(got.experts, experts)
    assert torch.equal(got.offsets, offsets)
    assert torch.equal(got.rows, rows)
    within(got.weights, weights, tol)
    w4.device_status()
    return got


# ------------------------------------------------------------------ router


@pytest.mark.parametrize("T", [0, 1, 3, 63, 64, 65, 333, 4099])
@pytest.mark.parametrize("E,top", [(1, 1), (4, 2), (8, 8), (31, 3), (60, 4), (64, 8), (128, 6), (160, 1), (500, 32)])
@pytest.mark.parametrize("dtype", [FP32, FP16, BF16])
def test_route(T, E, top, dtype):
    g = gen(T * 3 + E)
    logits = normal(g, T, E, std=2, dtype=dtype)  # 16-bit logits have ties
    for scoring in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            check_route(logits, top, scoring, renormalize)


def test_route_ties_and_zeros_go_to_the_lower_expert():
    x = torch.zeros((70, 64), device="cuda")
    x[::2, ::2] = -0.0
    x[5, 40:] = 3.0
    got = check_route(x, 8)
    assert got.experts[0].tolist() == list(range(8)) and got.experts[5].tolist() == list(range(40, 48))


@pytest.mark.parametrize("T", [5, 300])
def test_route_masked(T):
    """Experts of -inf are not chosen; rows of nothing else choose none."""
    g = gen(4)
    x = normal(g, T, 64)
    x[0] = -math.inf
    x[1, 3:] = -math.inf
    x[2, :] = -math.inf
    x[2, 63] = -80.0
    x[T // 2:, ::2] = -math.inf
    x[-1] = -math.inf
    for scoring in ("softmax", "sigmoid"):
        got = check_route(x, 8, scoring)
    assert got.experts[0].tolist() == [-1] * 8 and got.experts[2].tolist() == [63] + [-1] * 7
    everything = torch.full((T, 64), -math.inf, device="cuda")
    got = check_route(everything, 2)
    assert int(got.offsets[-1]) == 0 and got.rows.tolist() == list(range(2 * T))


def test_route_non_finite():
    x = torch.zeros((6, 8), device="cuda")
    x[0, 5] = math.nan
    x[1, 2] = math.inf
    x[2, 7], x[2, 1] = -math.nan, math.inf
    x[3] = torch.finfo(torch.float32).min
    x[4] = torch.finfo(torch.float32).max
    x[5] = -200.0
    got = w4.route(x, 2)
    # NaN before everything, then infinities
    assert got.experts[:3].tolist() == [[5, 0], [2, 0], [7, 1]]
    assert got.weights[0].isnan().all() and got.weights[1, 0].isnan() and got.weights[2].isnan().all()
    assert got.weights[3:].tolist() == [[0.5, 0.5]] * 3
    assert w4.route(x, 2, scoring="sigmoid").weights[5].tolist() == [0.0, 0.0]  # both underflow
    w4.device_status()


def test_route_strided_logits_streams_and_graphs():
    g = gen(9)
    wide = normal(g, 200, 100, dtype=BF16)
    check_route(wide[:, 7:71], 4)
    check_route(wide[::2, 1:33], 4)
    x = normal(g, 200, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = w4.route(x, 4, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want = check_route(x, 4)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        got = w4.route(x, 4)
    for seed in (1, 2):
        x.copy_(normal(gen(seed), 200, 64))
        graph.replay()
        torch.cuda.synchronize()
        want = w4.route(x, 4)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------ products


def experts(g, E, K, N, group):
    return w4.stack_experts([w4.quantize_pack(normal(g, K, N, std=0.02), group) for _ in range(E)])


def rounding(path, dtype):
    """Relative error of a weight on a path: the codes are exact where rows are few."""
    return 0.0 if path == "decode" else ref.WEIGHT_ERROR[dtype]


def guarded(*shape, dtype):
    n = math.prod(shape)
    full = torch.full((n + 128,), 7.0, dtype=dtype, device="cuda")
    return full, full[64:64 + n].view(shape)


def check_products(g, pe, routing, dtype, path, silu=True, plain=True, combine=True):
    T, top = routing.experts.shape
    W = ref.weights_of(pe)
    tokens, each = normal(g, T, pe.K, dtype=dtype), normal(g, T, top, pe.K, dtype=dtype)
    u = rounding(path, dtype)
    terms = ref.terms_of(pe, dtype) if path == "decode" else None
    for A in (tokens, each):
        y, tol = ref.products(A, W, routing.experts, u, terms)
        if plain:
            full, out = guarded(T, top, pe.N, dtype=dtype)
            assert w4.gemm_experts(A, pe, routing, path=path, out=out) is out
            within(out, y, tol)
            assert (full[:64] == 7).all() and (full[-64:] == 7).all()
            assert torch.equal(w4.gemm_experts(A, pe, routing, path=path), out)
        if silu and pe.N % 32 == 0:
            full, out = guarded(T, top, pe.N // 2, dtype=dtype)
            w4.gemm_experts(A, pe, routing, silu_mul=True, path=path, out=out)
            within(out, *ref.silu_mul(y, tol))
            assert (full[:64] == 7).all() and (full[-64:] == 7).all()
        if combine:
            full, out = guarded(T, pe.N, dtype=dtype)
            w4.gemm_experts(A, pe, routing, combine=True, path=path, out=out)
            within(out, *ref.combine(y, tol, routing.weights, routing.experts, ref.U[dtype]))
            assert (full[:64] == 7).all() and (full[-64:] == 7).all()
            assert torch.equal(w4.gemm_experts(A, pe, routing, combine=True, path=path), out)
    w4.device_status()


PATHS = ["decode", "tensor-pair"]
SHAPES = [(1, 64, 16, 64), (7, 128, 48, 128), (4, 640, 96, 128), (8, 128, 32, 64), (5, 192, 208, 64), (4, 256, 288, 256), (3, 1024, 160, 128),
          (4, 1408, 96, 64), (2, 2048, 544, 128), (16, 384, 64, 384), (2, 4096, 48, 512), (2, 5120, 32, 1024)]


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("E,K,N,group", SHAPES)
@pytest.mark.parametrize("T", [1, 2, 9, 15, 40])
@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_products(E, K, N, group, T, dtype, path):
    g = gen(E + K + N + T)
    routing = w4.route(normal(g, T, E), min(2, E))
    check_products(g, experts(g, E, K, N, group), routing, dtype, path)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("T,E,top", [(1, 64, 8), (7, 200, 32), (33, 40, 40 - 8), (130, 8, 1), (520, 3, 2), (40, 512, 4)])
def test_products_of_many_experts_and_rows(T, E, top, path):
    g = gen(T + E)
    routing = w4.route(normal(g, T, E), top, scoring="sigmoid", renormalize=False)
    check_products(g, experts(g, E, 128, 64, 128), routing, BF16, path)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("K,group", [(64, 64), (128, 128), (192, 64), (320, 64), (512, 128), (576, 192)])
@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_many_tiles_of_little_work(K, group, dtype, path):
    """Several tiles (items) for every block, each with as little as one stage
    of K: the streams run on across them. Experts of few rows, of one or two
    parts, and of several tiles."""
    g = gen(K)
    E, N, T = 24, 1056, 1500
    x = normal(g, T, E) + torch.linspace(-4, 3, E, device="cuda")
    routing = w4.route(x, 4)
    counts = routing.offsets.diff()
    assert int(counts.min()) < 40 and int(counts.max()) > 600
    check_products(g, experts(g, E, K, N, group), routing, dtype, path)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("T", [1, 6, 300])
def test_uneven_and_empty_experts(T, path):
    """All tokens to two experts of ten; some tokens, or all, to none."""
    g = gen(T)
    pe = experts(g, 10, 256, 96, 128)
    x = normal(g, T, 10)
    x[:, 3] += 50
    x[:, 8] += 40
    check_products(g, pe, w4.route(x, 2), FP16, path)
    x[::2] = -math.inf
    x[1::3, :8] = -math.inf
    check_products(g, pe, w4.route(x, 3), FP16, path)
    x[:] = -math.inf
    routing = w4.route(x, 2)
    A = normal(g, T, 256, dtype=FP16)
    assert not w4.gemm_experts(A, pe, routing, path=path).any()
    assert not w4.gemm_experts(A, pe, routing, silu_mul=True, path=path).any()
    assert not w4.gemm_experts(A, pe, routing, combine=True, path=path).any()
    w4.device_status()


@pytest.mark.parametrize("path", PATHS)
def test_a_non_finite_row_stays_in_its_own_result(path):
    g = gen(2)
    pe = experts(g, 4, 256, 64, 128)
    routing = w4.route(normal(g, 21, 4), 2)
    A = normal(g, 21, 256, dtype=FP16)
    want = w4.gemm_experts(A, pe, routing, path=path)
    A[5, 17] = math.nan
    A[6, 200] = math.inf
    got = w4.gemm_experts(A, pe, routing, path=path)
    others = [t for t in range(21) if t not in (5, 6)]
    assert torch.equal(got[others], want[others]) and got[5].isnan().all() and not got[6].isfinite().any()


@pytest.mark.parametrize("path", PATHS)
def test_no_tokens(path):
    g = gen(1)
    pe = experts(g, 4, 128, 64, 128)
    routing = w4.route(torch.empty((0, 4), device="cuda"), 2)
    assert routing.offsets.tolist() == [0] * 5
    A = torch.empty((0, 128), dtype=FP16, device="cuda")
    assert w4.gemm_experts(A, pe, routing, path=path).shape == (0, 2, 64)
    assert w4.gemm_experts(A, pe, routing, combine=True, path=path).shape == (0, 64)


@pytest.mark.parametrize("path", PATHS)
def test_bad_routing_is_recorded_and_touches_nothing_else(path):
    g = gen(3)
    pe = experts(g, 4, 128, 64, 128)
    good = w4.route(normal(g, 9, 4), 2)
    A = normal(g, 9, 128, dtype=FP16)
    want = w4.gemm_experts(A, pe, good, path=path)
    for name, at, value in (("rows", 3, -1), ("rows", 0, 18), ("rows", 5, 1 << 30), ("offsets", 4, 19), ("offsets", 2, 1 << 30),
                            ("offsets", 0, -5)):
        bad = w4.Routing(*(t.clone() for t in good))
        lost = int(good.rows[at]) if name == "rows" else None
        getattr(bad, name)[at] = value
        full, out = guarded(9, 2, 64, dtype=FP16)
        w4.gemm_experts(A, pe, bad, path=path, out=out)
        w4.gemm_experts(A, pe, bad, combine=True, path=path)
        with pytest.raises(w4.W4A16Error) as e:
            w4.device_status()
        assert e.value.code == -6 and "0x80" in str(e.value)
        assert (full[:64] == 7).all() and (full[-64:] == 7).all()
        if lost is not None:  # every other choice as before, the one that is not listed left alone
            keep = [f for f in range(18) if f != lost]
            assert torch.equal(out.view(18, 64)[keep], want.view(18, 64)[keep]) and (out.view(18, 64)[lost] == 7).all()
    w4.device_status()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("T", [1, 3, 10, 20])
def test_offsets_that_give_an_expert_everything_or_too_much(T, path):
    """All choices with one expert, which no router answers: recorded or
    computed, and nothing outside the result is written."""
    g = gen(T)
    pe = experts(g, 4, 256, 64, 128)
    good = w4.route(normal(g, T, 4), 3)
    bad = w4.Routing(good.experts, good.weights, good.rows, torch.tensor([0, 0, 3 * T, 3 * T, 3 * T], dtype=torch.int32, device="cuda"))
    full, out = guarded(T, 3, 64, dtype=FP16)
    w4.gemm_experts(normal(g, T, 256, dtype=FP16), pe, bad, path=path, out=out)
    assert (full[:64] == 7).all() and (full[-64:] == 7).all()
    try:
        w4.device_status()
    except w4.W4A16Error as e:
        assert "0x80" in str(e)
    w4.device_status()


@pytest.mark.parametrize("path", PATHS)
def test_streams_graphs_and_workspaces(path):
    g = gen(6)
    pe = experts(g, 8, 256, 64, 128)
    x, A = normal(g, 20, 8), normal(g, 20, 256, dtype=BF16)
    want = w4.gemm_experts(A, pe, w4.route(x, 2), combine=True, path=path)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = w4.gemm_experts(A, pe, w4.route(x, 2, stream=side), combine=True, path=path, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    need = w4.experts_workspace_size(20, 2, pe, combine=True, path=path)
    buf = torch.zeros(need + 256, dtype=torch.uint8, device="cuda")
    buf[need:] = 0xA5
    got = w4.gemm_experts(A, pe, w4.route(x, 2), combine=True, path=path, workspace=buf[:need])
    assert torch.equal(got, want) and (buf[need:] == 0xA5).all() and not buf[:w4.FLAG_BYTES].any()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        routing = w4.route(x, 2)
        got = w4.gemm_experts(A, pe, routing, combine=True, path=path, workspace=buf[:need])
    for seed in (1, 2, 3):  # other experts, other counts
        x.copy_(normal(gen(seed), 20, 8))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, w4.gemm_experts(A, pe, w4.route(x, 2), combine=True, path=path))
    with pytest.raises(w4.W4A16Error, match="WORKSPACE_TOO_SMALL"):
        w4.gemm_experts(A, pe, routing, combine=True, path=path, workspace=buf[:need - 1])
    w4.device_status()


def test_a_layer_of_experts():
    """Router, gate and up, down and the sum together, against the layer in 64 bits."""
    g = gen(12)
    T, E, top, hidden, inner = 37, 16, 4, 512, 384
    gate_up, down = experts(g, E, hidden, 2 * inner, 128), experts(g, E, inner, hidden, 128)
    x, gate = normal(g, T, hidden, dtype=FP16), normal(g, hidden, E, std=0.1)
    logits = x.float() @ gate
    routing = w4.route(logits, top)
    h = w4.gemm_experts(x, gate_up, routing, silu_mul=True)
    got = w4.gemm_experts(h, down, routing, combine=True)
    e, w, _, _, _ = ref.route(logits, top, "softmax", True)
    u = ref.WEIGHT_ERROR[FP16]
    y, tol = ref.products(x, ref.weights_of(gate_up), e, u, ref.terms_of(gate_up, FP16))
    act, tol = ref.silu_mul(y, tol)
    W = ref.weights_of(down)
    y, t2 = ref.products(act, W, e, u, ref.terms_of(down, FP16))
    # h's own error and rounding go through down
    _, mag = ref.products(tol + u * (act.abs() + tol), W.abs(), e)
    within(got, *ref.combine(y, t2 + mag / ((inner + 8) * ref.E32), w, e, u))
    w4.device_status()
