"""A captured step of a decoder stack with experts beside eager calls that need
a larger workspace on the same stream."""
import pytest
import torch

import bit_weight_only_g128_gb300 as w4
from bit_weight_only_g128_gb300 import run_layer
from test_gpu_experts import FP16, experts, gen, normal
from test_gpu_run_experts import BATCH, LAYERS, SHAPE

pytestmark = pytest.mark.gpu


def test_replays_after_the_streams_workspace_has_grown():
    a, b = (run_layer.Stack(SHAPE, LAYERS, BATCH, 64, seed=3) for _ in range(2))
    x, token = (torch.randn((n, SHAPE.hidden), device="cuda").half() for n in (6, BATCH))
    for s in (a, b):
        s.prompt(x, [3, 1, 2])
    want = [a.step(token).clone() for _ in range(4)]
    g = gen(1)
    pe, A = experts(g, 4, 128, 512, 128), normal(g, 2000, 3, 128, dtype=FP16)
    routing = w4.route(normal(g, 2000, 4), 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(b.step(token), want[0])  # the stream's workspace
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = b.step(token)
    before = w4.stream_workspace(1, 0, side.cuda_stream)
    size, address = before.numel(), before.data_ptr()
    del before
    with torch.cuda.stream(side):
        sums = w4.gemm_experts(A, pe, routing, combine=True)
        assert w4.stream_workspace(1, 0, side.cuda_stream).numel() > size
        others = [torch.full((size,), 5, dtype=torch.uint8, device="cuda") for _ in range(4)]
        assert all(t.data_ptr() != address for t in others), "the graph's workspace was given away"
    for w in want[1:]:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
    assert all((t == 5).all() for t in others)
    with torch.cuda.stream(side):
        assert torch.equal(w4.gemm_experts(A, pe, routing, combine=True), sums)
    torch.cuda.synchronize()
    w4.device_status()


def test_a_graph_whose_workspace_was_made_in_another_capture():
    """Neither stream has had a call before: the second graph runs without the
    first's zero-fill."""
    g = gen(5)
    pw = w4.quantize_pack(normal(g, 1024, 512, std=0.02), 128)
    x = normal(g, 40, 1024, dtype=FP16)
    want = w4.gemm(x, pw, path="tensor", parts=4)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for graph in graphs:
        with torch.cuda.graph(graph, stream=side):
            outs.append(w4.gemm(x, pw, path="tensor", parts=4))
            inside = w4.stream_workspace(1, 0, side.cuda_stream)
    inside[:w4.FLAG_BYTES] = 0xFF  # as memory may be before the first graph has run
    torch.cuda.synchronize()
    for i in (1, 0, 1):
        outs[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want)
    with torch.cuda.stream(side):
        assert w4.stream_workspace(1, 0, side.cuda_stream) is not inside
        assert torch.equal(w4.gemm(x, pw, path="tensor", parts=4), want)
    torch.cuda.synchronize()
    w4.device_status()
