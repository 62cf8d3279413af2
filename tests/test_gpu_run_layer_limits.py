"""run_layer.Stack at and beyond the tokens that it holds."""
import pytest
import torch

import bit_weight_only_g128_gb300 as w4
from bit_weight_only_g128_gb300 import run_layer

pytestmark = pytest.mark.gpu

SHAPE = run_layer.Shape(hidden=512, heads=8, kv_heads=2, intermediate=768, head_dim=64)


def rows(n):
    return torch.randn((n, SHAPE.hidden), device="cuda").half()


def test_tokens_beyond_the_longest_sequence_are_refused():
    stack = run_layer.Stack(SHAPE, 1, 2, 32)
    stack.prompt(rows(31), [30, 1])
    for _ in range(2):
        stack.step(rows(2))
    before = stack.lens.clone()
    with pytest.raises(ValueError, match="33 tokens"):
        stack.step(rows(2))
    with pytest.raises(ValueError, match="40 tokens"):
        stack.prompt(rows(37), [0, 37])
    for x, counts in ((rows(3), [1]), (rows(1), [2, -1]), (rows(3), [1, 1]), (rows(1), [1, 1])):
        with pytest.raises(ValueError, match="do not fit"):
            stack.prompt(x, counts)
    assert torch.equal(stack.lens, before)
    stack.prompt(rows(29), [0, 29])  # the other sequence still has room
    assert torch.isfinite(stack.prompt(rows(0), [0, 0])).all()
    stack.clear()
    stack.prompt(rows(64), [32, 32])
    w4.device_status()


def test_a_replayed_step_beyond_the_longest_sequence_is_recorded():
    stack = run_layer.Stack(SHAPE, 2, 2, 16)
    token = rows(2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        stack.step(token)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        stack.step(token)
    for _ in range(15):
        graph.replay()
    w4.device_status()
    kept = [(a.cache.k.clone(), a.cache.v.clone()) for a in stack.layers]
    for _ in range(40):
        graph.replay()
    with pytest.raises(w4.W4A16Error) as e:
        w4.device_status()
    assert e.value.code == -6 and "0x80" in str(e.value)
    for a, (k, v) in zip(stack.layers, kept):
        assert torch.equal(a.cache.k, k) and torch.equal(a.cache.v, v)
    stack.clear()
    stack.prompt(rows(10), [4, 6])
    w4.device_status()
