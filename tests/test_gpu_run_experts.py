"""Decoder stacks with experts and with norms of query and key heads: router,
products grouped by expert, their sum and the attention's operators together,
against the layers in 64 bits."""
import dataclasses

import pytest
import torch

import bit_weight_only_g128_gb300 as w4
import experts_ref
import layer_ref as ref
from bit_weight_only_g128_gb300 import run_layer

pytestmark = pytest.mark.gpu

SHAPE = run_layer.Shape(hidden=512, heads=8, kv_heads=2, intermediate=384, head_dim=64, experts=8, top_k=3, qk_norm=True)
LAYERS, BATCH = 2, 3


@pytest.fixture
def routed(monkeypatch):
    """Every router call's answer, checked on its own logits."""
    answers, real = [], w4.route

    def route(logits, top_k, **more):
        got = real(logits, top_k, **more)
        experts, weights, rows, offsets, tol = experts_ref.route(logits, top_k, "softmax", True)
        assert torch.equal(got.experts, experts) and torch.equal(got.rows, rows) and torch.equal(got.offsets, offsets)
        ref.within(got.weights, weights, tol)
        answers.append(got)
        return got

    monkeypatch.setattr(w4, "route", route)
    return answers


def normed(x, weight, eps=1e-5):
    return x * (x.square().mean(2, keepdim=True) + eps).rsqrt() * weight.double()


def reference(stack, x, chosen):
    """Hidden states of one sequence [n, hidden] in 64 bits. chosen: each
    layer's experts [n, top_k]: next to a border between two experts the
    stack's 16 bits may fall on either side, so that they are taken from it."""
    s, n = stack.shape, len(x)
    h, x = torch.zeros_like(x, dtype=torch.float64), x.double()
    pos = torch.arange(n, device="cuda")
    hidden = torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1)
    for layer, experts in zip(stack.layers, chosen):
        qkv_w, o_w = (w4.dequantize(pw, dtype=stack.dtype).double() for pw in (layer.qkv, layer.o))
        y, h = ref.rms_norm(x, layer.norm1, h)
        qkv = (y @ qkv_w).view(n, s.heads + 2 * s.kv_heads, s.head_dim)
        q, k, v = qkv.split([s.heads, s.kv_heads, s.kv_heads], 1)
        if s.qk_norm:
            q, k = normed(q, layer.q_norm), normed(k, layer.k_norm)
        q, k = (ref.rope(t, stack.cos_sin, pos, False) for t in (q, k))
        k, v = (t.repeat_interleave(s.heads // s.kv_heads, 1) for t in (k, v))
        w = torch.einsum("qhd,khd->hqk", q, k) * s.head_dim ** -0.5
        x = torch.einsum("hqk,khd->qhd", w.masked_fill(hidden, float("-inf")).softmax(2), v).reshape(n, -1) @ o_w
        y, h = ref.rms_norm(x, layer.norm2, h)
        score = torch.gather(y @ layer.router.double(), 1, experts.long())
        gu, _ = experts_ref.products(y, experts_ref.weights_of(layer.gate_up), experts)
        act, _ = experts_ref.silu_mul(gu, torch.zeros_like(gu))
        out, _ = experts_ref.products(act, experts_ref.weights_of(layer.down), experts)
        x = (score.softmax(1)[..., None] * out).sum(1)
    return h + x


@pytest.mark.parametrize("dtype,e4m3,qk_norm", [(torch.float16, False, True), (torch.bfloat16, False, True), (torch.float16, True, True),
                                                (torch.float16, False, False)])
def test_prompts_and_steps_match_the_definition(routed, dtype, e4m3, qk_norm):
    shape = dataclasses.replace(SHAPE, qk_norm=qk_norm)
    counts, steps = [37, 5, 150], 2
    stack = run_layer.Stack(shape, LAYERS, BATCH, 256, dtype=dtype, e4m3=e4m3, seed=1)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    xs = [torch.randn((n + steps, shape.hidden), generator=gen, device="cuda").to(dtype) for n in counts]
    got = [list(stack.prompt(torch.cat([x[:n] for x, n in zip(xs, counts)]), counts).split(counts))]
    got += [list(stack.step(torch.stack([x[n + i] for x, n in zip(xs, counts)])).split(1)) for i in range(steps)]
    w4.device_status()
    # each call's experts, by layer and sequence
    calls = [[routed[c * LAYERS + i].experts.split(counts if c == 0 else [1] * BATCH) for i in range(LAYERS)] for c in range(1 + steps)]
    # as the stack of dense layers: about 14 roundings of relative u on a path
    # (two of them weights' in gate/up and down), e4m3 keys and values to 2^-4
    per_layer = 14 * ref.U[dtype] + (2 * 2.0 ** -4 if e4m3 else 0)
    for b in range(BATCH):
        chosen = [torch.cat([calls[c][i][b] for c in range(1 + steps)]) for i in range(LAYERS)]
        want = reference(stack, xs[b], chosen)
        y = torch.cat([call[b] for call in got]).double()
        err = float((y - want).norm() / want.norm())
        assert err <= 2 * LAYERS * per_layer, (b, err)


def test_step_as_a_graph_equals_the_step():
    a, b = (run_layer.Stack(SHAPE, LAYERS, BATCH, 64, seed=3) for _ in range(2))
    x, token = (torch.randn((n, SHAPE.hidden), device="cuda").half() for n in (6, BATCH))
    for s in (a, b):
        s.prompt(x, [3, 1, 2])
    want = [a.step(token).clone() for _ in range(3)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = b.step(token)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = b.step(token)
    assert torch.equal(first, want[0])
    for w in want[1:]:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
    w4.device_status()


def test_command():
    res = run_layer.run("experts-64x8", layers=1, batch=2, prompt=40, steps=2)
    assert res["prompt_us_per_layer"] > 0 and res["step_us_per_layer"] > 0
