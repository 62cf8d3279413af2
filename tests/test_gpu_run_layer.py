"""The decoder stack of run_layer.py (W4A16 linears, norm, rotation, paged
cache, prompt and decode attention together) against the same layers in 64
bits from the dequantized weights."""
import pytest
import torch

import bit_weight_only_g128_gb300 as w4
import layer_ref as ref
from bit_weight_only_g128_gb300 import run_layer

pytestmark = pytest.mark.gpu

SHAPE = run_layer.Shape(hidden=512, heads=8, kv_heads=2, intermediate=768, head_dim=64)
LAYERS, BATCH = 2, 3


def reference(stack, xs):
    """Hidden states of whole sequences (a list of [n, hidden]) in 64 bits."""
    s, outs = stack.shape, []
    for x in xs:
        n = len(x)
        h, x = torch.zeros_like(x, dtype=torch.float64), x.double()
        pos = torch.arange(n, device="cuda")
        hidden = torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1)
        for layer in stack.layers:
            deq = [w4.dequantize(pw, dtype=stack.dtype).double() for pw in (layer.qkv, layer.o, layer.gate_up, layer.down)]
            y, h = ref.rms_norm(x, layer.norm1, h)
            qkv = (y @ deq[0]).view(n, s.heads + 2 * s.kv_heads, s.head_dim)
            turned = ref.rope(qkv[:, :s.heads + s.kv_heads], stack.cos_sin, pos, False)
            q, k, v = turned[:, :s.heads], turned[:, s.heads:], qkv[:, s.heads + s.kv_heads:]
            k, v = (t.repeat_interleave(s.heads // s.kv_heads, 1) for t in (k, v))
            w = torch.einsum("qhd,khd->hqk", q, k) * s.head_dim ** -0.5
            w = w.masked_fill(hidden, float("-inf")).softmax(2)
            x = torch.einsum("hqk,khd->qhd", w, v).reshape(n, -1) @ deq[1]
            y, h = ref.rms_norm(x, layer.norm2, h)
            gu = y @ deq[2]
            gate, up = gu[:, :s.intermediate], gu[:, s.intermediate:]
            x = (gate * torch.sigmoid(gate) * up) @ deq[3]
        outs.append(h + x)
    return outs


@pytest.mark.parametrize("dtype,e4m3,a8", [(torch.float16, False, False), (torch.bfloat16, False, False),
                                           (torch.float16, True, False), (torch.bfloat16, True, False),
                                           (torch.float16, False, True), (torch.bfloat16, True, True)])
def test_prompt_pieces_and_steps_match_the_definition(dtype, e4m3, a8):
    counts, pieces, steps = [37, 5, 150], [[20, 5, 100], [17, 0, 50]], 3
    stack = run_layer.Stack(SHAPE, LAYERS, BATCH, 256, dtype=dtype, e4m3=e4m3, a8=a8, seed=1)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    xs = [torch.randn((n + steps, SHAPE.hidden), generator=gen, device="cuda").to(dtype) for n in counts]
    want = reference(stack, xs)
    got = [[] for _ in xs]
    done = [0] * BATCH
    for piece in pieces:
        rows = torch.cat([x[d:d + n] for x, d, n in zip(xs, done, piece)])
        out = stack.prompt(rows, piece).split(piece)
        for b in range(BATCH):
            got[b].append(out[b])
            done[b] += piece[b]
    for i in range(steps):
        out = stack.step(torch.stack([x[n + i] for x, n in zip(xs, counts)]))
        for b in range(BATCH):
            got[b].append(out[b:b + 1])
    w4.device_status()
    # A layer rounds about 12 values on a path to 16 bits (relative u each),
    # its e4m3 keys and values to 2^-4, its 8-bit activations (4 of them) to
    # half a step of max / 127, max about 4 times the root mean square; each
    # reaches the result with a factor of 2 at most in these layers.
    per_layer = 12 * ref.U[dtype] + (2 * 2.0 ** -4 if e4m3 else 0) + (4 * 0.5 * 4 / 127 if a8 else 0)
    for b in range(BATCH):
        y = torch.cat(got[b]).double()
        err = float((y - want[b]).norm() / want[b].norm())
        assert err <= 2 * LAYERS * per_layer, (b, err)


def test_command():
    res = run_layer.run("llama2-7b", layers=1, batch=2, prompt=40, steps=2)
    assert res["prompt_us_per_layer"] > 0 and res["step_us_per_layer"] > 0


def test_step_as_a_graph_equals_the_step():
    a, b = (run_layer.Stack(SHAPE, LAYERS, BATCH, 64, seed=3) for _ in range(2))
    x = torch.randn((6, SHAPE.hidden), device="cuda").half()
    token = torch.randn((BATCH, SHAPE.hidden), device="cuda").half()
    a.prompt(x, [3, 1, 2])
    b.prompt(x, [3, 1, 2])
    want = [a.step(token).clone() for _ in range(4)]
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
