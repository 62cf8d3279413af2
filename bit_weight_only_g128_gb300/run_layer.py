"""Run a stack of decoder layers: the W4A16 linears and the operators between.

    python -m bit_weight_only_g128_gb300.run_layer --model llama2-7b [--layers 2]
        [--batch 4] [--prompt 500] [--steps 32] [--cache e4m3] [--a8] [--bf16]

Layers of the model's shape with seeded random weights take the prompts of
`batch` sequences (of mixed lengths up to `prompt` tokens) through norm, qkv
GEMM, rotation with the cache's append, prompt attention, o_proj, norm, fused
gate/up and down GEMMs, and then `steps` single tokens per sequence through
the same with decode attention, the step captured once as a CUDA graph.
Prints one JSON line: the prompts' and a step's time per layer. ``Stack`` is
the same for use from Python.
"""
from __future__ import annotations

import argparse
import dataclasses
import json
from typing import List

import torch

import bit_weight_only_g128_gb300 as w4


@dataclasses.dataclass(frozen=True)
class Shape:
    hidden: int
    heads: int
    kv_heads: int
    intermediate: int
    head_dim: int = 128
    group: int = 128


SHAPES = {
    "llama2-7b": Shape(4096, 32, 32, 11008),
    "llama2-13b": Shape(5120, 40, 40, 13824),
    "llama2-70b": Shape(8192, 64, 8, 28672),
}


@dataclasses.dataclass
class Layer:
    qkv: w4.PackedWeight
    o: w4.PackedWeight
    gate_up: w4.PackedWeight
    down: w4.PackedWeight
    norm1: torch.Tensor
    norm2: torch.Tensor
    cache: w4.KVCache


def rotary_table(length: int, dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """cos_sin [length, dim] for rope_append: cosines, then sines, of the
    angles p * base^(-2i/dim)."""
    f = base ** (-torch.arange(0, dim, 2, device=device, dtype=torch.float64) / dim)
    angle = torch.arange(length, device=device, dtype=torch.float64)[:, None] * f
    return torch.cat([angle.cos(), angle.sin()], 1).float()


class Stack:
    """Decoder layers over one paged cache per layer and one page table for
    all. The sequences' pages are assigned at the start, in turn, for
    `longest` tokens each (rounded up to pages). Tokens beyond them are
    refused; those of a replayed graph, which the host does not see, are not
    stored and are recorded (device_status)."""

    def __init__(self, shape: Shape, layers: int, batch: int, longest: int, page: int = 16,
                 dtype: torch.dtype = torch.float16, e4m3: bool = False, a8: bool = False, seed: int = 0):
        self.shape, self.batch, self.page, self.dtype, self.a8 = shape, batch, page, dtype, a8
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        per = -(-longest // page)
        order = torch.randperm(batch * per, generator=gen, device="cuda").to(torch.int32)
        # a page more than a sequence has names a slot beyond the cache
        self._pages = torch.full((batch, per + 1), batch * per, dtype=torch.int32, device="cuda")
        self._pages[:, :per] = order.view(batch, per)
        self.table = self._pages[:, :per]
        self.capacity = per * page
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self._held = [0] * batch  # as far as the host knows
        self.cos_sin = rotary_table(self.capacity, shape.head_dim)
        scale = torch.full((shape.kv_heads,), 0.05, device="cuda") if e4m3 else None

        def weight(K, N):
            return w4.quantize_pack(torch.randn((K, N), generator=gen, device="cuda") * 0.02, shape.group)

        def ones():
            return (1 + 0.1 * torch.randn(shape.hidden, generator=gen, device="cuda")).to(dtype)

        h, d = shape.hidden, shape.head_dim
        self.layers: List[Layer] = [
            Layer(weight(h, (shape.heads + 2 * shape.kv_heads) * d), weight(shape.heads * d, h),
                  weight(h, 2 * shape.intermediate), weight(shape.intermediate, h), ones(), ones(),
                  w4.new_kv_cache(batch * per, shape.kv_heads, page, d, torch.float8_e4m3fn if e4m3 else dtype,
                                  scale, scale))
            for _ in range(layers)]

    def _norm_gemm(self, x, h, norm, pw, silu_mul=False):
        """The norm of x + h (h updated) times a weight, in 16 or 8 bits."""
        if self.a8:
            codes, s, _ = w4.rms_norm(x, norm, residual=h, quant="codes", residual_out=h)
            return w4.gemm_scaled(codes, s, pw, static_weights=True, silu_mul=silu_mul)
        y, _ = w4.rms_norm(x, norm, residual=h, residual_out=h)
        return w4.gemm(y, pw, static_weights=True, silu_mul=silu_mul)

    def _forward(self, x, h, positions, slots, attend):
        for layer in self.layers:
            qkv = self._norm_gemm(x, h, layer.norm1, layer.qkv)
            q = w4.rope_append(qkv, self.cos_sin, positions, slots, layer.cache)
            x = w4.gemm(attend(q, layer.cache).flatten(1), layer.o, static_weights=True, a8=self.a8)
            y = self._norm_gemm(x, h, layer.norm2, layer.gate_up, silu_mul=True)
            x = w4.gemm(y, layer.down, static_weights=True, a8=self.a8)
        return h.add_(x)

    def clear(self) -> None:
        """Forget the sequences' tokens."""
        self.lens.zero_()
        self._held = [0] * self.batch

    def _take(self, counts: List[int], rows: int) -> None:
        """Refuse new tokens that do not fit, or count them."""
        if len(counts) != self.batch or min(counts) < 0 or sum(counts) != rows:
            raise ValueError(f"{rows} rows and counts {counts} do not fit {self.batch} sequences")
        held = [a + n for a, n in zip(self._held, counts)]
        if max(held) > self.capacity:
            raise ValueError(f"a sequence of {max(held)} tokens is longer than the {self.capacity} that the stack holds")
        self._held = held

    def prompt(self, x: torch.Tensor, counts: List[int]) -> torch.Tensor:
        """The rows of counts[b] new tokens of every sequence, one after
        another ([sum(counts), hidden]); returns their hidden states. x is not
        changed."""
        self._take(counts, len(x))
        new = torch.tensor(counts, dtype=torch.int32, device="cuda")
        starts = torch.zeros(self.batch + 1, dtype=torch.int32, device="cuda")
        starts[1:] = new.cumsum(0)
        of = torch.repeat_interleave(torch.arange(self.batch, device="cuda"), new.long(), output_size=sum(counts))
        positions = torch.arange(len(x), device="cuda") - starts[of] + self.lens[of]
        self.lens += new
        return self._forward(x, torch.zeros_like(x), positions.int(), self._slots(of, positions.long()),
                             lambda q, cache: w4.attn_prompt(q, cache, self.table, starts, self.lens))

    def step(self, x: torch.Tensor) -> torch.Tensor:
        """One new token of every sequence ([batch, hidden]); returns their
        hidden states. Every launch is on the current stream and none waits
        for the host: it can be captured as a CUDA graph."""
        self._take([1] * self.batch, len(x))
        positions = self.lens.long()
        self.lens += 1
        of = torch.arange(self.batch, device="cuda")
        return self._forward(x, torch.zeros_like(x), positions.int(), self._slots(of, positions),
                             lambda q, cache: w4.attn_decode(q, cache, self.table, self.lens))

    def _slots(self, of, positions):
        page = (positions // self.page).clamp_(max=self._pages.shape[1] - 1)
        return self._pages[of, page].long() * self.page + positions % self.page


def run(model: str, layers: int, batch: int, prompt: int, steps: int, e4m3=False, a8=False, bf16=False, seed=0):
    shape = SHAPES[model]
    dtype = torch.bfloat16 if bf16 else torch.float16
    counts = [max(1, prompt * (batch - b) // batch) for b in range(batch)]
    stack = Stack(shape, layers, batch, prompt + steps + 8, dtype=dtype, e4m3=e4m3, a8=a8, seed=seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + 1)

    def rows(n):
        return torch.randn((n, shape.hidden), generator=gen, device="cuda").to(dtype)

    x = rows(sum(counts))
    mark = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
    stack.prompt(x, counts)  # warm-up; the timed prompt starts over
    stack.clear()
    mark[0].record()
    hidden = stack.prompt(x, counts)
    mark[1].record()
    token = rows(batch)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        stack.step(token)  # warm-up on the capturing stream: its workspaces
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = stack.step(token)
    graph.replay()
    mark[2].record()
    for _ in range(steps):
        graph.replay()
    mark[3].record()
    torch.cuda.synchronize()
    w4.device_status()
    if not (torch.isfinite(hidden).all() and torch.isfinite(out).all()):
        raise RuntimeError("hidden states are not finite")
    return {"model": model, "layers": layers, "batch": batch, "prompt_tokens": sum(counts), "steps": steps,
            "dtype": str(dtype).split(".")[-1], "cache": "e4m3" if e4m3 else "16-bit", "a8": a8,
            "prompt_us_per_layer": mark[0].elapsed_time(mark[1]) * 1e3 / layers,
            "step_us_per_layer": mark[2].elapsed_time(mark[3]) * 1e3 / steps / layers}


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--model", choices=sorted(SHAPES), default="llama2-7b")
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=500)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--cache", choices=["16-bit", "e4m3"], default="16-bit")
    ap.add_argument("--a8", action="store_true", help="W4A8 linears")
    ap.add_argument("--bf16", action="store_true")
    a = ap.parse_args()
    print(json.dumps(run(a.model, a.layers, a.batch, a.prompt, a.steps, a.cache == "e4m3", a.a8, a.bf16)))


if __name__ == "__main__":
    main()
