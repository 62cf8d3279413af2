"""Every call that a decoder stack makes, against its definition in 64 bits on
what the calls before it gave: prompts in pieces and single tokens, in every
type of activations, cache and linears. Element by element, and what each call
is given is what the layer's order says. The walk runs on the CPU; mistakes
planted in it are caught in every mode."""
import dataclasses

import pytest
import torch

import bit_weight_only_g128_gb300 as w4
import layer_ref as ref
from bit_weight_only_g128_gb300 import run_layer

pytestmark = pytest.mark.gpu

SHAPE = run_layer.Shape(hidden=512, heads=8, kv_heads=2, intermediate=768, head_dim=64)
LAYERS, BATCH, PAGE = 2, 3, 16
E4M3 = torch.float8_e4m3fn


def host(x):
    if isinstance(x, torch.Tensor):
        return x.detach().cpu().clone()
    if isinstance(x, w4.KVCache):
        return w4.KVCache(*(None if t is None else host(t) for t in (x.k, x.v, x.k_scale, x.v_scale)))
    return tuple(host(t) for t in x) if isinstance(x, tuple) else x


@dataclasses.dataclass
class Call:
    name: str
    args: tuple
    kwargs: dict
    result: object
    cache: object = None  # after the call


@pytest.fixture
def calls(monkeypatch):
    log = []

    def recorded(name, fn):
        def call(*args, **kwargs):
            given = host(tuple(args)), {k: host(v) for k, v in kwargs.items() if k != "residual_out"}
            result = fn(*args, **kwargs)
            cache = host(args[4]) if name == "rope_append" else None
            log.append(Call(name, *given, host(result), cache))
            return result
        return call

    for name in ("rms_norm", "gemm", "gemm_scaled", "rope_append", "attn_prompt", "attn_decode"):
        monkeypatch.setattr(w4, name, recorded(name, getattr(w4, name)))
    return log


# ------------------------------------------------------------------ the definitions


def same(a, b, what):
    assert a.shape == b.shape and a.dtype == b.dtype and torch.equal(a.view(torch.uint8), b.view(torch.uint8)), what


def check_norm(call, x, h, weight, a8):
    """Returns what a product takes and the residual stream."""
    assert call.name == "rms_norm"
    same(call.args[0], x, "norm of another input")
    same(call.args[1], weight, "another norm's weight")
    same(call.kwargs["residual"], h, "another residual stream")
    want, _ = ref.rms_norm(x, weight, h)
    new = call.result[-1]
    same(new, (x.float() + h.float()).to(x.dtype), "residual stream")
    K = x.shape[1]
    if not a8:
        ref.within(call.result[0], want, want.abs() * ref.norm_rel(K))
        return call.result[0], new
    codes, s, _ = call.result
    rel = 2 * ref.norm_rel(K)
    scale = want.abs().amax(1) / 127
    assert ((s.double() - scale).abs() <= rel * scale).all()
    assert ((codes.double() - want / scale[:, None]).abs() <= 0.5 + 127 * (rel + ref.E32)).all()
    return (codes, s), new


def check_gemm(call, x, pw, deq, silu=False):
    """x in 16 bits (with a8 quantized by the call), or codes and scales."""
    if isinstance(x, tuple):
        assert call.name == "gemm_scaled" and call.args[2] is pw
        same(call.args[0], x[0], "another input"), same(call.args[1], x[1], "other scales")
        a = x[0].double() * x[1].double()[:, None]
    else:
        assert call.name == "gemm" and call.args[1] is pw
        same(call.args[0], x, "another input")
        a = x.double()
        if call.kwargs.get("a8"):
            s = x.float().abs().amax(1) / 127
            s = torch.where(s > 0, s, torch.ones_like(s))
            a = (x.float() / s[:, None]).round().clamp(-127, 127).double() * s.double()[:, None]
    y = call.result
    u, K = ref.U[y.dtype], a.shape[1]
    want, mag = a @ deq, a.abs() @ deq.abs()
    tol = (u + (K + 8) * ref.E32) * mag  # a rounding of the weights, K additions
    assert bool(call.kwargs.get("silu_mul")) == silu
    if silu:
        tol = tol + u * want.abs()  # the two may be rounded before
        n = want.shape[1] // 2
        gate, up, tg, tu = want[:, :n], want[:, n:], tol[:, :n], tol[:, n:]
        want = gate * torch.sigmoid(gate)
        tol = 1.1 * tg * (up.abs() + tu) + want.abs() * (tu + 16 * ref.E32 * up.abs())  # |silu'| <= 1.1
        want = want * up
    ref.within(y, want, tol)
    return y


def check_rope(call, qkv, cos_sin, positions, placed, old, new):
    """q, and the cache's new tokens at their logical places `new` (sequence,
    token); the tokens there before are as they were."""
    assert call.name == "rope_append"
    same(call.args[0], qkv, "another qkv")
    assert torch.equal(call.args[1], cos_sin) and call.args[2].tolist() == positions
    H, hk, D = SHAPE.heads, SHAPE.kv_heads, SHAPE.head_dim
    x = qkv.view(len(qkv), H + 2 * hk, D)
    want = ref.rope(x[:, :H + hk], cos_sin, call.args[2], False)
    mag = x[:, :H + hk].double().abs().amax(2, keepdim=True) * 4 * ref.E32  # two products and a sum
    ref.within(call.result, want[:, :H], mag[:, :H].expand(-1, -1, D))
    after = placed(call.cache)
    for b, (k, v) in enumerate(old):
        n = k.shape[1]
        same(after[b][0][:, :n].contiguous(), k.contiguous(), "a key of an earlier token")
        same(after[b][1][:, :n].contiguous(), v.contiguous(), "a value of an earlier token")
    for i, t in enumerate((want[:, H:], x[:, H + hk:].double())):
        m = mag[:, H:] if i == 0 else torch.zeros_like(mag[:, H:])
        scale = (call.cache.k_scale, call.cache.v_scale)[i]
        got = torch.stack([after[b][i][:, token] for b, token in new])
        if scale is None:
            ref.within(got, t, m.expand_as(t))
            continue
        z = (t / scale.double()[:, None]).clamp(-448, 448)
        near = z.float().to(E4M3).double()
        # the nearest code; next to a midpoint of two codes either of them
        slack = 8 * ref.E32 * (z.abs() + m / scale.double()[:, None] / ref.E32)
        assert ((got.view(E4M3).double() - z).abs() <= (near - z).abs() + slack).all()
    return call.result, after


def check_attention(call, q, cache, table, starts, lens, zero, late):
    assert call.name in ("attn_prompt", "attn_decode")
    same(call.args[0], q, "other queries")
    if call.name == "attn_prompt":
        assert call.args[3].tolist() == starts
    assert call.args[-1].tolist() == lens
    for b, n in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        if lo == hi:
            continue
        out, _, tol, _ = ref.attention(q[lo:hi], cache, table[b], n, SHAPE.head_dim ** -0.5, n - (hi - lo) + late)
        ref.within(call.result[lo:hi], out * (not zero), tol)
    return call.result


class Walk:
    """The layers' order over the recorded calls. `mistake` plants one."""

    def __init__(self, stack, mistake=None):
        self.stack, self.mistake = stack, mistake
        self.table, self.cos_sin = host(stack.table), host(stack.cos_sin)
        if mistake == "page":
            self.table[2, [0, 1]] = self.table[2, [1, 0]]
        self.deq = [[host(w4.dequantize(pw, dtype=stack.dtype)).double() for pw in (l.qkv, l.o, l.gate_up, l.down)]
                    for l in stack.layers]
        self.lens = [0] * BATCH
        self.kept = [[(torch.empty(0),) * 2] * BATCH for _ in stack.layers]

    def placed(self, lens):
        def of(cache):
            """Bytes (or 16-bit values) of each sequence's keys and values: [kv heads, tokens, D]."""
            out = []
            for b, n in enumerate(lens):
                pages = self.table[b, : -(-n // PAGE)].long()
                kv = []
                for t in (cache.k, cache.v):
                    t = t.view(torch.uint8) if t.dtype == E4M3 else t
                    kv.append(t[pages].transpose(0, 1).reshape(t.shape[1], -1, t.shape[3])[:, :n])
                out.append(tuple(kv))
            return out
        return of

    def run(self, calls, x, counts, out):
        calls = iter(calls)
        a8, new = self.stack.a8, [(b, self.lens[b] + i) for b in range(BATCH) for i in range(counts[b])]
        before, self.lens = self.lens, [n + c for n, c in zip(self.lens, counts)]
        starts = [sum(counts[:b]) for b in range(BATCH + 1)]
        h = torch.zeros_like(x)
        for i, layer in enumerate(self.stack.layers):
            deq = self.deq[i]
            old = self.kept[i] if any(before) else []
            y, h = check_norm(next(calls), x, h, host(layer.norm1), a8)
            qkv = check_gemm(next(calls), y, layer.qkv, deq[0])
            call = next(calls)
            q, self.kept[i] = check_rope(call, qkv, self.cos_sin, [t for _, t in new], self.placed(self.lens), old, new)
            o = check_attention(next(calls), q, call.cache, self.table, starts, self.lens, self.mistake == "zero",
                                self.mistake == "late")
            x = check_gemm(next(calls), o.flatten(1), layer.o, deq[1])
            if self.mistake == "residual":
                h = torch.zeros_like(h)
            y, h = check_norm(next(calls), x, h, host(layer.norm2), a8)
            y = check_gemm(next(calls), y, layer.gate_up, deq[2], silu=True)
            x = check_gemm(next(calls), y, layer.down, deq[3])
        assert next(calls, None) is None
        same(out, (h.float() + x.float()).to(x.dtype), "hidden states")


MISTAKES = ["zero", "page", "late", "residual"]


@pytest.mark.parametrize("a8", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_every_call_is_its_definition(calls, dtype, e4m3, a8):
    stack = run_layer.Stack(SHAPE, LAYERS, BATCH, 256, page=PAGE, dtype=dtype, e4m3=e4m3, a8=a8, seed=1)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    runs = []
    for counts in ([20, 5, 100], [17, 0, 50], None, None):
        x = torch.randn((sum(counts) if counts else BATCH, SHAPE.hidden), generator=gen, device="cuda").to(dtype)
        given = host(x)
        del calls[:]
        out = stack.prompt(x, counts) if counts else stack.step(x)
        runs.append((list(calls), given, counts or [1] * BATCH, host(out)))
        same(host(x), given, "the input was changed")
    w4.device_status()
    walk = Walk(stack)
    for run in runs:
        walk.run(*run)
    for mistake in MISTAKES:
        with pytest.raises(AssertionError):
            walk = Walk(stack, mistake)
            for run in runs:
                walk.run(*run)
