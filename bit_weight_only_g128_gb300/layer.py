"""The other operators of a decoder layer: what stands between its linears.

RMS norm with the residual's addition (and an 8-bit result for the W4A8
product), the rotation of queries and keys with the append to a paged
key-value cache, and the attention of single new tokens and of prompts over
that cache. As the rest of the binding: thin calls of the C ABI
(include/w4a16.h), no fallback, work on the current stream of the tensors'
device unless `stream` is given (results and workspaces then belong to it).
The calls' argument checks and allocations are native (csrc/binding.cpp): a
call costs the host about as much as its launch. Call them through the package
(``bit_weight_only_g128_gb300.rms_norm`` and so on).
"""
from __future__ import annotations

import ctypes
import dataclasses
import importlib.util
import os
from typing import NamedTuple, Optional

import torch

import bit_weight_only_g128_gb300 as w4

_HALF = torch.float16
_BF16 = torch.bfloat16


@dataclasses.dataclass
class KVCache:
    """A paged key-value cache: k and v [pages, kv_heads, page_size, head_dim],
    fp16, bf16, or float8_e4m3fn with a float32 scale per head (value = code *
    scale)."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: Optional[torch.Tensor] = None
    v_scale: Optional[torch.Tensor] = None

    @property
    def nbytes(self) -> int:
        return 2 * self.k.numel() * self.k.element_size()


def new_kv_cache(pages: int, kv_heads: int, page_size: int, head_dim: int, dtype: torch.dtype = torch.float16,
                 k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                 device=None) -> KVCache:
    """A zero-filled cache; float8_e4m3fn needs the scales (float32 [kv_heads])."""
    shape = (pages, kv_heads, page_size, head_dim)
    k, v = (torch.zeros(shape, dtype=dtype, device=device or "cuda") for _ in range(2))
    return KVCache(k, v, k_scale, v_scale)


def _flat(t: torch.Tensor, name: str, n: int, dtype: torch.dtype, device) -> int:
    """Pointer of a contiguous tensor of n elements."""
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with {n} elements, got shape {tuple(t.shape)}")
    return t.data_ptr()


def _dtype16(t: torch.Tensor, name: str) -> int:
    if t.dtype is _HALF:
        return 0
    if t.dtype is _BF16:
        return w4.BF16
    raise ValueError(f"{name} must be float16 or bfloat16, got {t.dtype}")


def gemm_scaled(codes: torch.Tensor, row_scale: torch.Tensor, pw, out: Optional[torch.Tensor] = None,
                path: str = "auto", parts: int = 0, workspace: Optional[torch.Tensor] = None, stream=None,
                static_weights: bool = False, silu_mul: bool = False) -> torch.Tensor:
    """Y [M, N] = row_scale * (codes . dequant(pw)): the product of
    ``gemm(..., a8=True)`` for activations that are 8-bit codes already
    (``rms_norm(..., quant="codes")``), held as fp16 or bf16 integer values."""
    M, K = codes.shape
    if K != pw.K:
        raise ValueError(f"codes have K={K}, weight has K={pw.K}")
    flags = _dtype16(codes, "codes")
    dev = codes.device
    a_ptr = _flat(codes, "codes", M * K, codes.dtype, dev)
    s_ptr = _flat(row_scale, "row_scale", M, torch.float32, dev)
    if stream is not None:
        with w4._on_stream(stream, dev):
            return gemm_scaled(codes, row_scale, pw, out, path, parts, workspace, None, static_weights, silu_mul)
    if dev.index != torch._C._cuda_getDevice():  # the library works on the current device
        with torch.cuda.device(dev):
            return gemm_scaled(codes, row_scale, pw, out, path, parts, workspace, None, static_weights, silu_mul)
    if out is None:
        out = torch.empty((M, pw.N // 2 if silu_mul else pw.N), dtype=codes.dtype, device=dev)
    y_ptr = _flat(out, "out", M * (pw.N // 2 if silu_mul else pw.N), codes.dtype, dev)
    st = w4._stream(None, dev.index)
    ws_ptr, ws_bytes = None, 0
    need = w4.workspace_size(M, pw.N, pw.K, pw.group, path, parts, silu_mul, False, dev.index)
    if need:
        if workspace is None:
            workspace = w4.stream_workspace(need, dev.index, st)
        ws_ptr, ws_bytes = w4._workspace_args(workspace, dev)
    rc = w4.lib().w4a16_gemm_scaled(
        a_ptr, s_ptr, pw.Wq.data_ptr(), pw.Sp.data_ptr(), pw.Zp.data_ptr(), M, pw.N, pw.K, pw.group, y_ptr,
        ws_ptr, ws_bytes, w4._PATHS[path] | (w4.STATIC_WEIGHTS if static_weights else 0)
        | (w4.SILU_MUL if silu_mul else 0) | flags, parts, st)
    if rc:
        w4._check(rc, "w4a16_gemm_scaled")
    return out


_native_module = None


def _native():
    """The native part of the binding, with the loaded library's entry points
    (raises if either has not been built)."""
    global _native_module
    if _native_module is None:
        from .build import BINDING, binding_version
        lib = w4.lib()
        if not os.path.exists(BINDING):
            raise ImportError(f"{BINDING} is missing: build it with `python -m bit_weight_only_g128_gb300.build`")
        if binding_version() != torch.__version__:
            raise ImportError(f"{BINDING} was compiled for another PyTorch ({binding_version() or 'unknown'}, this is "
                              f"{torch.__version__}): build it again")
        spec = importlib.util.spec_from_file_location("_binding", BINDING)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.bind(*[ctypes.cast(getattr(lib, "w4a16_" + name), ctypes.c_void_p).value for name in
                      ("rms_norm", "rope_append_norm", "attn_workspace_size", "attn_decode", "attn_prompt",
                       "route_workspace_size", "route", "experts_workspace_size", "gemm_experts")],
                    w4._check, w4.stream_workspace)
        _native_module = module
    return _native_module


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, eps: float = 1e-5,
             quant: Optional[str] = None, out: Optional[torch.Tensor] = None,
             residual_out: Optional[torch.Tensor] = None, stream=None):
    """y = h * (mean h^2 + eps)^(-1/2) * weight with h = x + residual, per row
    of x [M, K] (fp16 or bf16; rows may be strided).

    Returns y, or with `residual` (y, h), h the new residual stream
    (`residual_out`, which may be `residual` itself, or a new tensor). With
    `quant` y's place is taken by its 8-bit codes and their row scales
    (float32 [M], y ~ code * scale): "int8" as int8, "codes" as integer
    values of x's type, which gemm_scaled multiplies.
    """
    return (_native_module or _native()).rms_norm(x, weight, residual, eps, quant, out, residual_out, stream)


def rope_append(qkv: torch.Tensor, cos_sin: torch.Tensor, positions: torch.Tensor, slots: torch.Tensor,
                cache: KVCache, interleaved: bool = False, out: Optional[torch.Tensor] = None,
                stream=None, q_norm: Optional[torch.Tensor] = None, k_norm: Optional[torch.Tensor] = None,
                eps: float = 1e-5) -> torch.Tensor:
    """Rotate the query and key heads of qkv [T, (heads + 2 kv_heads) *
    head_dim] by `positions` (int32 [T]) and append keys and values to
    `cache` at `slots` (int64 [T], page * page_size + place; negative: not
    stored). cos_sin float32 [table_len, rotary]: the cosines of a position's
    rotary/2 angles, then the sines. Returns the queries [T, heads, head_dim].

    With `q_norm` and `k_norm` (each [head_dim] of qkv's type, or None) every
    query (key) head is x * (mean x^2 + eps)^(-1/2) * weight before its
    rotation, in the same pass.
    """
    native = _native_module or _native()
    if q_norm is None and k_norm is None:
        return native.rope_append(qkv, cos_sin, positions, slots, cache, interleaved, out, stream)
    return native.rope_append(qkv, cos_sin, positions, slots, cache, interleaved, out, stream, q_norm, k_norm, eps)


def attn_workspace_size(tokens: int, batch: int, heads: int, kv_heads: int, head_dim: int) -> int:
    """Scratch bytes of an attn_decode (tokens = batch) or attn_prompt call on
    the current device."""
    b = ctypes.c_size_t()
    w4._check(w4.lib().w4a16_attn_workspace_size(tokens, batch, heads, kv_heads, head_dim, ctypes.byref(b)),
              "w4a16_attn_workspace_size")
    return b.value


def attn_decode(q: torch.Tensor, cache: KVCache, table: torch.Tensor, lens: torch.Tensor,
                scale: Optional[float] = None, out: Optional[torch.Tensor] = None, return_lse: bool = False,
                workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of one new token per sequence over the cache: q [batch,
    heads, head_dim] (rows may be strided), table int32 [batch, pages] the
    page numbers of each sequence, lens int32 [batch] its cached tokens (the
    new one among them; 0: zeros and -inf). scale defaults to
    head_dim^(-1/2). Returns out, or (out, lse) with lse float32 [batch,
    heads] the logarithm of the softmax's sum. `workspace` as for gemm."""
    return (_native_module or _native()).attend(q, cache, table, None, lens, scale, out, return_lse, workspace, stream)


def attn_prompt(q: torch.Tensor, cache: KVCache, table: torch.Tensor, starts: torch.Tensor, lens: torch.Tensor,
                scale: Optional[float] = None, out: Optional[torch.Tensor] = None, return_lse: bool = False,
                workspace: Optional[torch.Tensor] = None, stream=None):
    """Causal attention of prompts, or pieces of prompts behind what is cached
    of them: q [T, heads, head_dim], sequence b has its rows starts[b] ..
    starts[b + 1) (int32 [batch + 1]) and lens[b] cached tokens, the new ones
    last and already appended. The rest as attn_decode."""
    return (_native_module or _native()).attend(q, cache, table, starts, lens, scale, out, return_lse, workspace, stream)


# ------------------------------------------------------------------ experts


@dataclasses.dataclass
class PackedExperts:
    """The packed int4 weights of a layer's experts, all K x N: the buffers of
    one expert (PackedWeight) after those of another."""
    Wq: torch.Tensor       # int32 [experts * K*N/8]
    Sp: torch.Tensor       # float16 [experts * K/group * N]
    Zp: torch.Tensor       # int32 [experts * K/group * N / 8]
    experts: int
    K: int
    N: int
    group: int

    @property
    def nbytes(self) -> int:
        return self.Wq.numel() * 4 + self.Sp.numel() * 2 + self.Zp.numel() * 4

    def expert(self, e: int):
        """Expert e as a PackedWeight (the same memory)."""
        if not 0 <= e < self.experts:
            raise IndexError(f"expert {e} of {self.experts}")
        return w4.PackedWeight(*(t.view(self.experts, -1)[e] for t in (self.Wq, self.Sp, self.Zp)), self.K, self.N,
                               self.group)


def stack_experts(weights) -> PackedExperts:
    """The PackedWeights of experts, alike in K, N and group, as one (copied)."""
    weights = list(weights)
    if not weights:
        raise ValueError("no experts")
    first = weights[0]
    for w in weights:
        if (w.K, w.N, w.group) != (first.K, first.N, first.group):
            raise ValueError(f"experts differ: {w.K} x {w.N} group {w.group} beside {first.K} x {first.N} group "
                             f"{first.group}")
    return PackedExperts(*(torch.cat([getattr(w, n) for w in weights]) for n in ("Wq", "Sp", "Zp")), len(weights),
                         first.K, first.N, first.group)


class Routing(NamedTuple):
    """What route answers and gemm_experts takes. A choice is token * top_k +
    j, the j-th expert of a token."""
    experts: torch.Tensor  # int32 [T, top_k], descending; -1: none
    weights: torch.Tensor  # float32 [T, top_k]
    rows: torch.Tensor     # int32 [T * top_k]: the choices by expert, those of none last
    offsets: torch.Tensor  # int32 [experts + 1]: expert e's are rows[offsets[e]:offsets[e + 1]]


def route(logits: torch.Tensor, top_k: int, scoring: str = "softmax", renormalize: bool = True,
          workspace: Optional[torch.Tensor] = None, stream=None) -> Routing:
    """The router: of logits [T, experts] (fp16, bf16 or fp32; rows may be
    strided) each token's top_k largest, in descending order, equal ones by
    the lower index, their weights (softmax over all experts, or "sigmoid" of
    each; with `renormalize` divided by the chosen ones' sum) and the choices
    by expert. A logit of -inf is never chosen: its place has expert -1 and
    weight 0 (a row of -inf, for a padded token, chooses no expert).
    `workspace` as for gemm."""
    return Routing(*(_native_module or _native()).route(logits, top_k, scoring, renormalize, workspace, stream))


def experts_workspace_size(T: int, top_k: int, pe: PackedExperts, silu_mul: bool = False, combine: bool = False,
                           path: str = "auto") -> int:
    """Scratch bytes of a gemm_experts call on the current device."""
    b = ctypes.c_size_t()
    flags = w4._PATHS[path] | (w4.SILU_MUL if silu_mul else 0) | (w4.EXPERTS_COMBINE if combine else 0)
    w4._check(w4.lib().w4a16_experts_workspace_size(T, top_k, pe.experts, pe.N, pe.K, pe.group, flags, ctypes.byref(b)),
              "w4a16_experts_workspace_size")
    return b.value


def gemm_experts(A: torch.Tensor, pe: PackedExperts, routing: Routing, silu_mul: bool = False, combine: bool = False,
                 out: Optional[torch.Tensor] = None, path: str = "auto", workspace: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """Every token's rows times its experts' weights, grouped by expert.

    A [T, K] gives each of a token's choices the token's row, A [T, top_k, K]
    a row of its own (fp16 or bf16). Returns Y [T, top_k, N], choice (t, j)
    times expert routing.experts[t, j] (zeros where that is -1); with
    `silu_mul` (pe's columns are [gate | up]) silu(gate) * up, [T, top_k,
    N/2]; with `combine` the sum over j weighted by routing.weights, [T, N].
    `path`: "auto", "decode" (few rows per expert: weights unrounded) or
    "tensor-pair" (many: weights rounded once to A's type). `workspace` as for
    gemm."""
    return (_native_module or _native()).gemm_experts(A, pe, routing, silu_mul, combine, out, w4._PATHS[path], workspace,
                                                      stream)
