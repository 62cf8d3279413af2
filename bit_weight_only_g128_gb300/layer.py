"""The other operators of a decoder layer: what stands between its linears.

RMS norm with the residual's addition (and an 8-bit result for the W4A8
product), the rotation of queries and keys with the append to a paged
key-value cache, and the attention of single new tokens and of prompts over
that cache. As the rest of the binding: thin calls of the C ABI
(include/w4a16.h), no fallback, work on the current stream of the tensors'
device unless `stream` is given. Call them through the package
(``bit_weight_only_g128_gb300.rms_norm`` and so on).
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional

import torch

import bit_weight_only_g128_gb300 as w4

_HALF = torch.float16
_BF16 = torch.bfloat16
_E4M3 = torch.float8_e4m3fn


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


def _rows(t: torch.Tensor, name: str, cols: int, dtype: torch.dtype, device) -> int:
    """Row stride of a 2-D tensor [M, cols] with adjacent columns."""
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or t.shape[1] != cols:
        raise ValueError(f"{name} must have {cols} columns, got shape {tuple(t.shape)}")
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    return max(t.stride(0), cols) if t.shape[0] > 1 else cols


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
    if out is None:
        out = torch.empty((M, pw.N // 2 if silu_mul else pw.N), dtype=codes.dtype, device=dev)
    y_ptr = _flat(out, "out", M * (pw.N // 2 if silu_mul else pw.N), codes.dtype, dev)
    st = w4._stream(stream, dev.index)
    ws_ptr, ws_bytes = None, 0
    need = w4.workspace_size(M, pw.N, pw.K, pw.group, path, parts, silu_mul, False, dev.index)
    if need:
        if workspace is None:
            workspace = w4.stream_workspace(need, dev.index, st)
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    rc = w4.lib().w4a16_gemm_scaled(
        a_ptr, s_ptr, pw.Wq.data_ptr(), pw.Sp.data_ptr(), pw.Zp.data_ptr(), M, pw.N, pw.K, pw.group, y_ptr,
        ws_ptr, ws_bytes, w4._PATHS[path] | (w4.STATIC_WEIGHTS if static_weights else 0)
        | (w4.SILU_MUL if silu_mul else 0) | flags, parts, st)
    if rc:
        w4._check(rc, "w4a16_gemm_scaled")
    return out


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
    flags = _dtype16(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x must be [M, K], got shape {tuple(x.shape)}")
    M, K = x.shape
    dev, dt = x.device, x.dtype
    ldx = _rows(x, "x", K, dt, dev)
    w_ptr = _flat(weight, "weight", K, dt, dev)
    r_ptr, ldr, h_ptr, ldh, h = None, 0, None, 0, None
    if residual is not None:
        if residual.shape[0] != M:
            raise ValueError(f"residual has {residual.shape[0]} rows, x has {M}")
        ldr = _rows(residual, "residual", K, dt, dev)
        r_ptr = residual.data_ptr()
        h = residual_out if residual_out is not None else torch.empty((M, K), dtype=dt, device=dev)
        if h.shape[0] != M:
            raise ValueError(f"residual_out has {h.shape[0]} rows, x has {M}")
        ldh = _rows(h, "residual_out", K, dt, dev)
        h_ptr = h.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out goes with residual")
    y_ptr = codes_ptr = aq_ptr = s_ptr = scale = None
    if quant is None:
        y = out if out is not None else torch.empty((M, K), dtype=dt, device=dev)
        y_ptr = _flat(y, "out", M * K, dt, dev)
    elif quant in ("int8", "codes"):
        kind = torch.int8 if quant == "int8" else dt
        y = out if out is not None else torch.empty((M, K), dtype=kind, device=dev)
        ptr = _flat(y, "out", M * K, kind, dev)
        aq_ptr, codes_ptr = (ptr, None) if quant == "int8" else (None, ptr)
        scale = torch.empty((M,), dtype=torch.float32, device=dev)
        s_ptr = scale.data_ptr()
    else:
        raise ValueError(f"quant must be None, 'int8' or 'codes', got {quant!r}")
    rc = w4.lib().w4a16_rms_norm(x.data_ptr(), ldx, r_ptr, ldr, w_ptr, M, K, eps, flags, y_ptr, codes_ptr, aq_ptr,
                                 s_ptr, h_ptr, ldh, w4._stream(stream, dev.index))
    if rc:
        w4._check(rc, "w4a16_rms_norm")
    if quant is None:
        return y if h is None else (y, h)
    return (y, scale) if h is None else (y, scale, h)


def _cache_args(cache: KVCache, dt: torch.dtype, dev):
    """(k, v, k_scale, v_scale pointers, flags, shape) of a cache for 16-bit
    type dt on device dev."""
    k, v = cache.k, cache.v
    shape = k.shape
    if len(shape) != 4 or v.shape != shape:
        raise ValueError(f"cache k and v must be [pages, kv_heads, page_size, head_dim] alike, got {tuple(shape)} "
                         f"and {tuple(v.shape)}")
    if k.dtype is _E4M3:
        if cache.k_scale is None or cache.v_scale is None:
            raise ValueError("a float8_e4m3fn cache needs k_scale and v_scale")
        scales = (_flat(cache.k_scale, "k_scale", shape[1], torch.float32, dev),
                  _flat(cache.v_scale, "v_scale", shape[1], torch.float32, dev))
        flags = w4.CACHE_E4M3
    else:
        if cache.k_scale is not None or cache.v_scale is not None:
            raise ValueError("scales go with a float8_e4m3fn cache only")
        scales, flags = (None, None), 0
        if k.dtype is not dt:
            raise ValueError(f"the cache must be {dt} or float8_e4m3fn, got {k.dtype}")
    if v.dtype is not k.dtype or k.device != dev or v.device != dev or not k.is_cuda:
        raise ValueError(f"cache k and v must be CUDA tensors of one type on {dev}")
    if not k.is_contiguous() or not v.is_contiguous():
        raise ValueError("cache k and v must be contiguous")
    return (k.data_ptr(), v.data_ptr()) + scales, flags, shape


def rope_append(qkv: torch.Tensor, cos_sin: torch.Tensor, positions: torch.Tensor, slots: torch.Tensor,
                cache: KVCache, interleaved: bool = False, out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """Rotate the query and key heads of qkv [T, (heads + 2 kv_heads) *
    head_dim] by `positions` (int32 [T]) and append keys and values to
    `cache` at `slots` (int64 [T], page * page_size + place; negative: not
    stored). cos_sin float32 [table_len, rotary]: the cosines of a position's
    rotary/2 angles, then the sines. Returns the queries [T, heads, head_dim].
    """
    flags = _dtype16(qkv, "qkv")
    dev, dt = qkv.device, qkv.dtype
    ptrs, cache_flags, (pages, kv_heads, page_size, head_dim) = _cache_args(cache, dt, dev)
    if qkv.dim() != 2 or qkv.shape[1] % head_dim or qkv.shape[1] // head_dim <= 2 * kv_heads:
        raise ValueError(f"qkv must be [T, (heads + 2 * {kv_heads}) * {head_dim}], got shape {tuple(qkv.shape)}")
    T, cols = qkv.shape
    heads = cols // head_dim - 2 * kv_heads
    ld = _rows(qkv, "qkv", cols, dt, dev)
    if cos_sin.dim() != 2:
        raise ValueError(f"cos_sin must be [table_len, rotary], got shape {tuple(cos_sin.shape)}")
    table_len, rotary = cos_sin.shape
    t_ptr = _flat(cos_sin, "cos_sin", table_len * rotary, torch.float32, dev)
    p_ptr = _flat(positions, "positions", T, torch.int32, dev)
    s_ptr = _flat(slots, "slots", T, torch.int64, dev)
    if out is None:
        out = torch.empty((T, heads, head_dim), dtype=dt, device=dev)
    q_ptr = _flat(out, "out", T * heads * head_dim, dt, dev)
    rc = w4.lib().w4a16_rope_append(
        qkv.data_ptr(), ld, t_ptr, table_len, rotary, p_ptr, s_ptr, T, heads, kv_heads, head_dim, q_ptr, *ptrs,
        pages, page_size, flags | cache_flags | (w4.ROPE_INTERLEAVED if interleaved else 0),
        w4._stream(stream, dev.index))
    if rc:
        w4._check(rc, "w4a16_rope_append")
    return out


_ws_sizes = {}


def attn_workspace_size(tokens: int, batch: int, heads: int, kv_heads: int, head_dim: int,
                        device: Optional[int] = None) -> int:
    """Scratch bytes of an attn_decode (tokens = batch) or attn_prompt call on
    the current device (cached per device and arguments)."""
    dev = device if device is not None else (torch.cuda.current_device() if torch.cuda.is_available() else -1)
    key = (dev, tokens, batch, heads, kv_heads, head_dim)
    size = _ws_sizes.get(key)
    if size is None:
        b = ctypes.c_size_t()
        w4._check(w4.lib().w4a16_attn_workspace_size(tokens, batch, heads, kv_heads, head_dim, ctypes.byref(b)),
                  "w4a16_attn_workspace_size")
        size = _ws_sizes[key] = b.value
    return size


def _attend(q, cache, table, starts, lens, scale, out, return_lse, workspace, stream):
    flags = _dtype16(q, "q")
    dev, dt = q.device, q.dtype
    ptrs, cache_flags, (pages, kv_heads, page_size, head_dim) = _cache_args(cache, dt, dev)
    if q.dim() != 3 or q.shape[2] != head_dim:
        raise ValueError(f"q must be [tokens, heads, {head_dim}], got shape {tuple(q.shape)}")
    T, heads, _ = q.shape
    if q.stride(2) != 1 or (heads > 1 and q.stride(1) != head_dim):
        raise ValueError("q's heads must be adjacent")
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    ldq = max(q.stride(0), heads * head_dim) if T > 1 else heads * head_dim
    if table.dim() != 2:
        raise ValueError(f"table must be [batch, pages], got shape {tuple(table.shape)}")
    batch, max_pages = table.shape
    ldt = _rows(table, "table", max_pages, torch.int32, dev)
    if starts is None and T != batch:
        raise ValueError(f"q has {T} rows, the table {batch}")
    l_ptr = _flat(lens, "lens", batch, torch.int32, dev)
    c_ptr = None if starts is None else _flat(starts, "starts", batch + 1, torch.int32, dev)
    if out is None:
        out = torch.empty((T, heads, head_dim), dtype=dt, device=dev)
    o_ptr = _flat(out, "out", T * heads * head_dim, dt, dev)
    lse = torch.empty((T, heads), dtype=torch.float32, device=dev) if return_lse else None
    if scale is None:
        scale = head_dim ** -0.5
    st = w4._stream(stream, dev.index)
    ws_ptr, ws_bytes = None, 0
    need = attn_workspace_size(T, batch, heads, kv_heads, head_dim, dev.index)
    if need:
        if workspace is None:
            workspace = w4.stream_workspace(need, dev.index, st)
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    head = (q.data_ptr(), ldq, *ptrs, pages, page_size, table.data_ptr(), ldt, max_pages)
    tail = (heads, kv_heads, head_dim, scale, o_ptr, lse.data_ptr() if return_lse else None, ws_ptr, ws_bytes,
            flags | cache_flags, st)
    if starts is None:
        rc = w4.lib().w4a16_attn_decode(*head, l_ptr, batch, *tail)
    else:
        rc = w4.lib().w4a16_attn_prompt(*head, c_ptr, l_ptr, T, batch, *tail)
    if rc:
        w4._check(rc, "w4a16_attn_decode" if starts is None else "w4a16_attn_prompt")
    return (out, lse) if return_lse else out


def attn_decode(q: torch.Tensor, cache: KVCache, table: torch.Tensor, lens: torch.Tensor,
                scale: Optional[float] = None, out: Optional[torch.Tensor] = None, return_lse: bool = False,
                workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of one new token per sequence over the cache: q [batch,
    heads, head_dim] (rows may be strided), table int32 [batch, pages] the
    page numbers of each sequence, lens int32 [batch] its cached tokens (the
    new one among them; 0: zeros and -inf). scale defaults to
    head_dim^(-1/2). Returns out, or (out, lse) with lse float32 [batch,
    heads] the logarithm of the softmax's sum. `workspace` as for gemm."""
    return _attend(q, cache, table, None, lens, scale, out, return_lse, workspace, stream)


def attn_prompt(q: torch.Tensor, cache: KVCache, table: torch.Tensor, starts: torch.Tensor, lens: torch.Tensor,
                scale: Optional[float] = None, out: Optional[torch.Tensor] = None, return_lse: bool = False,
                workspace: Optional[torch.Tensor] = None, stream=None):
    """Causal attention of prompts, or pieces of prompts behind what is cached
    of them: q [T, heads, head_dim], sequence b has its rows starts[b] ..
    starts[b + 1) (int32 [batch + 1]) and lens[b] cached tokens, the new ones
    last and already appended. The rest as attn_decode."""
    return _attend(q, cache, table, starts, lens, scale, out, return_lse, workspace, stream)
