"""The operators of a decoder layer whose MLP is made of experts, as measured cases.

Three operators: the router (route: the experts of every token, their weights,
and the rows in the experts' order), the W4A16 products grouped by expert
(gemm_experts: gate and up with their activation fused, or down with the
weighted sum over a token's experts), and the norm of every query and key head
in the pass that rotates them and appends to the cache (rope_append with
q_norm and k_norm). ``own`` False computes them from elementary torch
operations in 32 bits, rounded once at the end; ``own`` True calls the
package's operators.
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # the next token of one user: the router, all latency
        route("route 1x64", tokens=1, experts=64, top=8),
        # a prompt's tokens, some rows of it padding
        route("route 4099x64 padded", tokens=4099, experts=64, top=8, padded=True),
        # a decode step of 16 sequences, all heads with keys of their own
        append("norms append 16 tokens", tokens=16, heads=32, kv_heads=32, page=16),
        # a ragged prompt with grouped heads into an 8-bit cache
        append("norms append 4001 tokens", tokens=4001, heads=64, kv_heads=8, page=64, dtype="bf16", cache="e4m3"),
        # the next token of one user, many small experts: gate and up, then down
        product("gate_up 1 of 64x8", tokens=1, experts=64, top=8, k=2048, n=2048, silu=True),
        product("down 1 of 64x8", tokens=1, experts=64, top=8, k=1024, n=2048),
        # a decode step of a small batch: most experts have a row or two
        product("gate_up 16 of 64x8", tokens=16, experts=64, top=8, k=2048, n=2048, silu=True, dtype="bf16"),
        # a decode step with few experts as large as the 7B model's MLP
        product("gate_up 32 of 8x2", tokens=32, experts=8, top=2, k=4096, n=22016, silu=True),
        # a large batch's decode step, about a dozen rows for each expert
        product("down 100 of 64x8", tokens=100, experts=64, top=8, k=1024, n=2048, dtype="bf16"),
        # prompts: gate and up of many small experts, down of the same
        product("gate_up 4099 of 64x8", tokens=4099, experts=64, top=8, k=2048, n=2048, silu=True, dtype="bf16"),
        product("down 4099 of 64x8", tokens=4099, experts=64, top=8, k=1024, n=2048),
        # a prompt through few experts as large as the 7B model's MLP
        product("down 2047 of 8x2", tokens=2047, experts=8, top=2, k=11008, n=4096),
    ]


def route(name, tokens, experts, top, dtype="fp32", scoring="softmax", renormalize=True, padded=False):
    return named(name, op="route", tokens=tokens, experts=experts, top=top, dtype=dtype, scoring=scoring, renormalize=renormalize, padded=padded)


def append(name, tokens, heads, kv_heads, page, dim=128, rotary=None, dtype="fp16", cache="", interleaved=False):
    return named(name, op="append", tokens=tokens, heads=heads, kv_heads=kv_heads, page=page, dim=dim, rotary=rotary or dim, dtype=dtype, cache=cache, interleaved=interleaved)


def product(name, tokens, experts, top, k, n, silu=False, group=128, dtype="fp16"):
    """Gate and up (silu: n columns in, n / 2 out, one row of A per token) or down (one row of A per choice, summed per token)."""
    return named(name, op="product", tokens=tokens, experts=experts, top=top, k=k, n=n, silu=silu, group=group, dtype=dtype)


def named(name, **case):
    return dict(case, name=name) if name else case


def log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case of the listed ones' ranges."""
    op = rng.choice(["route", "append", "product", "product", "product"])
    dtype = rng.choice(["fp16", "bf16"])
    experts = rng.choice([4, 8, 16, 60, 64, 128, 160])
    top = rng.choice([1, 2, 2, 4, 6, 8, 8])
    top = min(top, experts)
    if op == "route":
        tokens = log_uniform(rng, 1, 4099) | 1
        return route("", tokens, experts, top, rng.choice(["fp32", "fp32", "fp16", "bf16"]), rng.choice(["softmax", "softmax", "sigmoid"]), rng.random() < 0.7, rng.random() < 0.3)
    if op == "append":
        dim = rng.choice([64, 128, 128])
        group = rng.choice([1, 1, 2, 4, 5, 8, 8, 16])
        kv_heads = max(1, min(rng.choice([1, 2, 4, 5, 8, 8, 32, 40]), 80 // group))
        tokens = log_uniform(rng, 1, min(4001, (1 << 25) // ((group + 2) * kv_heads * dim))) | 1
        return append("", tokens, group * kv_heads, kv_heads, rng.choice([16, 16, 32, 64, 128]), dim, rng.choice([dim, dim, dim // 2]), dtype, rng.choice(["", "", "e4m3"]), rng.random() < 0.25)
    k, group = rng.choice([(512, 128), (1024, 128), (1408, 64), (2048, 128), (2048, 2048), (4096, 128), (5120, 128), (704, 64), (11008, 128)])
    silu = rng.random() < 0.5
    n = rng.choice([1056, 2048, 2080, 4096, 5120, 8160, 22016]) if silu else rng.choice([1040, 2000, 2048, 4096, 5120, 8192])
    while experts > 2 and experts * k * n > 3 << 28:  # hardly more weights than the largest listed experts have
        experts //= 2
    top = min(top, experts)
    # no more products than the longest listed prompt has
    tokens = log_uniform(rng, 1, max(1, min(4099, int(1.3e11 / (top * k * n))))) | 1
    return product("", tokens, experts, top, k, n, silu, group, dtype)


def work(case):
    t = case["tokens"]
    if case["op"] == "route":
        e, k = case["experts"], case["top"]
        return {"bytes": t * e * (4 if case["dtype"] == "fp32" else 2) + 12 * t * k + 4 * (e + 1), "flops": 5 * t * e}
    if case["op"] == "append":
        hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
        code = 1 if case["cache"] else 2
        return {"bytes": t * d * (2 * (hq + 2 * hk) + 2 * hq + 2 * hk * code) + t * (4 * case["rotary"] + 12) + 4 * d,
                "flops": t * (hq + hk) * (3 * case["rotary"] + 4 * d)}
    e, top, k, n = case["experts"], case["top"], case["k"], case["n"]
    used = e * (1 - (1 - top / e) ** t)  # experts that have a row, on average
    weights = used * k * n * (0.5 + 2.5 / case["group"])
    rows = t * k * 2 + t * top * n if case["silu"] else t * top * k * 2 + t * n * 2
    return {"bytes": weights + rows + 8 * t * top + 4 * (e + 1), "flops": 2 * t * top * k * n}


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    {"route": prepare_route, "append": prepare_append, "product": prepare_product}[case["op"]](s, case, gen)
    return s


def router_logits(case, gen):
    """Logits as routers give them: some experts are liked more than others."""
    liked = torch.randn((1, case["experts"]), generator=gen, device="cuda") * 0.5
    return torch.randn((case["tokens"], case["experts"]), generator=gen, device="cuda") + liked


def prepare_route(s, case, gen):
    s["logits"] = router_logits(case, gen).to(DTYPES[case["dtype"]])
    if case["padded"]:  # rows behind their sequences' ends: no expert may be chosen
        s["logits"][torch.rand((case["tokens"],), generator=gen, device="cuda") < 0.125] = -math.inf


def prepare_append(s, case, gen):
    dtype = DTYPES[case["dtype"]]
    t, hq, hk, d, page, rot = case["tokens"], case["heads"], case["kv_heads"], case["dim"], case["page"], case["rotary"]
    pages = -(-t // page) + 3
    order = torch.randperm(pages, generator=gen, device="cuda")
    if case["cache"]:
        s["k"], s["v"] = ((torch.randn((pages, hk, page, d), generator=gen, device="cuda") * 40).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn) for _ in "kv")
        s["k_scale"], s["v_scale"] = (0.02 + 0.02 * torch.rand((hk,), generator=gen, device="cuda") for _ in "kv")
    else:
        s["k"], s["v"] = (torch.randn((pages, hk, page, d), generator=gen, device="cuda").to(dtype) for _ in "kv")
        s["k_scale"] = s["v_scale"] = None
    s["qkv"] = (torch.randn((t, (hq + 2 * hk) * d), generator=gen, device="cuda") * 2).to(dtype)
    s["q_norm"], s["k_norm"] = ((1 + 0.2 * torch.randn((d,), generator=gen, device="cuda")).to(dtype) for _ in "qk")
    angle = torch.arange(t + 100, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    s["positions"] = torch.arange(100, t + 100, device="cuda", dtype=torch.int32)
    at = torch.arange(t, device="cuda")
    s["slots"] = order[at // page] * page + at % page


def prepare_product(s, case, gen):
    dtype = DTYPES[case["dtype"]]
    t, e, top, k, n, group = case["tokens"], case["experts"], case["top"], case["k"], case["n"], case["group"]
    logits = router_logits(case, gen)
    s["experts"], s["weights"], s["rows"], s["offsets"] = chosen(logits, top, "softmax", True)
    s["most"] = int(s["offsets"].diff().max())  # rows of the expert that has most: a plan of the plain form
    s["a"] = torch.randn((t, k) if case["silu"] else (t, top, k), generator=gen, device="cuda").to(dtype)
    # weights quantized per group of input channels, as codes, scales and zero points, and packed
    s["q"] = torch.empty((e, k, n), dtype=torch.uint8, device="cuda")
    s["s"] = torch.empty((e, k // group, n), dtype=torch.float16, device="cuda")
    s["z"] = torch.empty((e, k // group, n), dtype=torch.uint8, device="cuda")
    s["Wq"] = torch.empty((e, n // 16, k // 64, 8, 4, 2, 2), dtype=torch.int32, device="cuda")
    for i in range(e):
        w = (torch.randn((k, n), generator=gen, device="cuda") * 0.02).view(k // group, group, n)
        lo, hi = w.amin(1, keepdim=True), w.amax(1, keepdim=True)
        scale = ((hi - lo) / 15).half().float()
        zero = (-lo / scale).round().clamp(0, 15)
        code = ((w / scale).round() + zero).clamp(0, 15).to(torch.uint8).view(k, n)
        s["q"][i], s["s"][i], s["z"][i] = code, scale[:, 0].half(), zero[:, 0].to(torch.uint8)
        # strips of 16 columns, atoms of 64 rows: [strip, atom, g, t, s, r] words of eight codes
        x = code.view(k // 64, 2, 4, 8, n // 16, 2, 8).permute(4, 0, 6, 2, 1, 5, 3).int()
        s["Wq"][i] = sum(x[..., b] << 4 * int(f"{b:03b}"[::-1], 2) for b in range(8))
    s["Sp"] = s["s"].view(e, k // group, n // 16, 2, 8).permute(0, 2, 1, 4, 3).contiguous().view(-1)
    x = s["z"].view(e, k // group, n // 16, 2, 8).permute(0, 2, 1, 3, 4)
    s["Zp"] = (x[..., 0, :] | x[..., 1, :] << 4).contiguous().view(-1).view(torch.int32)
    s["Wq"] = s["Wq"].view(-1)


def chosen(logits, top, scoring, renormalize):
    """Experts, weights, rows by expert and offsets, in 32 bits."""
    x = logits.float()
    e = x.shape[1]
    best, experts = torch.sort(x, dim=1, descending=True, stable=True)
    best, experts = best[:, :top], experts[:, :top]
    if scoring == "softmax":
        highest = best[:, :1].masked_fill(best[:, :1] == -math.inf, 0)
        score, total = (best - highest).exp(), (x - highest).exp().sum(1, keepdim=True)
    else:
        score, total = 1 / (1 + (-best).exp()), torch.ones_like(best[:, :1])
    if renormalize:
        total = score.sum(1, keepdim=True)
    none = best == -math.inf
    weights = (score / total).masked_fill(none, 0)
    experts = experts.masked_fill(none, -1)
    flat = experts.flatten()
    rows = torch.sort(flat.masked_fill(flat < 0, e), stable=True)[1]
    offsets = torch.zeros(e + 1, dtype=torch.int64, device=x.device)
    offsets[1:] = (flat[:, None] == torch.arange(e, device=x.device)).sum(0).cumsum(0)
    return experts.int(), weights, rows.int(), offsets.int()


# ------------------------------------------------------------------ one pass


def run(s):
    case = s["case"]
    if own:
        return run_own(s, case)
    return {"route": plain_route, "append": plain_append, "product": plain_product}[case["op"]](s, case)


def run_own(s, case):
    import bit_weight_only_g128_gb300 as w4

    if case["op"] == "route":
        got = w4.route(s["logits"], case["top"], scoring=case["scoring"], renormalize=case["renormalize"])
        return got.experts, got.weights, got.rows, got.offsets
    if case["op"] == "append":
        cache = w4.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        q = w4.rope_append(s["qkv"], s["cos_sin"], s["positions"], s["slots"], cache, interleaved=case["interleaved"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
        return q, s["k"], s["v"]
    weights = w4.PackedExperts(s["Wq"], s["Sp"], s["Zp"], case["experts"], case["k"], case["n"], case["group"])
    routing = w4.Routing(s["experts"], s["weights"], s["rows"], s["offsets"])
    return w4.gemm_experts(s["a"], weights, routing, silu_mul=case["silu"], combine=not case["silu"])


def plain_route(s, case):
    return chosen(s["logits"], case["top"], case["scoring"], case["renormalize"])


def plain_append(s, case):
    hq, hk, d, page, rot = case["heads"], case["kv_heads"], case["dim"], case["page"], case["rotary"]
    x = s["qkv"].view(case["tokens"], hq + 2 * hk, d).float()
    y = x[:, : hq + hk]
    y = y * torch.rsqrt(y.square().mean(2, keepdim=True) + EPS)
    y = torch.cat([y[:, :hq] * s["q_norm"].float(), y[:, hq:] * s["k_norm"].float()], 1)
    turn = s["cos_sin"][s["positions"].long()][:, None]
    cos, sin = turn[..., : rot // 2], turn[..., rot // 2:]
    inter = case["interleaved"]
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if inter else (y[..., : rot // 2], y[..., rot // 2: rot])
    u, v = a * cos - b * sin, b * cos + a * sin
    y = torch.cat([torch.stack([u, v], -1).flatten(-2) if inter else torch.cat([u, v], -1), y[..., rot:]], -1)
    at, off = s["slots"] // page, s["slots"] % page
    store(s["k"], s["k_scale"], at, off, y[:, hq:])
    store(s["v"], s["v_scale"], at, off, x[:, hq + hk:])
    return y[:, :hq].to(s["qkv"].dtype), s["k"], s["v"]


def store(cache, scale, at, off, x):
    if scale is None:
        cache[at, :, off] = x.to(cache.dtype)
    else:
        codes = (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(cache.dtype)
        cache.view(torch.uint8)[at, :, off] = codes.view(torch.uint8)


def plain_product(s, case):
    t, e, top, k, n, group = case["tokens"], case["experts"], case["top"], case["k"], case["n"], case["group"]
    if t * top <= e:  # a product of its own for every choice
        of = s["experts"].flatten().long()
        q, scale, zero = s["q"][of], s["s"][of], s["z"][of]
    else:  # all experts, each with as many rows as the one that has most
        q, scale, zero = s["q"], s["s"], s["z"]
        place = torch.arange(s["most"], device="cuda")
        at = (s["offsets"][:-1, None] + place).clamp_(max=t * top - 1)
        live = place < s["offsets"].diff()[:, None]
    b = len(q)
    w = (q.view(b, k // group, group, n).float() - zero[:, :, None].float()) * scale[:, :, None].float()
    w = w.view(b, k, n)
    a = s["a"].float()
    a = a[:, None].expand(t, top, k).reshape(t * top, k) if case["silu"] else a.view(t * top, k)
    if t * top <= e:
        y = torch.bmm(a[:, None], w).view(t * top, n)
    else:
        rows = s["rows"].long()[at]
        y = torch.empty((t * top, n), dtype=torch.float32, device="cuda")
        y[rows[live]] = torch.bmm(a[rows], w)[live]
    if case["silu"]:
        gate, up = y[:, : n // 2], y[:, n // 2:]
        return (gate / (1 + (-gate).exp()) * up).view(t, top, n // 2).to(s["a"].dtype)
    return (y.view(t, top, n) * s["weights"][..., None]).sum(1).to(s["a"].dtype)


# ------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    if case["op"] == "product" and case["tokens"] * case["top"] * case["k"] * case["n"] > 1 << 42:
        return None
    s = prepare(case, seed)
    return {"route": exact_route, "append": exact_append, "product": exact_product}[case["op"]](s, case)


def exact_route(s, case):
    x = s["logits"].double()
    t, e = x.shape
    left, experts, best = x.clone(), [], []
    for _ in range(case["top"]):  # the largest that is left, the first of equals
        value = left.amax(1, keepdim=True)
        index = (left == value).int().argmax(1, keepdim=True)
        experts.append(index.masked_fill(value == -math.inf, -1))
        best.append(value)
        left.scatter_(1, index, -math.inf)
    experts, best = torch.cat(experts, 1), torch.cat(best, 1)
    p = torch.softmax(x, 1) if case["scoring"] == "softmax" else torch.sigmoid(x)
    weights = torch.where(experts < 0, 0.0, torch.gather(p, 1, experts.clamp(min=0)))
    if case["renormalize"]:
        total = weights.sum(1, keepdim=True)
        weights = weights / torch.where(total > 0, total, 1.0)
    place = torch.arange(t * case["top"], device="cuda")
    key = torch.where(experts < 0, e, experts).flatten() * (t * case["top"]) + place
    rows = torch.argsort(key)
    offsets = torch.searchsorted(key[rows], torch.arange(e + 1, device="cuda") * (t * case["top"]))
    return experts.int(), weights, rows.int(), offsets.int()


def exact_append(s, case):
    hq, hk, d, page, rot = case["heads"], case["kv_heads"], case["dim"], case["page"], case["rotary"]
    y = s["qkv"].double().view(-1, hq + 2 * hk, d).clone()
    for heads, weight in ((slice(0, hq), s["q_norm"]), (slice(hq, hq + hk), s["k_norm"])):
        x = y[:, heads]
        y[:, heads] = torch.einsum("thd,th,d->thd", x, (torch.einsum("thd,thd->th", x, x) / d + EPS) ** -0.5, weight.double())
    half = rot // 2
    turn = s["cos_sin"].double()[s["positions"].long()]
    turn = torch.complex(turn[:, :half], turn[:, half:])[:, None]
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, half), slice(half, rot))
    z = torch.complex(y[:, : hq + hk, first].contiguous(), y[:, : hq + hk, second].contiguous()) * turn
    y[:, : hq + hk, first], y[:, : hq + hk, second] = z.real, z.imag
    out = [y[:, :hq].contiguous()]
    for name, heads in (("k", slice(hq, hq + hk)), ("v", slice(hq + hk, None))):
        new = y[:, heads]
        if case["cache"]:  # held in 8 bits: the rounding to them is the operator's
            new = (new / s[name + "_scale"].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).double()
        flat = s[name].double().transpose(1, 2).reshape(-1, hk, d)
        flat[s["slots"]] = new
        out.append(flat.view(-1, page, hk, d).transpose(1, 2).contiguous())
    return tuple(out)


def exact_product(s, case):
    t, top, k, n, group = case["tokens"], case["top"], case["k"], case["n"], case["group"]
    y = torch.zeros((t, top, n), dtype=torch.float64, device="cuda")
    a = s["a"].double() if not case["silu"] else s["a"].double()[:, None].expand(t, top, k)
    for e in range(case["experts"]):
        token, place = torch.nonzero(s["experts"] == e, as_tuple=True)
        if len(token):
            code = s["q"][e].double() - s["z"][e].double().repeat_interleave(group, 0)
            y[token, place] = a[token, place] @ (code * s["s"][e].double().repeat_interleave(group, 0))
    if case["silu"]:
        return torch.nn.functional.silu(y[..., : n // 2]) * y[..., n // 2:]
    return torch.einsum("tjn,tj->tn", y, s["weights"].double())
