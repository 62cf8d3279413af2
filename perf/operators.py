"""The operators around the W4A16 linears of a decoder layer, as measured cases.

Four operators: the root-mean-square norm with the residual's addition
(rms_norm), the rotation of queries and keys with the append to the paged
key-value cache (rope_append), the attention of one new token per sequence
over that cache (attn_decode) and the causal attention of prompts or pieces of
prompts over it (attn_prompt). ``own`` False computes them from elementary
torch operations in 32 bits, rounded once at the end; ``own`` True calls the
package's operators.
"""
import math

import torch

own = False

EPS = 1e-5
E4M3_MAX = 448.0
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one token of the 7B model: the norm before a projection, all latency
        norm("norm 1x4096", rows=1, width=4096),
        # a padded-out batch of the 13B model that goes on in 8 bits (W4A8)
        norm("norm codes 333x5120", rows=333, width=5120, dtype="bf16", quant="codes"),
        # a 4096-row prompt of the 70B model
        norm("norm 4096x8192", rows=4096, width=8192, dtype="bf16"),
        # one decode step of 16 sequences of the 7B model (32 heads, all with keys of their own)
        append("append 16 tokens", tokens=16, heads=32, kv_heads=32, page=16),
        # a ragged prompt of the 70B model (64 heads over 8) into an 8-bit cache
        append("append 4001 tokens e4m3", tokens=4001, heads=64, kv_heads=8, page=64, dtype="bf16", cache="e4m3"),
        # one user's next token early in a chat, 70B heads
        decode("decode 1x777", batch=1, longest=777, heads=64, kv_heads=8, page=16),
        # a batch of the 7B model at mixed lengths, one slot of it empty
        decode("decode 16x4096 ragged", batch=16, longest=4096, heads=32, kv_heads=32, page=16, dtype="bf16", ragged=True, lse=True),
        # a full serving batch of the 70B model
        decode("decode 64x8190", batch=64, longest=8190, heads=64, kv_heads=8, page=64),
        # few users with long documents in an 8-bit cache
        decode("decode 3x100003 e4m3", batch=3, longest=100003, heads=64, kv_heads=8, page=128, dtype="bf16", cache="e4m3"),
        # a short question to the 7B model
        prompt("prompt 1x37", batch=1, new=37, before=0, heads=32, kv_heads=32, page=16),
        # pieces of several 13B prompts, each behind what is cached of it
        prompt("prompt 5x700 behind 1500", batch=5, new=700, before=1500, heads=40, kv_heads=40, page=16, dtype="bf16", ragged=True, lse=True),
        # a long prompt of the 70B model
        prompt("prompt 1x8192", batch=1, new=8192, before=0, heads=64, kv_heads=8, page=64),
    ]


def norm(name, rows, width, dtype="fp16", quant="", residual=True):
    return named(name, op="norm", rows=rows, width=width, dtype=dtype, quant=quant, residual=residual)


def append(name, tokens, heads, kv_heads, page, dim=128, rotary=None, dtype="fp16", cache="", interleaved=False):
    return named(name, op="append", tokens=tokens, heads=heads, kv_heads=kv_heads, page=page, dim=dim, rotary=rotary or dim, dtype=dtype, cache=cache, interleaved=interleaved)


def decode(name, batch, longest, heads, kv_heads, page, dim=128, dtype="fp16", cache="", ragged=False, lse=False):
    return named(name, op="decode", batch=batch, longest=longest, heads=heads, kv_heads=kv_heads, page=page, dim=dim, dtype=dtype, cache=cache, ragged=ragged, lse=lse)


def prompt(name, batch, new, before, heads, kv_heads, page, dim=128, dtype="fp16", cache="", ragged=False, lse=False):
    return named(name, op="prompt", batch=batch, new=new, before=before, heads=heads, kv_heads=kv_heads, page=page, dim=dim, dtype=dtype, cache=cache, ragged=ragged, lse=lse)


def named(name, **case):
    return dict(case, name=name) if name else case


def log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case of the listed ones' ranges. Row and token counts are made odd."""
    dtype = rng.choice(["fp16", "bf16"])
    cache = rng.choice(["", "", "e4m3"])
    dim = rng.choice([64, 128, 128])
    group = rng.choice([1, 1, 2, 4, 5, 8, 8, 16])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 8, 32, 40])
    kv_heads = max(1, min(kv_heads, 80 // group))
    page = rng.choice([16, 16, 32, 64, 128])
    op = rng.choice(["norm", "append", "decode", "decode", "prompt", "prompt"])
    if op == "norm":
        width = rng.choice([128, 1000, 2560, 4096, 5120, 8192, 11008, 13824, 28672])
        rows = log_uniform(rng, 1, min(4095, (1 << 25) // width)) | 1
        return norm("", rows, width, dtype, rng.choice(["", "", "codes", "int8"]), rng.random() < 0.8)
    if op == "append":
        tokens = log_uniform(rng, 1, min(4095, (1 << 25) // ((group + 2) * kv_heads * dim))) | 1
        return append("", tokens, group * kv_heads, kv_heads, page, dim, rng.choice([dim, dim, dim // 2]), dtype, cache, rng.random() < 0.25)
    if op == "decode":
        batch = log_uniform(rng, 1, 128)
        longest = log_uniform(rng, 1, min(100001, (1 << 29) // (batch * kv_heads * dim))) | 1
        return decode("", batch, longest, group * kv_heads, kv_heads, page, dim, dtype, cache, rng.random() < 0.7, rng.random() < 0.5)
    batch = log_uniform(rng, 1, 8)
    new = log_uniform(rng, 1, 2047) | 1
    before = rng.choice([0, log_uniform(rng, 1, 4096)])
    scores = batch * new * (new + before) * group * kv_heads
    if scores > 1 << 31:  # no more than the longest listed prompt
        new = max(1, int(new * (1 << 31) / scores)) | 1
    return prompt("", batch, new, before, group * kv_heads, kv_heads, page, dim, dtype, cache, rng.random() < 0.7, rng.random() < 0.5)


# ------------------------------------------------------------------ lengths


def lengths(case):
    """Cached tokens of each sequence, the new ones among them, and the new ones of each."""
    n = case["batch"]
    if case["op"] == "decode":
        lens = [case["longest"]] * n
        if case["ragged"]:  # spread evenly down from the longest, in mixed order, the last slot empty
            lens = [max(1, case["longest"] * (n - (b * 7) % n) // n) for b in range(n)]
            if n > 2:
                lens[-1] = 0
        return lens, [1] * n
    new, before = [case["new"]] * n, [case["before"]] * n
    if case["ragged"]:
        new = [max(1, case["new"] * (n - b) // n) for b in range(n)]
        before = [case["before"] * (b + 1) // n for b in range(n)]
    return [a + b for a, b in zip(new, before)], new


def work(case):
    if case["op"] == "norm":
        size = case["rows"] * case["width"]
        out = {"": 2, "codes": 2, "int8": 1}[case["quant"]]
        return {"bytes": size * (2 + out + (4 if case["residual"] else 0)) + 2 * case["width"] + (4 * case["rows"] if case["quant"] else 0),
                "flops": 5 * size}
    code = 1 if case["cache"] else 2
    if case["op"] == "append":
        t, hq, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        return {"bytes": t * d * (2 * (hq + 2 * hk) + 2 * hq + 2 * hk * code) + t * (4 * case["rotary"] + 12),
                "flops": 3 * t * (hq + hk) * case["rotary"]}
    lens, new = lengths(case)
    cached = 2 * sum(lens) * case["kv_heads"] * case["dim"] * code
    rows = sum(new) * case["heads"]
    table = sum(-(-n // case["page"]) for n in lens) * 4 + 4 * len(lens)
    pairs = sum(n if case["op"] == "decode" else q * (n - q) + q * (q + 1) // 2 for n, q in zip(lens, new))
    return {"bytes": cached + 4 * rows * case["dim"] + (4 * rows if case["lse"] else 0) + table, "flops": 4 * pairs * case["heads"] * case["dim"]}


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)

    s = {"case": case}
    if case["op"] == "norm":
        rows, width = case["rows"], case["width"]
        s["x"] = normal(rows, width)
        # a residual stream as decoders have it: wide, a few channels far out
        r = torch.randn((rows, width), generator=gen, device="cuda") * 3
        r[:, :: 97] *= 20
        s["residual"] = r.to(dtype) if case["residual"] else None
        s["weight"] = (1 + 0.2 * torch.randn((width,), generator=gen, device="cuda")).to(dtype)
        return s
    hq, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    lens, new = ([case["tokens"]], None) if case["op"] == "append" else lengths(case)
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    if case["cache"]:
        s["k"], s["v"] = ((torch.randn((pages, hk, page, d), generator=gen, device="cuda") * 40).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn) for _ in "kv")
        s["k_scale"], s["v_scale"] = (0.02 + 0.02 * torch.rand((hk,), generator=gen, device="cuda") for _ in "kv")
    else:
        s["k"], s["v"] = normal(pages, hk, page, d), normal(pages, hk, page, d)
        s["k_scale"] = s["v_scale"] = None
    if case["op"] == "append":
        t, rot = case["tokens"], case["rotary"]
        s["qkv"] = normal(t, (hq + 2 * hk) * d)
        angle = torch.arange(t + 100, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["positions"] = torch.arange(100, t + 100, device="cuda", dtype=torch.int32)
        at = torch.arange(t, device="cuda")
        s["slots"] = order[at // page].long() * page + at % page
        return s
    s["table"] = torch.zeros((len(lens), max(max(counts), 1)), dtype=torch.int32, device="cuda")
    first = 0
    for b, n in enumerate(counts):
        s["table"][b, :n] = order[first:first + n]
        first += n
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["longest"] = max(lens)
    s["q"] = normal(sum(new), hq, d)
    if case["op"] == "prompt":
        s["starts"] = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32, device="cuda")
        s["most"] = max(new)
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    case = s["case"]
    if own:
        return run_own(s, case)
    return {"norm": plain_norm, "append": plain_append, "decode": plain_decode, "prompt": plain_prompt}[case["op"]](s, case)


def run_own(s, case):
    import bit_weight_only_g128_gb300 as w4

    if case["op"] == "norm":
        got = w4.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, quant=case["quant"] or None)
        return as_values(got, s["x"].dtype) if case["quant"] == "int8" else got
    cache = w4.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if case["op"] == "append":
        q = w4.rope_append(s["qkv"], s["cos_sin"], s["positions"], s["slots"], cache, interleaved=case["interleaved"])
        return q, s["k"], s["v"]
    if case["op"] == "decode":
        return w4.attn_decode(s["q"], cache, s["table"], s["lens"], return_lse=case["lse"])
    return w4.attn_prompt(s["q"], cache, s["table"], s["starts"], s["lens"], return_lse=case["lse"])


def as_values(got, dtype):
    """(codes, scales, ...) with the 8-bit codes as the values they stand for."""
    values = torch.empty(got[0].shape, dtype=dtype, device=got[0].device)
    torch.mul(got[0], got[1][:, None], out=values)
    return (values,) + tuple(got[1:])


def plain_norm(s, case):
    dtype = s["x"].dtype
    h = s["x"].float()
    if case["residual"]:
        h = h + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
    if not case["quant"]:
        return (y.to(dtype), h.to(dtype)) if case["residual"] else y.to(dtype)
    scale = y.abs().amax(1) / 127
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    codes = (y / scale[:, None]).round().clamp(-127, 127)
    more = (h.to(dtype),) if case["residual"] else ()
    if case["quant"] == "int8":
        return as_values((codes.to(torch.int8), scale) + more, dtype)
    return (codes.to(dtype), scale) + more


def rotate(x, cos_sin, positions, interleaved):
    """x [tokens, heads, dim] with its first rotary dimensions turned, in 32 bits."""
    rot = cos_sin.shape[1]
    turn = cos_sin[positions.long()][:, None]
    cos, sin = turn[..., : rot // 2], turn[..., rot // 2:]
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., : rot // 2], x[..., rot // 2: rot])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def plain_append(s, case):
    hq, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    x = s["qkv"].view(case["tokens"], hq + 2 * hk, d)
    turned = rotate(x[:, : hq + hk], s["cos_sin"], s["positions"], case["interleaved"])
    at, off = s["slots"] // page, s["slots"] % page
    store(s["k"], s["k_scale"], at, off, turned[:, hq:])
    store(s["v"], s["v_scale"], at, off, x[:, hq + hk:].float())
    return turned[:, :hq].to(x.dtype), s["k"], s["v"]


def store(cache, scale, at, off, x):
    if scale is None:
        cache[at, :, off] = x.to(cache.dtype)
    else:
        codes = (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(cache.dtype)
        cache.view(torch.uint8)[at, :, off] = codes.view(torch.uint8)


def gathered(cache, scale, table, dtype=torch.float32):
    """[batch, kv heads, tokens of the table's pages, dim] of the cache's values."""
    b, n = table.shape
    if scale is None:
        x = cache[table].to(dtype)
    else:
        x = cache.view(torch.uint8)[table].view(cache.dtype).to(dtype) * scale.to(dtype)[:, None, None]
    return x.transpose(1, 2).reshape(b, cache.shape[1], n * cache.shape[2], cache.shape[3])


def attend(q, k, v, seen):
    """q [b, kv heads, rows, d], k and v [b, kv heads, tokens, d], seen [b, 1, rows, tokens] or
    alike: the softmax-weighted values and the logarithm of the softmax's sum, in 32 bits."""
    x = torch.matmul(q, k.transpose(2, 3)).mul_(q.shape[-1] ** -0.5)
    x = x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = x.sum(-1, keepdim=True)
    y = torch.matmul(x, v) / torch.where(total > 0, total, torch.ones_like(total))
    return y, (top + total.log()).squeeze(-1)


def plain_decode(s, case):
    b, hq, hk, d = case["batch"], case["heads"], case["kv_heads"], case["dim"]
    k, v = (gathered(s[n], s[n + "_scale"], s["table"]) for n in "kv")
    seen = torch.arange(k.shape[2], device="cuda") < s["lens"][:, None]
    y, lse = attend(s["q"].float().view(b, hk, hq // hk, d), k, v, seen[:, None, None])
    y = y.view(b, hq, d).to(s["q"].dtype)
    return (y, lse.view(b, hq)) if case["lse"] else y


def plain_prompt(s, case):
    b, hq, hk, d, n = case["batch"], case["heads"], case["kv_heads"], case["dim"], s["most"]
    k, v = (gathered(s[x], s[x + "_scale"], s["table"]) for x in "kv")
    new = s["starts"].diff()
    row = torch.arange(n, device="cuda")
    at = (s["starts"][:-1, None] + row).clamp_(max=len(s["q"]) - 1).long()  # padded: [b, n]
    q = s["q"].float()[at].view(b, n, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    last = (s["lens"] - new)[:, None] + row
    seen = (torch.arange(k.shape[2], device="cuda") <= last[..., None]).repeat(1, hq // hk, 1)
    y, lse = attend(q, k, v, seen[:, None])
    y = y.view(b, hk, hq // hk, n, d).permute(0, 3, 1, 2, 4).reshape(b * n, hq, d)
    # back to the packed rows
    of = torch.repeat_interleave(torch.arange(b, device="cuda"), new.long(), output_size=len(s["q"]))
    back = of * n + torch.arange(len(s["q"]), device="cuda") - s["starts"][of]
    y = y[back].to(s["q"].dtype)
    lse = lse.view(b, hk, hq // hk, n).permute(0, 3, 1, 2).reshape(b * n, hq)[back]
    return (y, lse) if case["lse"] else y


# ------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": exact_norm, "append": exact_append, "decode": exact_attention, "prompt": exact_attention}[case["op"]](s, case)


def exact_norm(s, case):
    h = s["x"].double() + (s["residual"].double() if case["residual"] else 0)
    y = torch.einsum("mk,m,k->mk", h, (torch.einsum("mk,mk->m", h, h) / case["width"] + EPS) ** -0.5, s["weight"].double())
    if not case["quant"]:
        return (y, h) if case["residual"] else y
    scale = torch.linalg.vector_norm(y, math.inf, dim=1) / 127
    scale[scale == 0] = 1
    codes = torch.round(y / scale[:, None])
    codes = codes * scale[:, None] if case["quant"] == "int8" else codes
    return (codes, scale) + ((h,) if case["residual"] else ())


def exact_append(s, case):
    hq, hk, d, page, rot = case["heads"], case["kv_heads"], case["dim"], case["page"], case["rotary"]
    x = s["qkv"].double().view(-1, hq + 2 * hk, d)
    half = rot // 2
    turn = s["cos_sin"].double()[s["positions"].long()]
    turn = torch.complex(turn[:, :half], turn[:, half:])[:, None]
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, half), slice(half, rot))
    z = torch.complex(x[:, : hq + hk, first].contiguous(), x[:, : hq + hk, second].contiguous()) * turn
    y = x.clone()
    y[:, : hq + hk, first], y[:, : hq + hk, second] = z.real, z.imag
    out = [y[:, :hq].contiguous()]
    for name, heads in (("k", slice(hq, hq + hk)), ("v", slice(hq + hk, None))):
        whole = s[name].double()
        new = y[:, heads]
        if case["cache"]:  # held in 8 bits: the rounding to them is the operator's
            new = (new / s[name + "_scale"].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).double()
        flat = whole.transpose(1, 2).reshape(-1, hk, d)
        flat[s["slots"]] = new
        out.append(flat.view(-1, page, hk, d).transpose(1, 2).contiguous())
    return tuple(out)


def exact_attention(s, case):
    lens, new = lengths(case)
    if sum(n * q for n, q in zip(lens, new)) * case["heads"] > 3 << 31:
        return None
    hk, d = case["kv_heads"], case["dim"]
    group = case["heads"] // hk
    y = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    first = 0
    for b, (n, q) in enumerate(zip(lens, new)):
        rows = slice(first, first + q)
        first += q
        if n == 0:
            continue
        pages = s["table"][b: b + 1, : -(-n // case["page"])]
        k, v = (gathered(s[x], s[x + "_scale"], pages, torch.float64)[0, :, :n] for x in "kv")
        hidden = torch.ones((q, n), dtype=torch.bool, device="cuda").triu_(n - q + 1)
        for h in range(hk):
            heads = slice(h * group, (h + 1) * group)
            logits = torch.einsum("qgd,nd->gqn", s["q"][rows, heads].double(), k[h]) / math.sqrt(d)
            logits.masked_fill_(hidden, -math.inf)
            lse[rows, heads] = torch.logsumexp(logits, 2).T
            y[rows, heads] = torch.einsum("gqn,nd->qgd", torch.softmax(logits, 2), v[h])
    return (y, lse) if case["lse"] else y
