"""Timed cases of the operators around a paged cache held in 4 bits: appending keys
and values, attention of new tokens over it, reading ranges of a quantised cache back,
and joining two partial attentions.

``run`` computes an operator from elementary torch operations, or (``own``)
through the library's public entry points.

The 4-bit cache: uint8 codes [num_pages, H_kv, page_size, d / 2], element 2 i of a row in
the low half of byte i (e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), and one
bfloat16 descale per row [num_pages, H_kv, page_size].
"""
from __future__ import annotations

import functools
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------- cases ----
def listed():
    return [
        # one decode step: a token of each request written, and read back
        dict(name="append_step", op="append", B=64, new=1, prefill=0, ctx=2048, page=64, H=32, H_kv=8, d=128,
             rot=128, dtype="bf16", signs=True, interleaved=False),
        # two long prompts among a decode batch: the bulk of a cache's writing
        dict(name="append_prompts", op="append", B=16, new=1, prefill=8192, ctx=2048, page=256, H=32, H_kv=8,
             d=128, rot=128, dtype="bf16", signs=True, interleaved=False),
        # a short prefix of one request, for a chunk of its prompt: latency
        dict(name="read_prefix_short", op="read", format="fp4", B=1, ctx=509, page=16, H_kv=8, d=128, dtype="bf16",
             signs=True, packed=False),
        # long prefixes of a batch of chunked prompts, padded to the longest
        dict(name="read_prefix_long", op="read", format="fp4", B=8, ctx=16384, page=64, H_kv=8, d=128,
             dtype="bf16", signs=True, packed=False),
        # a packed batch of ragged prefixes out of the 8-bit cache
        dict(name="read_fp8_ragged", op="read", format="fp8", B=32, ctx=4096, page=64, H_kv=4, d=128,
             dtype="fp16", signs=False, packed=True),
        # one request's next token: latency
        dict(name="decode_one_request", op="decode", B=1, ctx=1500, page=16, H=32, H_kv=8, n_q=1, d=128,
             dtype="bf16", signs=True, causal=True, ragged=False),
        # a decode batch of equal, long contexts: the bandwidth of the cache
        dict(name="decode_batch", op="decode", B=16, ctx=8192, page=256, H=32, H_kv=8, n_q=1, d=128,
             dtype="bf16", signs=True, causal=True, ragged=False),
        # contexts from none to 16 K, small heads
        dict(name="decode_ragged", op="decode", B=64, ctx=16384, page=64, H=32, H_kv=8, n_q=1, d=64,
             dtype="fp16", signs=False, causal=True, ragged=True),
        # four drafted tokens of each request checked at once, eight query heads to a key head
        dict(name="decode_drafts", op="decode", B=8, ctx=8192, page=32, H=32, H_kv=4, n_q=4, d=128,
             dtype="bf16", signs=True, causal=True, ragged=True),
        # a token's attention over a shared prefix and over its own tokens, joined
        dict(name="merge_step", op="merge", B=64, H=32, N=1, d=128, dtype="bf16", packed=False),
        # the chunks of two prompts: prefix and chunk joined
        dict(name="merge_chunks", op="merge", B=2, H=32, N=4096, d=128, dtype="bf16", packed=False),
        # the same over a packed batch, odd length
        dict(name="merge_packed", op="merge", B=1, H=12, N=5001, d=64, dtype="fp16", packed=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "read", "read", "decode", "decode", "decode", "merge"])
    dtype = rng.choice(["bf16", "fp16"])
    d = rng.choice([64, 128])
    H_kv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    signs = rng.random() < 0.5
    if op == "merge":
        packed = rng.random() < 0.5
        N = _log(rng, 1, 4096)
        return dict(op=op, B=1 if packed else rng.randint(1, max(1, min(64, 8192 // N))), H=H_kv * rng.choice([1, 3, 4]),
                    N=N, d=rng.choice([64, 128, 256]), dtype=dtype, packed=packed)
    if op == "append":
        return dict(op=op, B=_log(rng, 1, 64), new=rng.randint(1, 4), prefill=rng.choice([0, _log(rng, 2, 2048)]),
                    ctx=_log(rng, 8, 4096), page=page, H=H_kv * G, H_kv=H_kv, d=d, rot=16 * rng.randint(1, d // 16),
                    dtype=dtype, signs=signs, interleaved=rng.random() < 0.5)
    B, ctx = _log(rng, 1, 64), _log(rng, 1, 16384)
    while B * ctx * H_kv * d > 64 * 4096 * 8 * 64:  # no more than the largest listed ones
        ctx = (ctx + 1) // 2
    if op == "read":
        kind = rng.choice(["fp4", "fp4", "fp8", "16"])
        return dict(op=op, format=kind, B=B, ctx=ctx, page=page, H_kv=H_kv, d=128 if kind == "fp8" else d,
                    dtype=dtype, signs=signs and kind != "16", packed=rng.random() < 0.5)
    return dict(op=op, B=B, ctx=ctx, page=page, H=H_kv * G, H_kv=H_kv, n_q=rng.randint(1, 4), d=d, dtype=dtype,
                signs=signs, causal=rng.random() < 0.8, ragged=rng.random() < 0.7)


# ------------------------------------------------------------------ inputs ----
def _new_lengths(case):
    """(tokens in the cache, new tokens) of each request: every eighth one brings a
    prompt where the case has prompts, the others add a few tokens to a context."""
    B, ctx = case["B"], case["ctx"]
    old, new = [], []
    for b in range(B):
        if case["prefill"] and b % 8 == 0:
            old.append(0)
            new.append(max(1, case["prefill"] - 7 * b % max(1, case["prefill"] // 2)))
        else:
            old.append(1 + (ctx - 1) * (B - b) // B)
            new.append(case["new"])
    return old, new


def _lengths(case):
    """Contexts of a batch: from few tokens to ctx, and one of none in a batch of four or more."""
    B, ctx = case["B"], case["ctx"]
    if not case.get("ragged", True):
        return [ctx] * B
    got = [1 + (ctx - 1) * (B - b) // B for b in range(B)]
    if B >= 4:
        got[B // 2] = 0
    return got


def _firsts(case):
    """First position read of each request: every third one skips an eighth of its context."""
    return [n // 8 if b % 3 == 2 else 0 for b, n in enumerate(_lengths(case))]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pages(lens, page, seed, spare=3):
    """A block table of shuffled pages that hold `lens` tokens of each request."""
    need = [(n + page - 1) // page for n in lens]
    order = list(range(sum(need) + spare))
    random.Random(seed + 1).shuffle(order)
    width, rows, at = max(1, max(need)), [], 0
    for n in need:
        rows.append(order[at:at + n] + [0] * (width - n))
        at += n
    return _i32(rows), len(order)


def _tables_for(n, rot, base=10000.0):
    """float32 rotary tables of positions 0 .. n-1, as a model keeps them."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * base ** (-2.0 * i / rot)[None, :]
    return a.cos().float(), a.sin().float()


def prepare(case, seed):
    op = case["op"]
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    d = case["d"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dt)

    def codes(*shape):
        """e2m1 codes of rows whose largest values are near 6."""
        x = torch.randn(*shape[:-1], 2 * shape[-1], generator=g, device="cuda").mul_(2.2)
        return _pack(_code(x))

    def descales(*shape):
        return (torch.rand(*shape, generator=g, device="cuda") * 0.3 + 0.3).to(torch.bfloat16)

    if op == "merge":
        B, H, N = case["B"], case["H"], case["N"]
        shape = (N, H, d) if case["packed"] else (B, H, N, d)
        rows = (H, N) if case["packed"] else (B, H, N)
        s = dict(case=case)
        for part, level in (("a", 9.0), ("b", 7.0)):
            s["o_" + part] = normal(*shape)
            s["lse_" + part] = torch.randn(*rows, generator=g, device="cuda") + level
        # the first rows of a prompt have no prefix
        s["lse_a"][..., :N // 16] = -math.inf
        s["o_a"][(slice(0, N // 16),) if case["packed"] else (slice(None), slice(None), slice(0, N // 16))] = 0
        return s

    H_kv, page = case["H_kv"], case["page"]
    signs = None
    if case["signs"]:
        signs = torch.where(torch.rand(d, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    s = dict(case=case, signs=signs, page=page)
    if op == "append":
        old, new = _new_lengths(case)
        order = list(range(len(old)))
        random.Random(seed).shuffle(order)
        old, new = [old[i] for i in order], [new[i] for i in order]
        total, H = sum(new), case["H"]
        lens = [a + b for a, b in zip(old, new)]
        table, num = _pages(lens, page, seed)
        old_t, new_t = _i32(old).long(), _i32(new).long()
        cu = torch.cat([new_t.new_zeros(1), new_t.cumsum(0)])
        t = torch.arange(total, device="cuda")
        b = torch.searchsorted(cu, t, right=True) - 1
        pos = old_t[b] + t - cu[b]
        slots = table[b, pos // page].long() * page + pos % page
        rows = normal(total, H + 2 * H_kv, d)
        cos, sin = _tables_for(max(lens), case["rot"])
        s.update(q=rows[:, :H], k=rows[:, H:H + H_kv], v=rows[:, H + H_kv:], cos=cos, sin=sin, slots=slots,
                 positions=pos.to(torch.int32), table=table, lens=_i32(lens), first=_i32(old),
                 cu=cu.to(torch.int32), total=total)
        for name in ("k", "v"):
            s[name + "_cache"] = codes(num, H_kv, page, d // 2)
            s[name + "_descale"] = descales(num, H_kv, page)
        return s

    lens = _lengths(case)
    order = list(range(len(lens)))
    random.Random(seed).shuffle(order)
    first = _firsts(case) if op == "read" else [0] * len(lens)
    lens, first = [lens[i] for i in order], [first[i] for i in order]
    table, num = _pages(lens, page, seed)
    s.update(table=table, lens=_i32(lens), most=max(1, max(lens)))
    kind = case.get("format", "fp4")
    for name in ("k", "v"):
        if kind == "fp4":
            s[name + "_cache"] = codes(num, H_kv, page, d // 2)
            s[name + "_descale"] = descales(num, H_kv, page)
        elif kind == "fp8":
            x = torch.randn(num, page, H_kv, d, generator=g, device="cuda") * 100.0
            s[name + "_cache"] = x.clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)
            s[name + "_descale"] = torch.rand(num, H_kv, generator=g, device="cuda") * 0.005 + 0.005
        else:
            s[name + "_cache"] = normal(num, page, H_kv, d)
    if op == "decode":
        s["q"] = normal(case["B"], case["H"], case["n_q"], d)
        return s
    counts = [n - f for n, f in zip(lens, first)]
    s.update(first=_i32(first), n=max(1, max(counts)), cu=None)
    if case["packed"]:
        s["n"] = sum(counts)
        s["cu"] = _i32([sum(counts[:i]) for i in range(len(counts) + 1)])
    return s


# ----------------------------------------------------------------- plain forms ----
def _code(x):
    """Codes of the e2m1 values next to x, ties to the even one: 0 .. 7, 8 more below zero."""
    a = x.abs()
    n = (a > 0.25).to(torch.uint8)
    n += a >= 0.75
    n += a > 1.25
    n += a >= 1.75
    n += a > 2.5
    n += a >= 3.5
    n += a > 5.0
    return n + 8 * (x < 0).to(torch.uint8)


def _pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _values(packed):
    """float32 values of packed codes, [..., d]."""
    code = torch.stack([packed & 15, packed >> 4], -1).flatten(-2)
    n = (code & 7).float()
    a = torch.where(n < 4, 0.5 * n, torch.where(n < 6, n - 2.0, 2.0 * n - 8.0))
    return torch.where(code > 7, -a, a)


def _stage(x, span):
    """One stage of the Walsh-Hadamard sums: values `span` apart added and subtracted."""
    y = x.unflatten(-1, (x.shape[-1] // (2 * span), 2, span))
    a, b = y[..., 0, :], y[..., 1, :]
    return torch.stack([a + b, a - b], -2).flatten(-3)


def _hadamard(x):
    d = x.shape[-1]
    spans = [1 << i for i in range(d.bit_length() - 1)]
    return functools.reduce(_stage, spans, x) * (1.0 / math.sqrt(d))


def _transformed(x, signs):
    return x if signs is None else _hadamard(x * signs)


def _restored(x, signs):
    return x if signs is None else _hadamard(x) * signs


def _rotated(x, cos, sin, interleaved):
    """x [T, heads, d] in float32, cos and sin [T, 1, rot / 2]."""
    r = 2 * cos.shape[-1]
    y, rest = x[..., :r], x[..., r:]
    if interleaved:
        a, b = y[..., 0::2], y[..., 1::2]
    else:
        a, b = y[..., :r // 2], y[..., r // 2:]
    u, w = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([u, w], -1).flatten(-2) if interleaved else torch.cat([u, w], -1)
    return torch.cat([y, rest], -1)


def _plain_quantise(x):
    """Packed codes and bfloat16 descales of rows x [..., d]: amax / 6, rounded up."""
    amax = x.abs().amax(-1)
    up = (((amax / 6.0).view(torch.int32) + 0xFFFF) >> 16 << 16).view(torch.float32)
    descale = torch.where(amax > 0, up.clamp(min=2.0 ** -100), torch.zeros_like(up))
    x = torch.where(descale[..., None] > 0, x / descale[..., None], torch.zeros_like(x))
    return _pack(_code(x)), descale.to(torch.bfloat16)


def _plain_append(s):
    c = s["case"]
    dt, page = s["q"].dtype, s["page"]
    at = s["positions"].long()
    cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
    q = _rotated(s["q"].float(), cos, sin, c["interleaved"]).to(dt)
    k = _transformed(_rotated(s["k"].float(), cos, sin, c["interleaved"]), s["signs"])
    p, off = s["slots"] // page, s["slots"] % page
    s["k_cache"][p, :, off], s["k_descale"][p, :, off] = _plain_quantise(k)
    s["v_cache"][p, :, off], s["v_descale"][p, :, off] = _plain_quantise(s["v"].float())
    k = _values(s["k_cache"][p, :, off]) * s["k_descale"][p, :, off].float()[..., None]
    v = _values(s["v_cache"][p, :, off]) * s["v_descale"][p, :, off].float()[..., None]
    return {"q": q, "k": _restored(k, s["signs"]).to(dt), "v": v.to(dt), "k_descale": s["k_descale"],
            "v_descale": s["v_descale"]}


def _plain_rows(s, name, p, off):
    """float32 rows [..., H_kv, d] of pages p and offsets off, keys as they are stored."""
    kind = s["case"].get("format", "fp4")
    cache = s[name + "_cache"]
    if kind == "16":
        return cache[p, off].float()
    if kind == "fp8":
        return cache[p, off].view(E4M3).float() * s[name + "_descale"][p][..., None]
    heads = torch.arange(cache.shape[1], device="cuda")
    row = (p[..., None] * cache.shape[1] + heads) * s["page"] + off[..., None]
    return _values(cache.view(-1, cache.shape[-1])[row]) * s[name + "_descale"].view(-1)[row].float()[..., None]


def _plain_read(s):
    c = s["case"]
    dt, page = DTYPES[c["dtype"]], s["page"]
    lens, first = s["lens"].long(), s["first"].long()
    if c["packed"]:
        t = torch.arange(s["n"], device="cuda")
        b = torch.searchsorted(s["cu"].long(), t, right=True) - 1
        pos = first[b] + t - s["cu"].long()[b]
        inside = None
    else:
        b = torch.arange(c["B"], device="cuda")[:, None]
        pos = first[:, None] + torch.arange(s["n"], device="cuda")[None, :]
        inside = (pos < lens[:, None])[..., None, None]
        pos = torch.minimum(pos, (lens[:, None] - 1).clamp(min=0))
    p, off = s["table"][b, pos // page].long(), pos % page
    k = _restored(_plain_rows(s, "k", p, off), s["signs"])
    v = _plain_rows(s, "v", p, off)
    if inside is not None:
        k = torch.where(inside, k, torch.zeros_like(k)).transpose(1, 2)
        v = torch.where(inside, v, torch.zeros_like(v)).transpose(1, 2)
    return {"k": k.to(dt).contiguous(), "v": v.to(dt).contiguous()}


def _plain_decode(s):
    c = s["case"]
    B, H, H_kv, n_q, d = (c[x] for x in ("B", "H", "H_kv", "n_q", "d"))
    lens = s["lens"].long()
    N, page = s["most"], s["page"]
    j = torch.arange(N, device="cuda")
    inside = j[None, :] < lens[:, None]
    at = torch.minimum(j[None, :], (lens[:, None] - 1).clamp(min=0))
    p, off = s["table"][torch.arange(B, device="cuda")[:, None], at // page].long(), at % page
    q = _transformed(s["q"].float(), s["signs"]).view(B, H_kv, (H // H_kv) * n_q, d)
    k = _plain_rows(s, "k", p, off).transpose(1, 2)
    x = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    del k
    end = lens[:, None] + (torch.arange(n_q, device="cuda")[None, :] + 1 - n_q if c["causal"] else 0)
    end = torch.minimum(end, lens[:, None]).expand(B, n_q).repeat(1, H // H_kv)
    seen = (j[None, None, :] < end[:, :, None]) & inside[:, None, :]
    x = x.masked_fill(~seen[:, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = (x - m).exp_()
    l = e.sum(-1, keepdim=True)
    lse = (m + l.log())[..., 0].view(B, H, n_q)
    v = _plain_rows(s, "v", p, off).transpose(1, 2)
    o = torch.matmul(e, v) / torch.where(l == 0, torch.ones_like(l), l)
    return {"o": o.view(B, H, n_q, d).to(s["q"].dtype), "lse": lse}


def _plain_merge(s):
    a, b = s["lse_a"], s["lse_b"]
    m = torch.maximum(a, b)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    u, w = (a - m).exp(), (b - m).exp()
    l = u + w
    safe = torch.where(l == 0, torch.ones_like(l), l)
    u, w = u / safe, w / safe
    if s["case"]["packed"]:
        u, w = u.t(), w.t()
    o = s["o_a"].float() * u[..., None] + s["o_b"].float() * w[..., None]
    return {"o": o.to(s["o_a"].dtype), "lse": m + l.log()}


# ------------------------------------------------------------ the library's calls ----
def _own(s):
    import exact_tiled_attention_25_gb300 as attn
    c = s["case"]
    op = c["op"]
    if op == "merge":
        o, lse = attn.attn_merge(s["o_a"], s["lse_a"], s["o_b"], s["lse_b"])
        return {"o": o, "lse": lse}
    if op == "decode":
        o, lse = attn.attn_decode_paged_fp4(s["q"], s["k_cache"], s["v_cache"], s["k_descale"], s["v_descale"], s["table"],
                                            s["lens"], s["most"], causal=c["causal"], hadamard_signs=s["signs"])
        return {"o": o, "lse": lse}
    dt = DTYPES[c["dtype"]]
    if op == "append":
        q = attn.attn_cache_append_fp4(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_descale"], s["v_descale"],
                                       s["slots"], rope_cos=s["cos"], rope_sin=s["sin"], positions=s["positions"],
                                       hadamard_signs=s["signs"], q=s["q"], interleaved=c["interleaved"])
        k, v = attn.attn_cache_read_fp4(s["k_cache"], s["v_cache"], s["k_descale"], s["v_descale"], s["table"], s["lens"],
                                        s["total"], first=s["first"], cu_seqlens=s["cu"], hadamard_signs=s["signs"],
                                        dtype=dt)
        return {"q": q, "k": k, "v": v, "k_descale": s["k_descale"], "v_descale": s["v_descale"]}
    where = dict(first=s["first"], cu_seqlens=s["cu"])
    if c["format"] == "16":
        k, v = attn.attn_cache_read(s["k_cache"], s["v_cache"], s["table"], s["lens"], s["n"], **where)
    else:
        read = attn.attn_cache_read_fp4 if c["format"] == "fp4" else attn.attn_cache_read_fp8
        k, v = read(s["k_cache"], s["v_cache"], s["k_descale"], s["v_descale"], s["table"], s["lens"], s["n"],
                    hadamard_signs=s["signs"], dtype=dt, **where)
    return {"k": k, "v": v}


PLAIN = {"append": _plain_append, "read": _plain_read, "decode": _plain_decode, "merge": _plain_merge}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------- work ----
def work(case):
    op, d = case["op"], case["d"]
    if op == "merge":
        rows = case["B"] * case["H"] * case["N"]
        return {"bytes": rows * (6 * d + 12), "flops": 3.0 * rows * d}
    H_kv = case["H_kv"]
    stored = {"fp4": d + 4, "fp8": 2 * d, "16": 4 * d}[case.get("format", "fp4")]  # a key and a value
    if op == "append":
        old, new = _new_lengths(case)
        total = sum(new)
        tables = 4 * len(set(p for a, b in zip(old, new) for p in range(a, a + b))) * case["rot"]
        # rows read, codes and queries written; codes read back as rows
        nbytes = total * (4 * case["H"] * d + H_kv * (4 * d + 2 * stored + 4 * d) + 12) + tables
        return {"bytes": nbytes, "flops": total * (3.0 * case["H"] * d + 24.0 * H_kv * d)}
    lens = _lengths(case)
    if op == "read":
        counts = [n - f for n, f in zip(lens, _firsts(case))]
        rows = sum(counts) if case["packed"] else case["B"] * max(1, max(counts))
        return {"bytes": sum(counts) * H_kv * stored + rows * H_kv * 4 * d, "flops": 8.0 * sum(counts) * H_kv * d}
    keys, rows = sum(lens), case["B"] * case["H"] * case["n_q"]
    return {"bytes": keys * H_kv * stored + rows * (4 * d + 4), "flops": 4.0 * keys * case["H"] * case["n_q"] * d}


# --------------------------------------------------------------------- exact ----
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _mixing(d, signs):
    """The orthogonal matrix M of x -> x M, M = diag(signs) H / sqrt(d), or the identity."""
    if signs is None:
        return torch.eye(d, dtype=torch.float64, device="cuda")
    h = torch.ones(1, 1, dtype=torch.float64, device="cuda")
    while h.shape[0] < d:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return signs.double()[:, None] * h / math.sqrt(d)


def _exact_rows(s, name, b, lo, hi):
    """float64 [hi - lo, H_kv, d] of request b's positions lo .. hi - 1."""
    pos = torch.arange(lo, hi, device="cuda")
    p, off = s["table"][b].long()[pos // s["page"]], pos % s["page"]
    kind = s["case"].get("format", "fp4")
    if kind == "16":
        return s[name + "_cache"][p, off].double()
    if kind == "fp8":
        return s[name + "_cache"][p, off].view(E4M3).double() * s[name + "_descale"].double()[p][:, :, None]
    bytes_ = s[name + "_cache"][p, :, off].long()
    value = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float64, device="cuda")
    rows = torch.empty(*bytes_.shape[:-1], 2 * bytes_.shape[-1], dtype=torch.float64, device="cuda")
    rows[..., 0::2], rows[..., 1::2] = value[bytes_ % 16], value[bytes_ // 16]
    return rows * s[name + "_descale"][p, :, off].double()[:, :, None]


def _exact_quantised(x):
    """(values in steps of the descale, descale) of rows x in float64."""
    amax = x.abs().amax(-1)
    e = torch.floor(torch.log2(amax / 6.0).clamp(min=-100.0))
    step = torch.exp2(e - 7.0)  # bfloat16 keeps eight bits
    descale = torch.where(amax > 0, (torch.ceil(amax / 6.0 / step) * step).clamp(min=2.0 ** -100), torch.zeros_like(amax))
    y = torch.where(descale[..., None] > 0, x / descale[..., None], torch.zeros_like(x))
    table = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    hi = torch.searchsorted(table, y.abs().contiguous()).clamp(1, 7)
    a, b = table[hi - 1], table[hi]
    up = (y.abs() - a > b - y.abs()) | ((y.abs() - a == b - y.abs()) & (hi % 2 == 0))
    return torch.where(up, b, a) * torch.sign(y), descale


def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], case["d"]
    if op == "merge":
        a, b = s["lse_a"].double(), s["lse_b"].double()
        lse = torch.logaddexp(a, b)
        u, w = torch.exp(a - lse), torch.exp(b - lse)
        if case["packed"]:
            u, w = u.T, w.T
        return {"o": u[..., None] * s["o_a"].double() + w[..., None] * s["o_b"].double(), "lse": lse}
    M = _mixing(d, s["signs"])
    if op == "append":
        at = s["positions"].long()
        turn = torch.complex(s["cos"][at].double(), s["sin"][at].double())[:, None]
        half = turn.shape[-1]
        first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["interleaved"] else (
            slice(0, half), slice(half, 2 * half))
        got = {}
        for name in ("q", "k"):
            y = s[name].double()
            z = torch.complex(y[..., first], y[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
            got[name] = y
        p, off = s["slots"] // s["page"], s["slots"] % s["page"]
        for name, x in (("k", got["k"] @ M), ("v", s["v"].double())):
            values, scale = _exact_quantised(x)
            rows = values * scale[..., None]
            got[name] = rows @ M.T if name == "k" else rows
            all_ = s[name + "_descale"].double()
            all_[p, :, off] = scale
            got[name + "_descale"] = all_
        return got
    lens = s["lens"].tolist()
    if op == "read":
        ks, vs = [], []
        for b, (n, f) in enumerate(zip(lens, s["first"].tolist())):
            k, v = _exact_rows(s, "k", b, f, n) @ M.T, _exact_rows(s, "v", b, f, n)
            if not case["packed"]:
                k, v = (torch.nn.functional.pad(x, (0, 0, 0, 0, 0, s["n"] - x.shape[0])).transpose(0, 1) for x in (k, v))
            ks.append(k)
            vs.append(v)
        join = torch.cat if case["packed"] else torch.stack
        return {"k": join(ks), "v": join(vs)}
    B, H, H_kv, n_q = (case[x] for x in ("B", "H", "H_kv", "n_q"))
    G = H // H_kv
    o = torch.zeros(B, H, n_q, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, n_q), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        if n == 0:
            continue
        k, v = _exact_rows(s, "k", b, 0, n), _exact_rows(s, "v", b, 0, n)
        q = s["q"][b].double() @ M
        for t in range(n_q):
            m = n - n_q + t + 1 if case["causal"] else n
            if m <= 0:
                continue
            x = torch.einsum("jgd,mjd->jgm", q[:, t].view(H_kv, G, d), k[:m]) / math.sqrt(d)
            z = torch.logsumexp(x, -1)
            lse[b, :, t] = z.reshape(H)
            o[b, :, t] = torch.einsum("jgm,mjd->jgd", torch.exp(x - z[..., None]), v[:m]).reshape(H, d)
    return {"o": o, "lse": lse}
