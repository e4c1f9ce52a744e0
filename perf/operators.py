"""Timed cases of the operators around the attention kernels: cross attention
(forward, training step, single tokens), rotary positions, block tables and
slot maps, and appending keys and values to a paged cache.

``run`` computes an operator from elementary torch operations, or (``own``)
through the library's public entry points.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------- cases ----
def listed():
    return [
        # one new token of one request against its encoder states: latency
        dict(name="cross_token_one_request", op="cross_fwd", B=1, H=16, H_kv=16, N_q=1, N_k=1500, d=64,
             dtype="fp16", lens=False),
        # a decode batch's cross attention, grouped heads, encoder states of different lengths
        dict(name="cross_token_batch", op="cross_fwd", B=32, H=32, H_kv=8, N_q=1, N_k=2048, d=128,
             dtype="bf16", lens=True),
        # a small training batch: odd lengths, grouped heads, one sequence without encoder states
        dict(name="cross_train_ragged", op="cross_train", B=4, H=12, H_kv=4, N_q=509, N_k=1501, d=64,
             dtype="fp16", lens=True),
        # a long training step: the largest matrix products
        dict(name="cross_train_long", op="cross_train", B=2, H=16, H_kv=4, N_q=8192, N_k=4096, d=128,
             dtype="bf16", lens=True),
        # queries and keys of a prefill, halves of the head paired, [B, H, N, d]
        dict(name="rope_prefill", op="rope", B=2, H=32, H_kv=8, N=8192, d=128, rot=128, dtype="bf16",
             packed=False, interleaved=False, inverse=False),
        # gradients of a packed batch in rows of fused projections: neighbours paired, a quarter of the head
        dict(name="rope_grad_partial", op="rope", B=1, H=16, H_kv=16, N=16383, d=64, rot=16, dtype="fp16",
             packed=True, interleaved=True, inverse=True),
        # the tables of a long context, stretched eight times
        dict(name="rope_table_long", op="rope_table", n=131072, rot=128, base=500000.0, factor=8.0,
             orig_len=16384),
        # one decode step of a few requests
        dict(name="tables_decode", op="tables", B=16, new=1, prefill=0, ctx=8192, page=64),
        # a large mixed batch: an eighth of the requests bring a prompt
        dict(name="tables_mixed", op="tables", B=1024, new=1, prefill=2048, ctx=8192, page=16),
        # one decode step: rotate queries and keys, write keys and values to their slots
        dict(name="append_decode", op="append", B=64, new=1, prefill=0, ctx=2048, page=64, H=32, H_kv=8,
             d=128, rot=128, dtype="bf16", fp8=False, signs=False, interleaved=False),
        # one decode step into the 8-bit cache
        dict(name="append_fp8_decode", op="append", B=64, new=1, prefill=0, ctx=2048, page=64, H=32, H_kv=8,
             d=128, rot=128, dtype="bf16", fp8=True, signs=True, interleaved=False),
        # prompts into the 8-bit cache, keys transformed
        dict(name="append_fp8_prefill", op="append", B=16, new=1, prefill=8192, ctx=2048, page=256, H=32,
             H_kv=8, d=128, rot=128, dtype="bf16", fp8=True, signs=True, interleaved=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["cross_fwd", "cross_fwd", "cross_train", "cross_train", "rope", "rope", "rope_table",
                     "tables", "tables", "append", "append", "append"])
    dtype = rng.choice(["bf16", "fp16"])
    if op in ("cross_fwd", "cross_train"):
        H_kv = rng.choice([1, 2, 4, 8])
        H = H_kv * rng.choice([1, 2, 4])
        d = rng.choice([64, 128])
        if op == "cross_fwd" and rng.random() < 0.5:
            N_q, N_k, B = rng.randint(1, 8), _log(rng, 1, 8192), _log(rng, 1, 64)
        else:
            N_q, N_k, B = _log(rng, 1, 4096), _log(rng, 1, 4096), rng.randint(1, 4)
        while B * H * N_q * N_k * d > 2e10:  # well below the largest listed one
            N_q = (N_q + 1) // 2
        return dict(op=op, B=B, H=H, H_kv=H_kv, N_q=N_q, N_k=N_k, d=d, dtype=dtype,
                    lens=rng.random() < 0.7)
    if op == "rope":
        d = rng.choice([64, 128, 256])
        H_kv = rng.choice([1, 2, 4, 8])
        packed = rng.random() < 0.5
        return dict(op=op, B=1 if packed else rng.randint(1, 4), H=H_kv * rng.choice([1, 3, 4]), H_kv=H_kv,
                    N=_log(rng, 1, 8192), d=d, rot=16 * rng.randint(1, d // 16), dtype=dtype, packed=packed,
                    interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5)
    if op == "rope_table":
        return dict(op=op, n=_log(rng, 1, 131072), rot=rng.choice([16, 32, 64, 96, 128]),
                    base=rng.choice([10000.0, 500000.0]), factor=rng.choice([1.0, 2.0, 8.0]),
                    orig_len=rng.choice([0, 4096, 16384]))
    prefill = rng.choice([0, 0, _log(rng, 2, 2048)])
    B = _log(rng, 1, 1024 if op == "tables" else 128)
    page = rng.choice([16, 32, 64, 128, 256])
    case = dict(op=op, B=B, new=rng.randint(1, 4), prefill=prefill, ctx=_log(rng, 8, 4096), page=page)
    if op == "tables":
        return case
    fp8 = rng.random() < 0.6
    d = 128 if fp8 else rng.choice([64, 128, 256])
    H_kv = rng.choice([1, 2, 4, 8])
    case.update(B=min(B, 64), H=H_kv * rng.choice([1, 2, 4]), H_kv=H_kv, d=d, rot=16 * rng.randint(1, d // 16),
                dtype=dtype, fp8=fp8, signs=fp8 and rng.random() < 0.5, interleaved=rng.random() < 0.5)
    return case


# ------------------------------------------------------------------ inputs ----
def _kv_lengths(case):
    """Key lengths of a batch: from half of N_k to N_k, and one empty in a batch of four or more."""
    B, N_k = case["B"], case["N_k"]
    if not case["lens"]:
        return [N_k] * B
    got = [N_k - (N_k // 2) * i // max(1, B) for i in range(B)]
    if B >= 4:
        got[B // 2] = 0
    return got


def _request_lengths(case):
    """(tokens in the cache, new tokens) of each request: every eighth one (the
    first among them) brings a prompt where the case has prompts, the others add
    a few tokens to a context of some length."""
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


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _shuffled(lists, seed):
    order = list(range(len(lists[0])))
    random.Random(seed).shuffle(order)
    return [torch.tensor([x[i] for i in order], dtype=torch.int32, device="cuda") for x in lists]


def _tables_for(n, rot, base=10000.0):
    """float32 tables of positions 0 .. n-1, as a model keeps them."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * base ** (-2.0 * i / rot)[None, :]
    return a.cos().float(), a.sin().float()


def _pool(case, old, new, seed, spare=3):
    """A block table that holds the old tokens, and the free pages, from one shuffled pool."""
    page = case["page"]
    have = [(n + page - 1) // page for n in old]
    need = [(n + m + page - 1) // page for n, m in zip(old, new)]
    num_pages = sum(need) + spare
    order = list(range(num_pages))
    random.Random(seed + 1).shuffle(order)
    rows, at = [], 0
    width = max(need)
    for n in have:
        rows.append(order[at:at + n] + [-1] * (width - n))
        at += n
    dev = dict(dtype=torch.int32, device="cuda")
    return torch.tensor(rows, **dev), torch.tensor(order[at:], **dev), num_pages


def prepare(case, seed):
    op = case["op"]
    g = _gen(seed)
    dt = DTYPES.get(case.get("dtype"))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dt)

    if op in ("cross_fwd", "cross_train"):
        B, H, H_kv, N_q, N_k, d = (case[x] for x in ("B", "H", "H_kv", "N_q", "N_k", "d"))
        s = dict(case=case, q=normal(B, H, N_q, d), k=normal(B, H_kv, N_k, d), v=normal(B, H_kv, N_k, d),
                 lens=_shuffled([_kv_lengths(case)], seed)[0] if case["lens"] else None)
        if op == "cross_train":
            s["dout"] = normal(B, H, N_q, d)
        return s
    if op == "rope":
        B, H, H_kv, N, d = (case[x] for x in ("B", "H", "H_kv", "N", "d"))
        cos, sin = _tables_for(N + 64, case["rot"])
        if case["packed"]:
            # views into the rows of a fused projection, positions of several sequences back to back
            rows = normal(N, H + 2 * H_kv, d)
            pos = (torch.arange(N, device="cuda") * 7 + seed % 31) % (N + 64)
            return dict(case=case, q=rows[:, :H], k=rows[:, H:H + H_kv], cos=cos, sin=sin,
                        positions=pos.to(torch.int32))
        return dict(case=case, q=normal(B, H, N, d), k=normal(B, H_kv, N, d), cos=cos, sin=sin, positions=None)
    if op == "rope_table":
        return dict(case=case, first=seed % 64)
    old, new = _request_lengths(case)
    order = list(range(len(old)))
    random.Random(seed).shuffle(order)
    old, new = [old[i] for i in order], [new[i] for i in order]
    total = sum(new)
    dev = dict(dtype=torch.int32, device="cuda")
    table, free, num_pages = _pool(case, old, new, seed)
    s = dict(case=case, total=total, page=case["page"], old=torch.tensor(old, **dev),
             new=torch.tensor(new, **dev), table=table, free=free)
    if op == "tables":
        return s
    H, H_kv, d, page = case["H"], case["H_kv"], case["d"], case["page"]
    seq_lens, cu, slots, positions, _, table = _plain_tables(s)
    rows = normal(total, H + 2 * H_kv, d)
    cos, sin = _tables_for(max(a + b for a, b in zip(old, new)), case["rot"])
    s.update(q=rows[:, :H], k=rows[:, H:H + H_kv], v=rows[:, H + H_kv:], cos=cos, sin=sin, table=table,
             seq_lens=seq_lens, cu=cu, slots=slots, positions=positions, num_pages=num_pages, signs=None)
    shape = (num_pages, page, H_kv, d)
    if not case["fp8"]:
        s.update(kc=normal(*shape), vc=normal(*shape))
        return s
    for name in ("kc", "vc"):
        values = torch.randn(*shape, generator=g, device="cuda") * 100.0
        s[name] = values.clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)
        s[name + "_scale"] = torch.rand(num_pages, H_kv, generator=g, device="cuda") * 0.005 + 0.005
    if case["signs"]:
        s["signs"] = torch.where(torch.rand(d, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    return s


# ----------------------------------------------------------------- plain forms ----
def _plain_cross(s, train):
    c = s["case"]
    G = c["H"] // c["H_kv"]
    scale = 1.0 / math.sqrt(c["d"])
    q = s["q"].float()
    k = s["k"].float().repeat_interleave(G, 1)
    v = s["v"].float().repeat_interleave(G, 1)
    x = torch.matmul(q, k.transpose(2, 3)) * scale
    if s["lens"] is not None:
        out = torch.arange(c["N_k"], device="cuda")[None, :] >= s["lens"][:, None]
        x.masked_fill_(out[:, None, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = (x - m).exp_()
    del x
    l = p.sum(-1, keepdim=True)
    lse = (m + l.log())[..., 0]
    p = p / torch.where(l == 0, torch.ones_like(l), l)
    o = torch.matmul(p, v)
    dt = s["q"].dtype
    if not train:
        return {"o": o.to(dt), "lse": lse}
    do = s["dout"].float()
    dp = torch.matmul(do, v.transpose(2, 3))
    ds = p * (dp - (do * o).sum(-1, keepdim=True))
    del dp
    heads = (c["B"], c["H_kv"], G, c["N_k"], c["d"])
    dv = torch.matmul(p.transpose(2, 3), do).view(heads).sum(2)
    dk = (torch.matmul(ds.transpose(2, 3), q) * scale).view(heads).sum(2)
    dq = torch.matmul(ds, k) * scale
    return {"o": o.to(dt), "lse": lse, "dq": dq.to(dt), "dk": dk.to(dt), "dv": dv.to(dt)}


def _plain_rotate(x, cos, sin, interleaved, inverse):
    """x [..., d] in float32, cos and sin broadcast to [..., rot / 2]."""
    r = 2 * cos.shape[-1]
    y, rest = x[..., :r], x[..., r:]
    if interleaved:
        a, b = y[..., 0::2], y[..., 1::2]
    else:
        a, b = y[..., :r // 2], y[..., r // 2:]
    if inverse:
        sin = -sin
    u, w = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([u, w], -1).flatten(-2) if interleaved else torch.cat([u, w], -1)
    return torch.cat([y, rest], -1)


def _plain_rope(s):
    c = s["case"]
    if c["packed"]:
        at = s["positions"].long()
        cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
    else:
        cos, sin = s["cos"][:c["N"]], s["sin"][:c["N"]]
    q = _plain_rotate(s["q"].float(), cos, sin, c["interleaved"], c["inverse"])
    k = _plain_rotate(s["k"].float(), cos, sin, c["interleaved"], c["inverse"])
    return {"q": q.to(s["q"].dtype), "k": k.to(s["k"].dtype)}


#: Turns within the first context above which a frequency is kept, and below which it is stretched.
LOW, HIGH, ATTN_FACTOR = 1.0, 32.0, 1.1


def _plain_rope_table(s):
    c = s["case"]
    i = torch.arange(c["rot"] // 2, dtype=torch.float64, device="cuda")
    theta = c["base"] ** (-2.0 * i / c["rot"])
    keep = ((c["orig_len"] * theta / (2.0 * math.pi) - LOW) / (HIGH - LOW)).clamp(0.0, 1.0)
    keep = keep if c["orig_len"] else torch.zeros_like(keep)
    theta = theta * (keep + (1.0 - keep) / c["factor"])
    at = torch.arange(c["n"], dtype=torch.float64, device="cuda") + s["first"]
    angle = at[:, None] * theta[None, :]
    return {"cos": (angle.cos() * ATTN_FACTOR).float(), "sin": (angle.sin() * ATTN_FACTOR).float()}


def _plain_tables(s):
    """seq_lens, cu_seqlens, slots, positions, pages used, block table."""
    old, new, table, page = s["old"].long(), s["new"].long(), s["table"], s["page"]
    lens = old + new
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    have, need = (old + page - 1) // page, (lens + page - 1) // page
    after = (need - have).cumsum(0)
    first = after - (need - have)
    p = torch.arange(table.shape[1], device="cuda")[None, :]
    fresh = (p >= have[:, None]) & (p < need[:, None])
    at = (first[:, None] + p - have[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][at], table)
    t = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = old[b] + t - cu[b]
    slots = table[b, pos // page].long() * page + pos % page
    return (lens.to(torch.int32), cu.to(torch.int32), slots, pos.to(torch.int32), after[-1:].to(torch.int32),
            table)


def _plain_append(s):
    c = s["case"]
    at = s["positions"].long()
    cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
    q = _plain_rotate(s["q"].float(), cos, sin, c["interleaved"], False).to(s["q"].dtype)
    k = _plain_rotate(s["k"].float(), cos, sin, c["interleaved"], False).to(s["k"].dtype)
    s["kc"].view(-1, c["H_kv"], c["d"])[s["slots"]] = k
    s["vc"].view(-1, c["H_kv"], c["d"])[s["slots"]] = s["v"]
    return {"q": q, "kc": s["kc"], "vc": s["vc"]}


def _plain_append_8(x, codes, scale, slots, page):
    """Adds rows x [T, H_kv, d] (float32) to a cache of e4m3 codes with a scale
    for each page and head, in place."""
    num_pages, _, H_kv, d = codes.shape
    at, off = slots // page, slots % page
    new = torch.zeros(num_pages, H_kv, device="cuda")
    new.scatter_reduce_(0, at[:, None].expand(-1, H_kv), x.abs().amax(-1) / 448.0, "amax")
    start = torch.full((num_pages,), page, dtype=torch.int64, device="cuda")
    start.scatter_reduce_(0, at, off, "amin")
    touched, fresh = (start < page)[:, None], (start == 0)[:, None]
    before = torch.where(fresh, torch.zeros_like(scale), scale)
    after = torch.maximum(before, new)
    after = torch.where(after == 0, torch.ones_like(after), after)
    after = torch.where(touched, after, scale)
    values = codes.view(E4M3).float()
    again = values * (before / after)[:, None, :, None]
    row = torch.arange(page, device="cuda")[None, :]
    older = (touched & (row < start[:, None]))[:, :, None, None] & (after > before)[:, None, :, None]
    values = torch.where(older, again, values)
    values = torch.where(fresh[:, :, None, None], torch.zeros_like(values), values)
    values.view(-1, H_kv, d)[slots] = x / after[at][:, :, None]
    codes.copy_(values.clamp(-448.0, 448.0).to(E4M3).view(torch.uint8))
    scale.copy_(after)


def _hadamard(d, dtype):
    h = torch.ones(1, 1, dtype=dtype, device="cuda")
    while h.shape[0] < d:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h


def _plain_append_fp8(s):
    c = s["case"]
    at = s["positions"].long()
    cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
    q = _plain_rotate(s["q"].float(), cos, sin, c["interleaved"], False).to(s["q"].dtype)
    k = _plain_rotate(s["k"].float(), cos, sin, c["interleaved"], False)
    if s["signs"] is not None:
        k = torch.matmul(k * s["signs"], _hadamard(c["d"], torch.float32)) / math.sqrt(c["d"])
    _plain_append_8(k, s["kc"], s["kc_scale"], s["slots"], c["page"])
    _plain_append_8(s["v"].float(), s["vc"], s["vc_scale"], s["slots"], c["page"])
    return {"q": q, "kc": s["kc"].view(E4M3), "vc": s["vc"].view(E4M3), "k_scale": s["kc_scale"],
            "v_scale": s["vc_scale"]}


# ------------------------------------------------------------ the library's calls ----
def _own(s):
    import exact_tiled_attention_25_gb300 as attn
    c = s["case"]
    op = c["op"]
    if op == "cross_fwd":
        o, lse = attn.attn_cross_fwd(s["q"], s["k"], s["v"], s["lens"])
        return {"o": o, "lse": lse}
    if op == "cross_train":
        o, lse = attn.attn_cross_fwd(s["q"], s["k"], s["v"], s["lens"])
        dq, dk, dv = attn.attn_cross_bwd(s["q"], s["k"], s["v"], o, s["dout"], lse, s["lens"])
        return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    if op == "rope":
        q, k = attn.attn_rope(s["q"], s["k"], s["cos"], s["sin"], positions=s["positions"],
                              interleaved=c["interleaved"], inverse=c["inverse"])
        return {"q": q, "k": k}
    if op == "rope_table":
        cos, sin = attn.attn_rope_table(c["n"], c["rot"], base=c["base"], factor=c["factor"],
                                        orig_len=c["orig_len"], low=LOW, high=HIGH, attn_factor=ATTN_FACTOR,
                                        first=s["first"])
        return {"cos": cos, "sin": sin}
    if op == "tables":
        seq_lens, cu, slots, positions, used = attn.attn_block_tables(
            s["table"], s["old"], s["new"], s["free"], c["page"], s["total"])
        return {"seq_lens": seq_lens, "cu": cu, "slots": slots, "positions": positions, "used": used,
                "table": s["table"]}
    if not c["fp8"]:
        q = attn.attn_cache_append(s["k"], s["v"], s["kc"], s["vc"], s["slots"], rope_cos=s["cos"],
                                   rope_sin=s["sin"], positions=s["positions"], q=s["q"],
                                   interleaved=c["interleaved"])
        return {"q": q, "kc": s["kc"], "vc": s["vc"]}
    q = attn.attn_cache_append_fp8(s["k"], s["v"], s["kc"], s["vc"], s["kc_scale"], s["vc_scale"], s["table"],
                                   s["seq_lens"], s["cu"], rope_cos=s["cos"], rope_sin=s["sin"],
                                   hadamard_signs=s["signs"], q=s["q"], interleaved=c["interleaved"])
    return {"q": q, "kc": s["kc"].view(E4M3), "vc": s["vc"].view(E4M3), "k_scale": s["kc_scale"],
            "v_scale": s["vc_scale"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op in ("cross_fwd", "cross_train"):
        return _plain_cross(state, op == "cross_train")
    if op == "rope":
        return _plain_rope(state)
    if op == "rope_table":
        return _plain_rope_table(state)
    if op == "tables":
        seq_lens, cu, slots, positions, used, table = _plain_tables(state)
        return {"seq_lens": seq_lens, "cu": cu, "slots": slots, "positions": positions, "used": used,
                "table": table}
    return _plain_append_fp8(state) if state["case"]["fp8"] else _plain_append(state)


# ---------------------------------------------------------------------- work ----
def work(case):
    op = case["op"]
    if op in ("cross_fwd", "cross_train"):
        B, H, H_kv, N_q, d = (case[x] for x in ("B", "H", "H_kv", "N_q", "d"))
        keys = sum(_kv_lengths(case))
        rows = B * H * N_q
        flops = 4.0 * H * N_q * keys * d
        nbytes = 2 * (2 * rows * d + 2 * H_kv * keys * d) + 4 * rows
        if op == "cross_train":
            # dO read, dQ written; dK, dV written whole
            flops *= 3.5
            nbytes += 2 * (2 * rows * d + 2 * B * H_kv * case["N_k"] * d)
        return {"bytes": nbytes, "flops": flops}
    if op == "rope":
        x = case["B"] * case["N"] * (case["H"] + case["H_kv"])
        return {"bytes": 4 * x * case["d"] + 4 * case["N"] * case["rot"], "flops": 3.0 * x * case["rot"]}
    if op == "rope_table":
        return {"bytes": 4 * case["n"] * case["rot"], "flops": 3.0 * case["n"] * case["rot"]}
    old, new = _request_lengths(case)
    page, total = case["page"], sum(new)
    touched = sum((a + b + page - 1) // page - a // page for a, b in zip(old, new) if b)
    fresh = sum((a + b + page - 1) // page - (a + page - 1) // page for a, b in zip(old, new))
    if op == "tables":
        return {"bytes": 16 * len(old) + 12 * total + 4 * (touched + fresh), "flops": 4.0 * total}
    row_q, row_kv = case["H"] * case["d"], 2 * case["H_kv"] * case["d"]
    tables = 4 * len(set(p for a, b in zip(old, new) for p in range(a, a + b))) * case["rot"]
    if not case["fp8"]:
        return {"bytes": total * (4 * row_q + 4 * row_kv + 12) + tables,
                "flops": 3.0 * total * (row_q + row_kv // 2)}
    nbytes = total * (4 * row_q + 3 * row_kv) + tables + touched * case["H_kv"] * 16 + 4 * touched
    # the cleared rest of a fresh page
    nbytes += sum(-(a + b) % page for a, b in zip(old, new) if b and (a + b - 1) // page * page >= a) * row_kv
    return {"bytes": nbytes, "flops": total * (3.0 * row_q + 12.0 * row_kv)}


# --------------------------------------------------------------------- exact ----
def _exact_cross(case, s):
    B, H, H_kv, N_q, N_k, d = (case[x] for x in ("B", "H", "H_kv", "N_q", "N_k", "d"))
    scale = d ** -0.5
    lens = [N_k] * B if s["lens"] is None else s["lens"].tolist()
    wide = dict(dtype=torch.float64, device="cuda")
    o, lse = torch.zeros(B, H, N_q, d, **wide), torch.full((B, H, N_q), -math.inf, **wide)
    dq, dk, dv = torch.zeros(B, H, N_q, d, **wide), torch.zeros(B, H_kv, N_k, d, **wide), torch.zeros(
        B, H_kv, N_k, d, **wide)
    for b in range(B):
        n = lens[b]
        for h in range(H if n else 0):
            j = h // (H // H_kv)
            q, k, v = s["q"][b, h].double(), s["k"][b, j, :n].double(), s["v"][b, j, :n].double()
            x = q @ k.T * scale
            lse[b, h] = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[b, h][:, None])
            o[b, h] = p @ v
            if "dout" in s:
                do = s["dout"][b, h].double()
                ds = p * (do @ v.T - (do * o[b, h]).sum(1, keepdim=True))
                dq[b, h] = ds @ k * scale
                dk[b, j, :n] += ds.T @ q * scale
                dv[b, j, :n] += p.T @ do
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv} if "dout" in s else {"o": o, "lse": lse}


def _exact_rotate(x, at, cos, sin, interleaved, inverse):
    """Complex rotation of x [T, heads, d] (float64) by the tables' rows `at`."""
    half = cos.shape[1]
    turn = torch.complex(cos[at].double(), sin[at].double())[:, None]
    if inverse:
        turn = turn.conj()
    y = x.clone()
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (
        slice(0, half), slice(half, 2 * half))
    z = torch.complex(x[..., first], x[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _round_e4m3(x):
    """Nearest multiple of the e4m3 step of x's binade (ties to even), float64."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -9))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("cross_fwd", "cross_train"):
        return _exact_cross(case, s)
    if op == "rope":
        got = {}
        for name in ("q", "k"):
            x = s[name].double()
            if not case["packed"]:
                x = x.permute(0, 2, 1, 3).flatten(0, 1)
            at = s["positions"].long() if case["packed"] else torch.arange(case["N"], device="cuda").repeat(case["B"])
            y = _exact_rotate(x, at, s["cos"], s["sin"], case["interleaved"], case["inverse"])
            if not case["packed"]:
                y = y.unflatten(0, (case["B"], case["N"])).permute(0, 2, 1, 3)
            got[name] = y
        return got
    if op == "rope_table":
        rows = []
        for i in range(case["rot"] // 2):
            theta = math.exp(-math.log(case["base"]) * 2 * i / case["rot"])
            keep = 0.0
            if case["orig_len"]:
                keep = min(1.0, max(0.0, (case["orig_len"] * theta / math.tau - LOW) / (HIGH - LOW)))
            rows.append(theta * keep + theta / case["factor"] * (1.0 - keep))
        p = torch.arange(s["first"], s["first"] + case["n"], dtype=torch.float64, device="cuda")
        a = torch.outer(p, torch.tensor(rows, dtype=torch.float64, device="cuda"))
        return {"cos": ATTN_FACTOR * torch.cos(a), "sin": ATTN_FACTOR * torch.sin(a)}
    if op == "tables":
        return None  # whole numbers
    at = s["positions"].long()
    q = _exact_rotate(s["q"].double(), at, s["cos"], s["sin"], case["interleaved"], False)
    k = _exact_rotate(s["k"].double(), at, s["cos"], s["sin"], case["interleaved"], False)
    v = s["v"].double()
    H_kv, d, page = case["H_kv"], case["d"], case["page"]
    if not case["fp8"]:
        kc, vc = s["kc"].double(), s["vc"].double()
        kc.view(-1, H_kv, d)[s["slots"]] = k
        vc.view(-1, H_kv, d)[s["slots"]] = v
        return {"q": q, "kc": kc, "vc": vc}
    if s["signs"] is not None:
        k = (k * s["signs"].double()) @ _hadamard(d, torch.float64) / math.sqrt(d)
    got = {"q": q}
    pages = (s["slots"] // page).tolist()
    spans = {}
    for t, p in enumerate(pages):  # a page's new tokens are neighbours
        lo, hi = spans.get(p, (t, t))
        spans[p] = (min(lo, t), max(hi, t))
    for name, x, out in (("kc", k, "k_scale"), ("vc", v, "v_scale")):
        codes, scale = s[name].view(E4M3).double(), s[name + "_scale"].double()
        for p, (lo, hi) in spans.items():
            first = int(s["slots"][lo] % page)
            rows = x[lo:hi + 1]
            biggest = rows.abs().amax((0, 2)) / 448.0
            was = scale[p] if first else torch.zeros_like(scale[p])
            now = torch.maximum(was, biggest.float().double())
            now = torch.where(now == 0, torch.ones_like(now), now)
            if first:
                grown = (now > was)[None, :, None]
                codes[p, :first] = torch.where(grown, _round_e4m3(codes[p, :first] * (was / now)[None, :, None]),
                                               codes[p, :first])
            else:
                codes[p] = 0.0
            codes[p, first:first + hi + 1 - lo] = _round_e4m3(rows / now[None, :, None])
            scale[p] = now
        got[name], got[out] = codes, scale
    return got
