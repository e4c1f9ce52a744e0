"""4-bit (e2m1) cache rows, reading a paged cache back, and joining partial attentions --
TEST INFRASTRUCTURE.

* e2m1 (OCP E2M1): a sign bit, two exponent bits with bias 1, one mantissa bit: magnitudes 0,
  0.5, 1, 1.5, 2, 3, 4, 6.  Element 2 i of a row is the low half of byte i.
* A row x is held as descale = float32(amax|x|) / 6 rounded up to bfloat16, at least 2^-100 (0
  for a row of zeros, NaN for one with an infinity or a NaN), and code = e2m1(x / descale),
  nearest, ties to even.
* The cache is [num_pages, H_kv, page_size, d / 2] with descales [num_pages, H_kv, page_size].
* Keys are rotated, then transformed, x -> (x o signs) H_d / sqrt(d), in float32: each
  product, sum and scaling rounded by itself, the transform's sums by increasing span.
* Joining: softmax over a union of two key sets, from the log-sum-exps of both.
"""
from __future__ import annotations

import numpy as np

E2M1_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def e2m1_encode(x) -> np.ndarray:
    """Codes 0 .. 15 of values: nearest, ties to the even code, at most 6."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 6.0)
    best = np.zeros(x.shape, dtype=np.uint8)
    near = np.abs(a - E2M1_VALUES[0])
    for code in range(1, 8):
        dist = np.abs(a - E2M1_VALUES[code])
        take = (dist < near) | ((dist == near) & (code % 2 == 0))
        best, near = np.where(take, np.uint8(code), best), np.where(take, dist, near)
    return np.where(np.signbit(x), best | np.uint8(8), best).astype(np.uint8)


def e2m1_decode(packed) -> np.ndarray:
    """float64 values [..., d] of bytes [..., d / 2]."""
    b = np.asarray(packed, dtype=np.uint8)
    value = np.array(E2M1_VALUES + tuple(-v for v in E2M1_VALUES))
    return np.stack([value[b & 15], value[b >> 4]], -1).reshape(*b.shape[:-1], -1)


def row_descale(amax) -> np.ndarray:
    """float32 values (exact in bfloat16) of the descales of rows with these largest magnitudes."""
    out = np.empty(np.shape(amax), dtype=np.float32)
    for at, a in np.ndenumerate(np.asarray(amax, dtype=np.float32)):
        if not np.isfinite(a):
            out[at] = np.nan
        elif a == 0:
            out[at] = 0.0
        else:
            bits = int(np.float32(a / np.float32(6.0)).view(np.uint32))
            if bits & 0xFFFF:
                bits = (bits | 0xFFFF) + 1
            out[at] = max(np.uint32(bits).view(np.float32), np.float32(2.0 ** -100))
    return out


def quantize_rows(x):
    """(bytes [..., d / 2], descales float32 [...]) of float32 rows."""
    x = np.asarray(x, dtype=np.float32)
    descale = row_descale(np.max(np.abs(x), axis=-1))
    safe = np.where(descale > 0, descale, np.float32(1.0))
    with np.errstate(invalid="ignore"):
        code = e2m1_encode((np.where(np.isfinite(x), x, np.float32(0)) / safe[..., None]).astype(np.float32))
    code = np.where((descale > 0)[..., None], code, 0).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), descale


def key_rows_f32(k, positions, cos, sin, interleaved, signs):
    """float32 key rows [T, H_kv, d] as they are quantised."""
    x = np.asarray(k, dtype=np.float32).copy()
    if cos is not None:
        c, s = (np.asarray(t, np.float32)[positions][:, None] for t in (cos, sin))
        half = c.shape[-1]
        a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
        u, w = x[..., a].copy(), x[..., b].copy()
        x[..., a] = u * c - w * s
        x[..., b] = w * c + u * s
    if signs is not None:
        x = x * np.asarray(signs, np.float32)
        d, span = x.shape[-1], 1
        while span < d:
            y = x.reshape(*x.shape[:-1], d // (2 * span), 2, span)
            x = np.stack([y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]], -2).reshape(x.shape)
            span *= 2
        x = x * np.float32(1.0 / np.sqrt(d))
    return x


def append_fp4(x, codes, descale, slots):
    """Cache and descales after float32 rows x [T, H_kv, d] went to their slots (-1: none)."""
    codes, descale = np.array(codes), np.array(descale, dtype=np.float32)
    page = codes.shape[2]
    for t, slot in enumerate(np.asarray(slots)):
        if slot >= 0:
            codes[slot // page, :, slot % page], descale[slot // page, :, slot % page] = quantize_rows(x[t])
    return codes, descale


def dequantize_cache_fp4(codes, descale) -> np.ndarray:
    """float64 values [num_pages, page_size, H_kv, d]."""
    return np.swapaxes(e2m1_decode(codes) * np.asarray(descale, np.float64)[..., None], 1, 2)


def read_cache(values, table, lens, first, counts):
    """Rows [counts[b], H_kv, d] of each request from position first[b] on, zeros from lens[b] on."""
    page, out = values.shape[1], []
    for b, n in enumerate(counts):
        rows = np.zeros((n,) + values.shape[2:])
        for i in range(n):
            pos = int(first[b]) + i
            if pos < lens[b]:
                rows[i] = values[table[b][pos // page], pos % page]
        out.append(rows)
    return out


def merge_attention(o_a, lse_a, o_b, lse_b):
    """O [..., d] and LSE [...] over the union of two key sets."""
    o_a, o_b, la, lb = (np.asarray(x, np.float64) for x in (o_a, o_b, lse_a, lse_b))
    with np.errstate(invalid="ignore"):
        lse = np.logaddexp(la, lb)
        wa, wb = np.exp(la - lse), np.exp(lb - lse)
    none = lse == -np.inf
    wa, wb = np.where(none, 0.0, wa), np.where(none, 0.0, wb)
    part = lambda w, o: np.where(w[..., None] == 0, 0.0, w[..., None] * np.where(w[..., None] == 0, 0.0, o))
    return part(wa, o_a) + part(wb, o_b), lse
