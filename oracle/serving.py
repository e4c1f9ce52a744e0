"""What surrounds attention in a decoder layer -- TEST INFRASTRUCTURE.

Cross attention, rotary tables and rotations, block tables and slot maps, and
the e4m3 cache append, each written out from its definition in float64, one
row, request or page at a time.

* Cross attention: the softmax attention of ``attention.py`` with N_q query rows
  and N_k keys, of which batch entry b sees the first kv_lens[b]; without keys
  O = 0, L = -inf and all gradients are 0.
* Rotary tables: theta_i = base^(-2i/r); with a first context of L0 positions
  frequency i makes L0 theta_i / (2 pi) turns in it, is kept from `high` turns on,
  divided by `factor` up to `low` turns, and blended linearly between; L0 = 0
  divides all.  Rotation: (x, y) -> (x c - y s, y c + x s) on the pairs of the
  first r columns.
* Block tables: request b's tokens occupy its first ceil(len / page) pages; new
  pages come from the front of a free list, requests in order.
* e4m3 append: one float32 descale per (page, head); it grows to amax / 448 of
  the new rows, and a page whose first row is new starts from 0.  A growing
  descale requantises the page's earlier codes.
"""
from __future__ import annotations

import math

import numpy as np

from .attention import attention_backward_head, attention_forward_head
from .fp8 import E4M3_MAX, e4m3_decode, e4m3_encode, incoherent_transform


def attention_cross_forward(q, k, v, scale, kv_lens=None):
    """q [B, H, N_q, d]; k, v [B, H_kv, N_k, d] -> O [B, H, N_q, d], LSE [B, H, N_q]."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    B, H, N_q, d = q.shape
    G = H // k.shape[1]
    o = np.zeros((B, H, N_q, d))
    lse = np.full((B, H, N_q), -np.inf)
    for b in range(B):
        n = k.shape[2] if kv_lens is None else int(kv_lens[b])
        if n == 0:
            continue
        for h in range(H):
            o[b, h], lse[b, h] = attention_forward_head(q[b, h], k[b, h // G, :n], v[b, h // G, :n], scale)
    return o, lse


def attention_cross_backward(q, k, v, do, scale, kv_lens=None):
    """Gradients of sum(O * dO): dQ, and dK, dV summed over each group, 0 behind kv_lens."""
    q, k, v, do = (np.asarray(x, dtype=np.float64) for x in (q, k, v, do))
    G = q.shape[1] // k.shape[1]
    dq, dk, dv = np.zeros_like(q), np.zeros(k.shape), np.zeros(v.shape)
    for b in range(q.shape[0]):
        n = k.shape[2] if kv_lens is None else int(kv_lens[b])
        if n == 0:
            continue
        for h in range(q.shape[1]):
            j = h // G
            a, e, f = attention_backward_head(q[b, h], k[b, j, :n], v[b, j, :n], do[b, h], scale)
            dq[b, h] = a
            dk[b, j, :n] += e
            dv[b, j, :n] += f
    return dq, dk, dv


def rope_table(n, rot_dim, base=10000.0, factor=1.0, orig_len=0, low=1.0, high=32.0, attn_factor=1.0,
               first=0):
    """float64 cos, sin [n, rot_dim / 2]."""
    theta = np.empty(rot_dim // 2)
    for i in range(rot_dim // 2):
        t = base ** (-2.0 * i / rot_dim)
        g = 0.0
        if orig_len > 0:
            g = min(1.0, max(0.0, (orig_len * t / (2.0 * math.pi) - low) / (high - low)))
        theta[i] = g * t + (1.0 - g) * t / factor
    p = np.arange(first, first + n, dtype=np.float64)
    ang = p[:, None] * theta[None, :]
    return attn_factor * np.cos(ang), attn_factor * np.sin(ang)


def rope_rotate(x, cos, sin, interleaved=False, inverse=False):
    """Rows x [..., d] with a table row each (cos, sin [..., r / 2], broadcast)."""
    x = np.asarray(x, dtype=np.float64)
    c, s = np.asarray(cos, np.float64), np.asarray(sin, np.float64)
    s = -s if inverse else s
    half = c.shape[-1]
    y = x.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[..., a] = x[..., a] * c[..., i] - x[..., b] * s[..., i]
        y[..., b] = x[..., b] * c[..., i] + x[..., a] * s[..., i]
    return y


def block_tables(table, old_lens, new_lens, free_pages, page_size, capacity):
    """(table, seq_lens, cu_seqlens, slots, positions, pages used) after the step."""
    table = np.array(table)
    free = list(free_pages)
    slots, positions = [-1] * capacity, [-1] * capacity
    cu, lens, used, t = [0], [], 0, 0
    for b, (old, new) in enumerate(zip(old_lens, new_lens)):
        for lp in range(-(-int(old) // page_size), -(-(int(old) + int(new)) // page_size)):
            table[b, lp] = free[used]
            used += 1
        for pos in range(int(old), int(old) + int(new)):
            slots[t] = int(table[b, pos // page_size]) * page_size + pos % page_size
            positions[t] = pos
            t += 1
        lens.append(int(old) + int(new))
        cu.append(t)
    return table, np.array(lens), np.array(cu), np.array(slots), np.array(positions), used


def key_rows(k, positions, cos, sin, interleaved, signs):
    """Rows [T, H_kv, d] rotated by their positions' table rows and transformed."""
    x = np.asarray(k, dtype=np.float64)
    if cos is not None:
        x = rope_rotate(x, np.asarray(cos)[positions][:, None], np.asarray(sin)[positions][:, None], interleaved)
    return x if signs is None else incoherent_transform(x, signs)


def append_fp8(x, codes, descale, slots):
    """Codes [pages, page, H_kv, d] and descales [pages, H_kv] after rows x [T, H_kv, d]
    (held in float32, as the kernels do) go to their slots."""
    x = np.asarray(x).astype(np.float32)
    codes, descale = np.array(codes), np.array(descale, dtype=np.float32)
    page = codes.shape[1]
    slots = np.asarray(slots)
    for p in sorted(set((slots // page).tolist())):
        rows = np.nonzero(slots // page == p)[0]
        off = slots[rows] % page
        for h in range(codes.shape[2]):
            before = np.float32(0.0) if off.min() == 0 else descale[p, h]
            after = max(before, np.float32(np.abs(x[rows, h]).max()) / np.float32(E4M3_MAX))
            # a descale of 2^-90 at least, where there is anything but zeros
            after = max(after, np.float32(2.0 ** -90)) if after > 0 else np.float32(1.0)
            if off.min() == 0:
                codes[p, :, h] = 0
            elif after > before:
                ratio = np.float32(before / after)
                old = e4m3_decode(codes[p, :off.min(), h]).astype(np.float32)
                codes[p, :off.min(), h] = e4m3_encode((old * ratio).astype(np.float32))
            codes[p, off, h] = e4m3_encode((x[rows, h] / after).astype(np.float32))
            descale[p, h] = after
    return codes, descale
