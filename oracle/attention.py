"""Attention over a paged cache held in 8 bits (oracle).  Test infrastructure only; float64 numpy, one sequence and head
at a time, written from the formulas.

Sources: Hy3 295B MoE practice, sections 1.1 (grouped query heads, per-head RMS norm of queries and keys, rotation) and
4 (cache written by slot); the inference note's section on KV paging.

Readings: pages of a fixed number of tokens, E4M3 codes and one power of two per (page, head), the smallest exponent
e >= -64 that brings the page's new tokens of that head within 448, never below the page's present exponent while it
holds earlier tokens of the same sequence; those are rounded again when it grows.  A NaN in a token's key or value is
kept as a NaN key row, its value elements as zeros.
"""
from __future__ import annotations

import math

import numpy as np

from .mx import e4m3_decode, e4m3_encode, e4m3_round


def norm_rotate(x, pos, cos_sin, rot, interleaved, weight=None, eps=1e-6):
    """x [n, heads, D] float64 of tokens at positions pos [n]."""
    x = np.array(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    out = x.copy()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c, s = (cos_sin[pos, i].astype(np.float64)[:, None], cos_sin[pos, rot // 2 + i].astype(np.float64)[:, None])
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., a] * s + x[..., b] * c
    return out


def scale_exponent(amax: float) -> int:
    e = -64
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def quantise(x, e):
    """E4M3 codes of x * 2^-e; infinities saturate, NaN becomes 0x7F."""
    x = np.asarray(x, np.float64)
    codes = e4m3_encode(e4m3_round(np.clip(np.nan_to_num(x, nan=0.0), -3.4e38, 3.4e38) * 2.0 ** -e))
    return np.where(np.isnan(x), np.uint8(0x7F), codes).astype(np.uint8)


def values(codes, e):
    v = e4m3_decode(codes) * 2.0 ** e
    return np.where((np.asarray(codes) & 0x7F) == 0x7F, np.nan, v)


def append(k, v, cache, q_start, kv_len, page_table):
    """k, v [T, Hkv, D] float64 (already normalised and rotated); cache: dict of k_codes, v_codes [n, Hkv, page, D] and
    k_scale, v_scale [n, Hkv] uint8, changed in place."""
    k, v = np.array(k), np.array(v)
    bad = np.isnan(k).any(-1) | np.isnan(v).any(-1)
    k[bad] = np.nan
    v = np.where(np.isnan(v), 0.0, v)
    page = cache["k_codes"].shape[2]
    for b in range(len(kv_len)):
        t0, n, total = int(q_start[b]), int(q_start[b + 1] - q_start[b]), int(kv_len[b])
        first = total - n
        for j in range(first // page, (total + page - 1) // page) if n else ():
            lo, hi = max(first, j * page), min(total, (j + 1) * page)
            p = page_table[b, j]
            for name, x in (("k", k), ("v", v)):
                codes, scale = cache[name + "_codes"], cache[name + "_scale"]
                for h in range(codes.shape[1]):
                    new = x[t0 + lo - first:t0 + hi - first, h]
                    mag = np.abs(new[np.isfinite(new)])
                    e = scale_exponent(mag.max() if mag.size else 0.0)
                    old = int(scale[p, h]) - 127
                    if j * page < first:
                        e = max(e, old)
                        if e > old:
                            kept = codes[p, h, :first - j * page]
                            codes[p, h, :first - j * page] = quantise(values(kept, old), e)
                    scale[p, h] = e + 127
                    codes[p, h, lo - j * page:hi - j * page] = quantise(new, e)


def read(cache, name, b, lo, hi, page_table):
    """Tokens [lo, hi) of sequence b, [hi - lo, Hkv, D] float64; NaN rows for tokens on no page."""
    codes, scale = cache[name + "_codes"], cache[name + "_scale"]
    page = codes.shape[2]
    out = np.full((max(0, hi - lo), codes.shape[1], codes.shape[3]), np.nan)
    for i in range(lo, hi):
        p = page_table[b, i // page]
        if 0 <= p < codes.shape[0]:
            out[i - lo] = values(codes[p, :, i % page], scale[p].astype(np.int64)[:, None] - 127)
    return out


def attention(q, cache, q_start, kv_len, page_table, scale, causal=True, window=0):
    """(out, spread) [T, Hq, D]: the attention output and sum_j p_j |v_j|, which rounding errors are measured by."""
    T, Hq, D = q.shape
    Hkv, page = cache["k_codes"].shape[1:3]
    out, spread = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    for b in range(len(kv_len)):
        t0, n, total = int(q_start[b]), int(q_start[b + 1] - q_start[b]), int(kv_len[b])
        k, v = read(cache, "k", b, 0, total, page_table), read(cache, "v", b, 0, total, page_table)
        on_page = np.array([0 <= page_table[b, j // page] < cache["k_codes"].shape[0] for j in range(total)], bool)
        for i in range(n):
            pos = total - n + i
            j = np.arange(total)
            seen = on_page & ((j <= pos) if causal else True) & ((j > pos - window) if window else True)
            idx = np.nonzero(seen)[0]
            if not idx.size:
                continue
            for h in range(Hq):
                z = (k[idx, h // (Hq // Hkv)] @ q[t0 + i, h]) * scale
                p = np.exp(z - z.max())
                p /= p.sum()
                vv = v[idx, h // (Hq // Hkv)]
                out[t0 + i, h] = p @ vv
                spread[t0 + i, h] = p @ np.abs(vv)
    return out, spread


def rope_table(max_pos, rot, base):
    pos = np.arange(max_pos, dtype=np.float64)[:, None]
    angle = pos * np.array([math.pow(base, -2.0 * i / rot) for i in range(rot // 2)])
    return np.concatenate([np.cos(angle), np.sin(angle)], 1)
