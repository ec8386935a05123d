"""What a long conversation adds to the attention over the paged cache (oracle).  Test infrastructure only; float64 numpy, one
sequence and head at a time, written from the formulas.

Readings: a token's rotation takes each frequency's angle from its position on that frequency's axis; a shared prefix is seen whole
by all of its readers' tokens, in one softmax with the sequence's own tokens; a cached token's weight is the sum of the
probabilities that queries gave it; of a sequence the tokens of the largest weights stay, in their order, on pages whose
scale is the largest of those that the tokens had.
"""
from __future__ import annotations

import numpy as np

from .attention import quantise, read, values


def rope_rows(positions, axes, table):
    """rows [T, rot] of positions [n_axes, T]."""
    half = len(axes)
    rows = np.zeros((positions.shape[1], 2 * half))
    for f, axis in enumerate(axes):
        rows[:, f] = table[positions[axis], f]
        rows[:, half + f] = table[positions[axis], half + f]
    return rows


def _visible(total, n, i, causal, window, table, page, n_pages):
    """Places of a sequence's own tokens that its new token i sees."""
    j, pos = np.arange(total), total - n + i
    on_page = np.array([0 <= table[x // page] < n_pages for x in range(total)], bool)
    return np.nonzero(on_page & ((j <= pos) if causal else True) & ((j > pos - window) if window else True))[0]


def shared_attention(q, cache, q_start, kv_len, page_table, scale, prefix=None, causal=True, window=0):
    """(out, spread, lse): as attention.attention, and [T, Hq] the logarithms of the denominators.  prefix: (starts of the
    readers' tokens [n+1], lengths [n], page table)."""
    T, Hq, D = q.shape
    n_pages, Hkv, page = cache["k_codes"].shape[:3]
    out, spread, lse = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    if prefix is not None:
        shared = [(read(cache, "k", g, 0, int(n), prefix[2]), read(cache, "v", g, 0, int(n), prefix[2])) for g, n in enumerate(prefix[1])]
        reads = np.searchsorted(prefix[0], np.arange(T), side="right") - 1
    for b in range(len(kv_len)):
        t0, n, total = int(q_start[b]), int(q_start[b + 1] - q_start[b]), int(kv_len[b])
        k, v = read(cache, "k", b, 0, total, page_table), read(cache, "v", b, 0, total, page_table)
        for i in range(n):
            idx = _visible(total, n, i, causal, window, page_table[b], page, n_pages)
            kk, vv = k[idx], v[idx]
            if prefix is not None:
                pk, pv = shared[reads[t0 + i]]
                kk, vv = np.concatenate([pk, kk]), np.concatenate([pv, vv])
            if not len(kk):
                continue
            for h in range(Hq):
                z = (kk[:, h // (Hq // Hkv)] @ q[t0 + i, h]) * scale
                p = np.exp(z - z.max())
                lse[t0 + i, h] = z.max() + np.log(p.sum())
                p /= p.sum()
                out[t0 + i, h] = p @ vv[:, h // (Hq // Hkv)]
                spread[t0 + i, h] = p @ np.abs(vv[:, h // (Hq // Hkv)])
    return out, spread, lse


def weights(q, lse, cache, q_start, kv_len, page_table, scale, weight, fresh=False, causal=True, window=0):
    """(weights after the call, what it added, which were written): [n_pages, Hkv, page]."""
    Hq = q.shape[1]
    n_pages, Hkv, page = cache["k_codes"].shape[:3]
    out, added, written = np.array(weight, np.float64), np.zeros(weight.shape), np.zeros(weight.shape, bool)
    for b in range(len(kv_len)):
        t0, n, total = int(q_start[b]), int(q_start[b + 1] - q_start[b]), int(kv_len[b])
        if not n:
            continue
        k, first = read(cache, "k", b, 0, total, page_table), total - n
        add = np.zeros((total, Hkv))
        for i in range(n):
            idx = _visible(total, n, i, causal, window, page_table[b], page, n_pages)
            for h in range(Hq):
                if idx.size and np.isfinite(lse[t0 + i, h]) and np.isfinite(q[t0 + i, h]).all():
                    add[idx, h // (Hq // Hkv)] += np.exp((k[idx, h // (Hq // Hkv)] @ q[t0 + i, h]) * scale - lse[t0 + i, h])
        for j in range(max(0, first - window + 1) if window else 0, total):
            p, s = page_table[b, j // page], j % page
            if 0 <= p < n_pages:
                a = np.nan_to_num(add[j], nan=0.0)
                out[p, :, s] = a + (0.0 if fresh or j >= first else out[p, :, s])
                added[p, :, s], written[p, :, s] = a, True
    return out, added, written


def evict(cache, weight, kv_len, page_table, keep, new_table, sink, recent):
    """(new lengths, kept [B, Hkv, width]); cache (as attention.append's) and weight are changed in place."""
    n_pages, Hkv, page = cache["k_codes"].shape[:3]
    B, width = new_table.shape[0], new_table.shape[1] * page
    new_len, kept = np.zeros(B, np.int32), np.full((B, Hkv, width), -1, np.int32)
    before = {x: a.copy() for x, a in cache.items()}
    old = np.array(weight, np.float64)
    for b in range(B):
        n = int(kv_len[b])
        m = new_len[b] = min(n, int(keep[b]))
        j = np.arange(n)
        src, slot = page_table[b, j // page], j % page
        for h in range(Hkv):
            w = old[src, h, slot]
            w = np.where(w > 0, w, 0.0)
            w[(j < sink) | (j >= n - recent)] = np.inf
            tie = (j >= sink) & (j < n - recent)                      # an infinite weight comes after the tokens that stay anyway
            best = np.lexsort((j, tie, -w))[:m]
            tok = np.sort(best)
            kept[b, h, :m] = tok
            for i in range(0, m, page):
                t = tok[i:i + page]
                p, at = new_table[b, i // page], np.arange(len(t))
                weight[p, h, at] = old[src[t], h, slot[t]]
                for x in "kv":
                    e = before[x + "_scale"][src[t], h].astype(np.int64) - 127
                    cache[x + "_scale"][p, h] = e.max() + 127
                    for r in at:
                        codes = before[x + "_codes"][src[t[r]], h, slot[t[r]]]
                        cache[x + "_codes"][p, h, r] = codes if e[r] == e.max() else quantise(values(codes, int(e[r])), int(e.max()))
    return new_len, kept
