"""Attention beside the MoE layer, in float64 NumPy: cache slots, head norm and
rotation, causal attention over packed prompts, attention of single tokens over
paged keys with a shared prefix.

The formulas are the definitions themselves, one row at a time; nothing is
shared with the HIP path.
"""
from __future__ import annotations

import numpy as np


def kv_slots(cached, new, free_pages, table, page, max_new, position_base=0):
    """-> (table, slots [max_new], positions [max_new], cu_new [B + 1], counts [3])."""
    table = np.array(table, dtype=np.int64)
    blocks = table.shape[1]
    slots = np.full(max_new, -1, np.int64)
    positions = np.zeros(max_new, np.int64)
    cu = [0]
    needed = lost = 0
    for b, (c, n) in enumerate(zip(cached, new)):
        c, n = min(max(int(c), 0), blocks * page), max(int(n), 0)
        for block in range(-(-c // page), min(-(-(c + n) // page), blocks)):
            table[b, block] = free_pages[needed] if needed < len(free_pages) else -1
            needed += 1
        for i in range(n):
            pos = c + i
            t = cu[-1] + i
            held = pos // page < blocks and table[b, pos // page] >= 0
            lost += not held
            if t < max_new:
                positions[t] = position_base + pos
                slots[t] = table[b, pos // page] * page + pos % page if held else -1
        cu.append(cu[-1] + n)
    return table, slots, positions, np.array(cu), np.array([min(needed, len(free_pages)), needed, lost])


def norm_rope(x, weight, eps, cos_sin, positions, interleaved):
    """x [T, heads, D] float64; weight [D] or None; cos_sin [P, rot] or None."""
    y = np.array(x, dtype=np.float64)
    T, H, D = y.shape
    if weight is not None:
        y = y / np.sqrt((y ** 2).sum(axis=-1, keepdims=True) / D + eps) * weight
    if cos_sin is None:
        return y
    rot = cos_sin.shape[1]
    out = y.copy()
    for t in range(T):
        p = min(max(int(positions[t]), 0), cos_sin.shape[0] - 1)
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            c, s = float(cos_sin[p, i]), float(cos_sin[p, rot // 2 + i])
            out[t, :, a] = y[t, :, a] * c - y[t, :, b] * s
            out[t, :, b] = y[t, :, b] * c + y[t, :, a] * s
    return out


def attend(q, k, v, scale):
    """One query q [D] over keys k [n, D], v [n, Dv] -> (out [Dv], lse); no key: (0, -inf)."""
    if k.shape[0] == 0:
        return np.zeros(v.shape[1]), -np.inf
    with np.errstate(invalid="ignore", over="ignore"):
        s = (k @ q) * scale
        m = np.max(s)
        w = np.exp(s - m)
        return (w / w.sum()) @ v, m + np.log(w.sum())


def attn_prompt(q, k, v, cu_q, cu_k, scale):
    """q [Tq, Hq, D], k [Tk, Hkv, D], v [Tk, Hkv, Dv] float64 -> (out, lse)."""
    Tq, Hq, _ = q.shape
    G = Hq // k.shape[1]
    out, lse = np.zeros((Tq, Hq, v.shape[2])), np.full((Tq, Hq), -np.inf)
    for b in range(len(cu_q) - 1):
        lq, lk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        for i in range(lq):
            n = max(0, min(lk, i + lk - lq + 1))
            rows = slice(cu_k[b], cu_k[b] + n)
            for h in range(Hq):
                out[cu_q[b] + i, h], lse[cu_q[b] + i, h] = attend(q[cu_q[b] + i, h], k[rows, h // G], v[rows, h // G], scale)
    return out, lse


def attn_decode(q, k_cache, v_cache, table, lens, prefix_table, prefix_len, scale):
    """q [B, Hq, D]; caches [pages, page, Hkv, D] float64 -> (out, lse)."""
    B, Hq, _ = q.shape
    _, page, Hkv, _ = k_cache.shape
    G = Hq // Hkv
    out, lse = np.zeros((B, Hq, v_cache.shape[3])), np.full((B, Hq), -np.inf)
    for b in range(B):
        at = [(prefix_table[j // page], j % page) for j in range(prefix_len)]
        at += [(table[b][j // page], j % page) for j in range(max(0, int(lens[b])))]
        pg, off = np.array([x for x, _ in at], np.int64), np.array([y for _, y in at], np.int64)
        for h in range(Hq):
            out[b, h], lse[b, h] = attend(q[b, h], k_cache[pg, off, h // G], v_cache[pg, off, h // G], scale)
    return out, lse
