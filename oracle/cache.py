"""A cache held in 4 bits, the pages of a cache and the norms of the residual stream, in NumPy (float64).

The formulas are the definitions themselves; nothing is shared with the HIP path.
"""
from __future__ import annotations

import numpy as np

from .formats import e2m1_value, e4m3_value, round_to_e2m1_magnitude, round_to_e4m3, unpack_codes


def nvfp4_rows(x, scale):
    """float64 [..., dim] -> (codes u8 [..., dim / 2], E4M3 scales u8 [..., dim / 16]) under the global ``scale``."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(x.shape[:-1] + (x.shape[-1] // 16, 16))
    s = round_to_e4m3(np.abs(b).max(axis=-1) / 6.0 / scale)
    unit = (e4m3_value(s) * scale)[..., None]
    code = np.where(unit > 0, round_to_e2m1_magnitude(np.abs(b) / np.where(unit > 0, unit, 1.0)), 0)
    code = (code | np.where(np.signbit(b) & (unit > 0), 8, 0)).astype(np.uint8).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), s


def nvfp4_values(codes, scales, scale):
    v = e2m1_value(unpack_codes(codes))
    return (v.reshape(v.shape[:-1] + (v.shape[-1] // 16, 16)) * (e4m3_value(scales) * scale)[..., None]).reshape(v.shape)


def cache_values(k, k_scale, v, v_scale, k_global, v_global):
    """The four arrays of a cache -> keys, values [pages, page, heads, dim]."""
    kk = nvfp4_values(k, k_scale, k_global)
    vv = nvfp4_values(v, np.swapaxes(v_scale, 2, 3), v_global)
    return np.swapaxes(kk, 1, 2), np.swapaxes(vv, 1, 2)


def gather(rows, table, cu, total, prefix_table, prefix_len, out):
    """rows [pages, page, ...] -> out [total, ...]: the sequences' first keys, those of the prefix before their own."""
    out = np.array(out)
    page = rows.shape[1]
    for b in range(len(cu) - 1):
        for i in range(cu[b + 1] - cu[b]):
            j = i if i < prefix_len else i - prefix_len
            tab = prefix_table if i < prefix_len else table[b]
            p = tab[j // page] if j // page < len(tab) else -1
            out[cu[b] + i] = rows[p, j % page] if 0 <= p < rows.shape[0] else 0
    return out


def held(length, page, blocks):
    return min(-(-max(int(length), 0) // page), blocks)


def fork(table, lens, parents, children, free_pages, page, buffers):
    """-> (table, lens, buffers, counts)."""
    table, lens, buffers = np.array(table), np.array(lens), [np.array(b) for b in buffers]
    n, blocks = table.shape
    pages = buffers[0].shape[0]
    need = taken = 0
    for p, c in zip(parents, children):
        if not (0 <= p < n and 0 <= c < n) or p == c:
            continue
        length = min(max(int(lens[p]), 0), blocks * page)
        whole = length // page
        table[c, :whole] = table[p, :whole]
        lens[c] = length
        if length % page:
            new = free_pages[need] if need < len(free_pages) and 0 <= free_pages[need] < pages else -1
            need += 1
            taken += new >= 0
            table[c, whole] = new
            if new < 0:
                lens[c] = whole * page
            elif 0 <= table[p, whole] < pages:
                for b in buffers:
                    b[new] = b[table[p, whole]]
    return table, lens, buffers, np.array([taken, need])


def live(table, lens, page, num_pages):
    pages = {int(p) for row, n in zip(table, lens) for p in row[:held(n, page, len(row))]}
    return sorted(p for p in pages if 0 <= p < num_pages)


def free_pages(table, lens, page, num_pages):
    """-> (free [num_pages]: ascending, then -1; counts)."""
    used = set(live(table, lens, page, num_pages))
    free = [p for p in range(num_pages) if p not in used]
    return np.array(free + [-1] * len(used)), np.array([len(free), len(used)])


def compact(table, lens, page, buffers):
    """-> (table, buffers, counts)."""
    buffers = [np.array(b) for b in buffers]
    pages = buffers[0].shape[0]
    used = live(table, lens, page, pages)
    n = len(used)
    holes = [p for p in range(n) if p not in set(used)]
    to = dict(zip([p for p in used if p >= n], holes))
    out = np.full(np.shape(table), -1, np.int64)
    for b, (row, length) in enumerate(zip(table, lens)):
        for i in range(held(length, page, len(row))):
            if 0 <= row[i] < pages:
                out[b, i] = to.get(int(row[i]), row[i])
    for src, dst in to.items():
        for b in buffers:
            b[dst] = b[src]
    return out, buffers, np.array([n, len(to)])


def rms_norm(x, weight, eps):
    return x / np.sqrt((x * x).sum(axis=-1, keepdims=True) / x.shape[-1] + eps) * weight


def block_norm(x, weight, residual=None, post_weight=None, gate=None, scale=1.0, eps=1e-6):
    """float64 -> (h, y)."""
    b = np.asarray(x, dtype=np.float64)
    if post_weight is not None:
        b = rms_norm(b, post_weight, eps)
    if gate is not None:
        b = b * gate
    h = b * scale
    if residual is not None:
        h = residual + h
    return h, rms_norm(h, weight, eps)
