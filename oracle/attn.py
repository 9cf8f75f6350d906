"""The attention-layer operators from their definitions, in fp64 NumPy.

Test infrastructure, sharing no code with the HIP path: block tables and slot
maps, norms with the position rotation, attention over a paged cache, and the
commit of accepted paths.  Everything is written stream by stream and row by
row.
"""
from __future__ import annotations

import math

import numpy as np


def ancestors(parent, t):
    """Row t and its ancestors within one window (local indices, root first)."""
    path = []
    while t >= 0:
        path.append(t)
        t = parent[t]
    return path[::-1]


def local_parents(row_start, parent, s):
    """The window's parents (a chain's if ``parent`` is None)."""
    a, b = int(row_start[s]), int(row_start[s + 1])
    if parent is None:
        return list(range(-1, b - a - 1))
    return [int(p) for p in parent[a:b]]


def tables(page, row_start, parent, kv_len, page_count, free_count, free_pages, block_table, slots, positions):
    """The outputs of one call, from copies of its inputs and of its in/out arrays."""
    table, free = block_table.copy(), list(map(int, free_pages))
    counts, slots, positions = page_count.copy(), np.full_like(slots, -1), np.full_like(positions, -1)
    top = int(free_count)
    n = len(kv_len)
    want = []
    for s in range(n):
        rows = int(row_start[s + 1] - row_start[s])
        w = 0 if kv_len[s] < 0 else -(-(int(kv_len[s]) + rows) // page)
        if w > table.shape[1]:
            w = None                       # does not fit its table: as it is, without slots
        want.append(w)
    for s in range(n):
        if want[s] is not None:
            for j in range(want[s], int(page_count[s])):
                free[top] = int(table[s, j])
                top += 1
            if want[s] < page_count[s]:
                counts[s] = want[s]
    served = [want[s] is not None and kv_len[s] >= 0 for s in range(n)]
    out_of_pages = False
    for s in range(n):
        if want[s] is None or want[s] <= page_count[s]:
            continue
        grow = want[s] - int(page_count[s])
        out_of_pages = out_of_pages or grow > top
        if out_of_pages:
            served[s] = False
            for j in range(int(page_count[s]), want[s]):     # no pages: and none that an earlier round named
                if 0 <= table[s, j] < len(free):
                    table[s, j] = -1
            continue
        for j in range(int(page_count[s]), want[s]):
            top -= 1
            table[s, j] = free[top]
        counts[s] = want[s]
    for s in range(n):
        par = local_parents(row_start, parent, s)
        ok = served[s] and all(-1 <= p < t for t, p in enumerate(par))
        for t in range(len(par)):
            r = int(row_start[s]) + t
            at = int(kv_len[s]) + t
            slots[r] = int(table[s, at // page]) * page + at % page if ok else -1
            positions[r] = int(kv_len[s]) + len(ancestors(par, t)) - 1 if ok else -1
    return dict(block_table=table, free_pages=np.array(free, np.int32), page_count=counts, free_count=top, slots=slots,
                positions=positions)


def normed(x, w, eps):
    """RMS norm over the last axis; w None: x itself."""
    x = np.asarray(x, np.float64)
    if w is None:
        return x
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(w, np.float64)


def rotated(x, positions, inv_freq, interleaved, scale=1.0):
    """[R][H][d] with each row's first 2 len(inv_freq) channels rotated, and the
    magnitude of each result (the sum of its terms' magnitudes)."""
    y, mag = np.array(x, np.float64), np.abs(np.array(x, np.float64))
    half = len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        t = np.asarray(positions, np.float64) * float(inv_freq[i])
        c, s = np.cos(t)[:, None] * scale, np.sin(t)[:, None] * scale
        y[:, :, a], y[:, :, b] = x[:, :, a] * c - x[:, :, b] * s, x[:, :, b] * c + x[:, :, a] * s
        mag[:, :, a] = mag[:, :, b] = (np.abs(x[:, :, a]) + np.abs(x[:, :, b])) * abs(scale)
    return y, mag


def window(page, row_start, parent, kv_len, block_table, q, k, v, scale, gate=None):
    """Attention of every packed row: (out, mag, reach), [R][hq][d], [R][hq][d] and
    [R][hq].  k, v: the cache's values [pages][hkv][page][d].  mag is sum p |v|
    times the gate; reach the largest sum |q_c k_c| * |scale| of a visible key."""
    R, hq, d = q.shape
    hkv = k.shape[1]
    out, mag, reach = np.zeros((R, hq, d)), np.zeros((R, hq, d)), np.zeros((R, hq))
    for s in range(len(kv_len)):
        par = local_parents(row_start, parent, s)
        for t in range(len(par)):
            r = int(row_start[s]) + t
            keys = list(range(int(kv_len[s]))) + [int(kv_len[s]) + u for u in ancestors(par, t)]
            pages = np.array([block_table[s, j // page] for j in keys])
            offs = np.array([j % page for j in keys])
            for h in range(hq):
                kk, vv = k[pages, h // (hq // hkv), offs], v[pages, h // (hq // hkv), offs]
                x = kk @ q[r, h] * scale
                p = np.exp(x - np.max(x))
                p /= p.sum()
                g = 1.0 if gate is None else 1.0 / (1.0 + np.exp(-gate[r, h]))
                out[r, h], mag[r, h] = p @ vv * g, p @ np.abs(vv) * g
                reach[r, h] = np.max(np.abs(kk) @ np.abs(q[r, h])) * abs(scale)
    return out, mag, reach


def window_bound(ref, mag, reach, d):
    """How far a bf16 result may be from ``ref``: half a step of the result and of
    each weight (2^-8), and the exponentials' error from fp32 scores (d products
    and sums: d 2^-24 of their magnitude, twice, for the term and the sum) with
    2^-18 for the fp32 exponentials, sums and gate."""
    return 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -18 + 2.0 * (d + 8) * 2.0 ** -24 * reach[..., None]) * 1.01 * mag + 1e-37


def commit(page, row_start, parent, accept, kv_len, block_table, *pools):
    """The pools ([pages][hkv][page] + ...) and lengths after the accepted paths moved."""
    pools = [p.copy() for p in pools]
    out = np.array(kv_len).copy()
    for s in range(len(kv_len)):
        a, b = int(row_start[s]), int(row_start[s + 1])
        if not a <= accept[s] < b:
            continue
        par = local_parents(row_start, parent, s)
        if any(not -1 <= p < t for t, p in enumerate(par)):
            continue
        path = ancestors(par, int(accept[s]) - a)
        for j, t in enumerate(path):
            src, dst = int(kv_len[s]) + t, int(kv_len[s]) + j
            for p in pools:
                p[block_table[s, dst // page], :, dst % page] = p[block_table[s, src // page], :, src % page]
        out[s] += len(path)
    return pools, out


def default_scale(d):
    return 1.0 / math.sqrt(d)
