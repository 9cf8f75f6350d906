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


def prompt(page, row_start, kv_len, block_table, q, k, v, scale, gate=None):
    """As ``window`` for chains of any length, a stream and head at a time."""
    R, hq, d = q.shape
    G = hq // k.shape[1]
    out, mag, reach = np.zeros((R, hq, d)), np.zeros((R, hq, d)), np.zeros((R, hq))
    for s in range(len(kv_len)):
        a, b, c = int(row_start[s]), int(row_start[s + 1]), int(kv_len[s])
        if a == b:
            continue
        at = np.arange(c + b - a)
        pages, offs = np.asarray(block_table)[s][at // page], at % page
        hidden = at[None, :] > c + np.arange(b - a)[:, None]
        for h in range(hq):
            kk, vv = k[pages, h // G, offs], v[pages, h // G, offs]
            x = np.where(hidden, -np.inf, q[a:b, h] @ kk.T * scale)
            p = np.exp(x - x.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            g = 1.0 if gate is None else 1.0 / (1.0 + np.exp(-gate[a:b, h]))
            out[a:b, h], mag[a:b, h] = p @ vv * g, p @ np.abs(vv) * g
            reach[a:b, h] = np.where(hidden, 0.0, np.abs(q[a:b, h]) @ np.abs(kk).T).max(1) * abs(scale)
    return out, mag, reach


E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx_values(codes, exps):
    """The values of MXFP4 rows: codes [..][d / 2] (even channels in the low halves), exps [..][d / 32]."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    y = np.where(c >= 8, -1.0, 1.0) * E2M1[c & 7]
    e = np.repeat(exps.astype(np.int64), 32, -1)
    return np.where(e > 252, np.nan, np.ldexp(y, np.where(e > 252, 127, e) - 127))


def mx_quantise(y):
    """fp32 rows [..][d] in MXFP4: the exponent that puts a block's largest
    magnitude into [3.5, 7) (within 25 .. 252; 255 if a value is not finite), and
    of the 8 magnitudes the nearest, of two as near the one with the even code."""
    y = np.asarray(y, np.float32).astype(np.float64)
    b = y.reshape(*y.shape[:-1], -1, 32)
    fin = np.isfinite(b).all(-1)
    top = np.where(fin, np.abs(np.where(np.isfinite(b), b, 0.0)).max(-1), 1.0)
    e = np.full(top.shape, 25)
    for x in range(25, 252):                       # the least exponent that the rule allows
        e = np.where(top >= 7.0 * 2.0 ** (x - 127), x + 1, e)
    a = np.where(fin[..., None], np.abs(np.where(np.isfinite(b), b, 0.0)) / np.ldexp(1.0, e - 127)[..., None], 0.0)
    far = np.abs(a[..., None] - E2M1)
    near = far == far.min(-1, keepdims=True)
    order = np.array([0, 2, 4, 6, 1, 3, 5, 7])
    code = order[np.argmax(near[..., order], -1)]
    code = np.where(fin[..., None], code + 8 * np.signbit(b), 0).astype(np.uint8).reshape(y.shape)
    return code[..., 0::2] | code[..., 1::2] << 4, np.where(fin, e, 255).astype(np.uint8)


def read(page, row_start, first, block_table, pool, out):
    """The rows of ``out`` [R][hkv][d] after reading pool's values [pages][hkv][page][d] back."""
    out = out.copy()
    for s in range(len(first)):
        for r in range(int(row_start[s]), int(row_start[s + 1])):
            at = int(first[s]) + r - int(row_start[s])
            out[r] = pool[block_table[s, at // page], :, at % page]
    return out


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
