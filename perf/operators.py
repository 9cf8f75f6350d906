"""Measured cases of the attention-layer operators: block tables and slot maps
built on the device (``kv_tables``), per-head norms with the position rotation
and the paged cache write (``attn_prep``), attention of steps, windows and
draft trees over the paged cache (``attn_window``), and the commit of accepted
tree paths (``attn_commit``).

``run`` computes them in elementary torch operations, or, where ``own`` is
true, through the framework's entry points.  ``exact`` computes the same from
the definitions in 64 bits.

Layouts: a cache is K and V of ``[pages][kv heads][page size][d]`` (bf16, or
e4m3 with one fp32 scale a row in ``[pages][kv heads][page size]``); stream s
keeps its cache row i in page ``block_table[s][i // page size]``, row
``i % page size``; packed rows of stream s are ``row_start[s]`` up to
``row_start[s + 1]``; ``parent`` holds a tree row's parent within its window
(-1: the row follows the cache).
"""
import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
TINY = 2.0 ** -100       # the least row maximum an e4m3 scale is made from
MAX_ROWS = 16            # rows of a verify window


def _gdn():
    from verify_causal_conv1d_amd import gdn
    return gdn


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # One small request's next token: nothing but latency.
        dict(name="tables step 1", op="tables", n=1, rows=1, lo=100, hi=100, page=16, tree=False, prompt=0),
        # A round of 16 streams' draft trees; two streams have finished.
        dict(name="tables round 16", op="tables", n=16, rows=16, lo=400, hi=9000, page=64, tree=True, prompt=0),
        # A full server: 500 streams step, 63 release their pages, 62 are admitted.
        dict(name="tables server 500", op="tables", n=500, rows=4, lo=60, hi=30000, page=16, tree=False, prompt=300),
        # One stream's next token on the 27B-like layer's attention heads.
        dict(name="prep step 1", op="prep", rows=1, hq=24, hkv=4, d=256, rot=64, page=64, e4m3=False, inter=False, pos=5000),
        # 16 x 16 verify rows into an e4m3 cache, interleaved pairs, the whole head rotated.
        dict(name="prep verify e4m3", op="prep", rows=249, hq=32, hkv=8, d=128, rot=128, page=16, e4m3=True, inter=True, pos=131000),
        # The packed prompt pass of the 27B-like layer.
        dict(name="prep prompts", op="prep", rows=8306, hq=24, hkv=4, d=256, rot=64, page=64, e4m3=False, inter=False, pos=0),
        # One small request's next token.
        dict(name="attn step 1", op="attn", n=1, rows=1, lo=100, hi=100, hq=4, hkv=2, d=64, page=16, e4m3=False, tree=False, gate=False),
        # Decode of 16 ragged streams on the 27B-like layer's heads, gated.
        dict(name="attn step 16", op="attn", n=16, rows=1, lo=1000, hi=16384, hq=24, hkv=4, d=256, page=64, e4m3=False, tree=False, gate=True),
        # One stream at the end of a 256K context, e4m3 cache.
        dict(name="attn step 256K e4m3", op="attn", n=1, rows=1, lo=262143, hi=262143, hq=24, hkv=4, d=256, page=256, e4m3=True, tree=False, gate=True),
        # 16 ragged streams' draft trees of up to 16 rows, the verify round.
        dict(name="attn tree 16", op="attn", n=16, rows=16, lo=700, hi=8191, hq=24, hkv=4, d=256, page=64, e4m3=False, tree=True, gate=True),
        # The accepted paths of one stream's tree and of a round of 16 streams.
        dict(name="commit 1", op="commit", n=1, rows=7, lo=333, hi=333, hkv=2, d=128, page=16, e4m3=False),
        dict(name="commit 16 e4m3", op="commit", n=16, rows=16, lo=100, hi=2000, hkv=4, d=256, page=64, e4m3=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "prep", "attn", "attn", "commit"])
    page = rng.choice([16, 32, 64, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 6, 8])
    d = rng.choice([64, 128, 256])
    e4m3 = rng.random() < 0.4
    if op == "tables":
        hi = _log(rng, 1, 30000)
        tree = rng.random() < 0.5
        return dict(op=op, n=_log(rng, 1, 500), rows=rng.randint(1, MAX_ROWS), lo=_log(rng, 1, hi), hi=hi, page=page,
                    tree=tree, prompt=0 if tree else _log(rng, 1, 300))
    if op == "prep":
        rows = _log(rng, 1, min(8306, 8306 * 32 * 256 // ((hq + 2 * hkv) * d)))
        return dict(op=op, rows=rows, hq=hq, hkv=hkv, d=d, rot=2 * rng.randint(1, d // 2), page=page, e4m3=e4m3,
                    inter=rng.random() < 0.5, pos=_log(rng, 1, 250000))
    if op == "commit":
        hi = _log(rng, 1, 2000)
        return dict(op=op, n=_log(rng, 1, 16), rows=rng.randint(1, MAX_ROWS), lo=_log(rng, 1, hi), hi=hi,
                    hkv=min(hkv, 4), d=d, page=page, e4m3=e4m3)
    n = _log(rng, 1, 64)
    rows = rng.choice([1, 1, rng.randint(2, MAX_ROWS), MAX_ROWS])
    hi = _log(rng, 1, min(200000, (1 << 28) // (n * hkv * d), (24 << 20) * 2 // (n * rows * hq)))
    return dict(op=op, n=n, rows=rows, lo=_log(rng, 1, hi), hi=hi, hq=hq, hkv=hkv, d=d, page=page, e4m3=e4m3,
                tree=rows > 1 and rng.random() < 0.5, gate=rng.random() < 0.5)


# ---- sizes that follow from a case alone --------------------------------------

def _lens(c):
    """Cache rows of each stream: spread over lo..hi by their logarithm, in a mixed order."""
    n = c["n"]
    if n == 1:
        return [c["hi"]]
    r = [int(round(c["lo"] * (c["hi"] / c["lo"]) ** (i / (n - 1)))) for i in range(n)]
    step = next(k for k in range(max(1, n // 3), n + 1) if math.gcd(k, n) == 1)
    return [r[(i * step) % n] for i in range(n)]


def _rows(c):
    """Window rows of each stream: one for steps, else ragged up to the case's rows (the first has them all)."""
    m = c["rows"]
    return [m if m == 1 or i == 0 else 1 + (7 * i + 3) % m for i in range(c["n"])]


def _streams(c):
    """(kv_len, rows, pages held) of each stream of a tables case: of every eight,
    one has finished (kv_len -1) and, where there are prompts, one is admitted."""
    got = []
    for i, (ln, m) in enumerate(zip(_lens(c), _rows(c))):
        held = -(-ln // c["page"])
        if i % 8 == 3:
            got.append((-1, 0, held))
        elif i % 8 == 5 and c["prompt"]:
            got.append((0, 1 + (c["prompt"] * (1 + i % 5)) // 5, 0))
        else:
            got.append((ln, m, held))
    return got


def _visible(ln, m):
    """Keys that a chain window's rows attend to, all rows together."""
    return m * ln + m * (m + 1) // 2


def work(case):
    c = case
    if c["op"] == "tables":
        st, page = _streams(c), c["page"]
        rows = sum(m for _, m, _ in st)
        moved = sum(abs(-(-(max(ln, 0) + m) // page) - h) if ln >= 0 else h for ln, m, h in st)
        # lengths, counts and row starts in, counts out; each moved page is read and written; slots and positions out
        return {"bytes": 4.0 * (4 * c["n"] + 1 + 2 * moved + (3 if c["tree"] else 2) * rows), "flops": 0.0}
    if c["op"] == "prep":
        e = 1 if c["e4m3"] else 2
        kv = 2 * c["hkv"] * c["d"]
        per = 2 * (2 * c["hq"] * c["d"] + kv) + e * kv + (8 * c["hkv"] if c["e4m3"] else 0) + 8
        return {"bytes": float(c["rows"] * per), "flops": float(c["rows"] * (c["hq"] + c["hkv"]) * (4 * c["d"] + 6 * c["rot"] // 2))}
    e = 1 if c["e4m3"] else 2
    lens, rows = _lens(c), _rows(c)
    if c["op"] == "commit":
        # a path is about half its tree; each of its rows is read and written
        moved = sum((m + 1) // 2 for m in rows)
        return {"bytes": float(4 * c["hkv"] * moved * (c["d"] * e + (4 if c["e4m3"] else 0)) + 16 * c["n"]), "flops": 0.0}
    keys = sum(ln + m for ln, m in zip(lens, rows))
    pairs = sum(_visible(ln, m) for ln, m in zip(lens, rows))
    kv = 2.0 * keys * c["hkv"] * (c["d"] * e + (4 if c["e4m3"] else 0))
    return {"bytes": kv + sum(rows) * c["hq"] * c["d"] * 2.0 * (3 if c["gate"] else 2), "flops": 4.0 * c["hq"] * c["d"] * pairs}


# ---- inputs -------------------------------------------------------------------

def _starts(rows):
    s = [0]
    for m in rows:
        s.append(s[-1] + m)
    return s


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _parents(rows, host):
    """Draft trees: row 0 follows the cache, row t a row drawn from the four before it."""
    p = []
    for m in rows:
        for t in range(m):
            p.append(-1 if t == 0 else t - 1 - int(torch.randint(0, min(t, 4), (1,), generator=host)))
    return _int(p)


def _quantise(x):
    """e4m3 rows with scale = max|row| / 448."""
    s = x.float().abs().amax(-1).clamp(min=TINY) / E4M3_MAX
    return (x.float() / s[..., None]).to(torch.float8_e4m3fn), s


def _cache(c, pages, g):
    """K and V pools with values as the norm and the projection leave them."""
    shape = (pages, c["hkv"], c["page"], c["d"])
    k = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    v = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    if not c["e4m3"]:
        return dict(k=k, v=v, k_scale=None, v_scale=None)
    (k, ks), (v, vs) = _quantise(k), _quantise(v)
    return dict(k=k, v=v, k_scale=ks, v_scale=vs)


def _paged(c, lens, rows, g, spare=5):
    """A block table over shuffled pages with room for every stream's window."""
    need = [-(-(ln + m) // c["page"]) for ln, m in zip(lens, rows)]
    pages = sum(need) + spare
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for s, k in enumerate(need):
        table[s, :k] = perm[at:at + k]
        at += k
    return table, pages


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    host = torch.Generator().manual_seed(int(seed))
    if c["op"] == "tables":
        st, page = _streams(c), c["page"]
        held = [h for _, _, h in st]
        want = [-(-(max(ln, 0) + m) // page) for ln, m, _ in st]
        pages = sum(max(h, w) for h, w in zip(held, want)) + 7
        perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        blocks = max(max(held), max(want)) + 2
        table = torch.full((c["n"], blocks), -1, dtype=torch.int32, device=DEV)
        at = 0
        for s, h in enumerate(held):
            table[s, :h] = perm[at:at + h]
            at += h
        rows = [m for _, m, _ in st]
        free = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
        free[:pages - at] = perm[at:]
        total = sum(rows)
        return dict(c=c, row_start=_int(_starts(rows)), kv_len=_int([ln for ln, _, _ in st]), page_count=_int(held),
                    parent=_parents(rows, host) if c["tree"] else None, free_pages=free, free_count=_int([pages - at]),
                    block_table=table, page_count_out=torch.zeros(c["n"], dtype=torch.int32, device=DEV),
                    free_count_out=torch.zeros(1, dtype=torch.int32, device=DEV),
                    slots=torch.zeros(total, dtype=torch.int32, device=DEV),
                    positions=torch.zeros(total, dtype=torch.int32, device=DEV))
    if c["op"] == "prep":
        R, hq, hkv, d = c["rows"], c["hq"], c["hkv"], c["d"]
        pages = -(-R // c["page"]) + 3
        # the projection's output: each query head beside its gate, then the keys, then the values
        x = torch.randn((R, (2 * hq + 2 * hkv) * d), generator=g, device=DEV, dtype=torch.bfloat16)
        q = x[:, :2 * hq * d].view(R, hq, 2 * d)[:, :, :d]
        k = x[:, 2 * hq * d:(2 * hq + hkv) * d].view(R, hkv, d)
        v = x[:, (2 * hq + hkv) * d:].view(R, hkv, d)
        slots = torch.randperm(pages * c["page"], generator=g, device=DEV)[:R].to(torch.int32)
        inv = (1e7 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])).to(torch.float32).to(DEV)
        w = 1.0 + 0.2 * torch.randn((2, d), generator=g, device=DEV)
        return dict(c=c, q=q, k=k, v=v, q_norm=w[0].contiguous(), k_norm=w[1].contiguous(), inv_freq=inv, slots=slots,
                    positions=(torch.arange(R, device=DEV) % 4722 + c["pos"]).to(torch.int32),
                    q_out=torch.zeros((R, hq, d), dtype=torch.bfloat16, device=DEV), cache=_cache(c, pages, g))
    lens, rows = _lens(c), _rows(c)
    table, pages = _paged(c, lens, rows, g)
    total = sum(rows)
    s = dict(c=c, row_start=_int(_starts(rows)), kv_len=_int(lens), block_table=table, cache=_cache(c, pages, g))
    if c["op"] == "commit":
        s["parent"] = _parents(rows, host)
        # a row about half way into each window, so that its path skips rows
        s["accept"] = _int([a + m - 1 - int(torch.randint(0, (m + 1) // 2, (1,), generator=host)) for a, m in zip(_starts(rows), rows)])
        s["kv_len_out"] = torch.zeros(c["n"], dtype=torch.int32, device=DEV)
        return s
    hq, d = c["hq"], c["d"]
    # queries a little larger than unit norm: softmax rows with a few leading keys
    s["q"] = (1.5 * torch.randn((total, hq, d), generator=g, device=DEV)).to(torch.bfloat16)
    x = torch.randn((total, hq, 2 * d), generator=g, device=DEV, dtype=torch.bfloat16)
    s["gate"] = x[:, :, d:] if c["gate"] else None
    s["parent"] = _parents(rows, host) if c["tree"] else None
    s["out"] = torch.zeros((total, hq, d), dtype=torch.bfloat16, device=DEV)
    s["max_kv"] = max(ln + m for ln, m in zip(lens, rows))
    if own:  # the memory for partial results that a program allocates once for its largest call
        b = _gdn().attn_workspace_bytes(hq, c["hkv"], d, c["n"], total, c["rows"], s["max_kv"])
        s["workspace"] = torch.empty(max(b, 16), dtype=torch.uint8, device=DEV)
    return s


# ---- one pass -------------------------------------------------------------------

def run(state):
    s = state
    return {"tables": _tables, "prep": _prep, "attn": _attn, "commit": _commit}[s["c"]["op"]](s)


def _tables(s):
    c = s["c"]
    if own:
        _gdn().kv_tables(s["row_start"], s["kv_len"], s["page_count"], s["free_count"], s["free_pages"], s["block_table"],
                         s["slots"], s["positions"], page_size=c["page"], parent=s["parent"],
                         page_count_out=s["page_count_out"], free_count_out=s["free_count_out"])
    else:
        _plain_tables(s)
    return {k: s[k] for k in ("block_table", "free_pages", "page_count_out", "free_count_out", "slots", "positions")}


def _prep(s):
    c, m = s["c"], s["cache"]
    if own:
        _gdn().attn_prep(s["q"], s["k"], s["v"], s["q_norm"], s["k_norm"], s["inv_freq"], s["positions"], s["slots"],
                         s["q_out"], m["k"], m["v"], m["k_scale"], m["v_scale"], eps=1e-6, interleaved=c["inter"])
    else:
        _plain_prep(s)
    return dict(m, q=s["q_out"])


def _attn(s):
    m = s["cache"]
    if own:
        _gdn().attn_window(s["row_start"], s["kv_len"], s["block_table"], s["q"], m["k"], m["v"], s["out"], s["workspace"],
                           max_kv=s["max_kv"], max_rows=s["c"]["rows"], parent=s["parent"], gate=s["gate"],
                           k_scale=m["k_scale"], v_scale=m["v_scale"])
    else:
        _plain_attn(s)
    return s["out"]


def _commit(s):
    m = s["cache"]
    if own:
        _gdn().attn_commit(s["row_start"], s["accept"], s["kv_len"], s["block_table"], m["k"], m["v"], k_scale=m["k_scale"],
                           v_scale=m["v_scale"], parent=s["parent"], kv_len_out=s["kv_len_out"], max_rows=s["c"]["rows"])
    else:
        _plain_commit(s)
    return dict(m, kv_len=s["kv_len_out"])


# ---- the plain forms ---------------------------------------------------------------

def _owners(row_start, total):
    """Stream and place within its window of each packed row."""
    r = torch.arange(total, device=row_start.device)
    s = torch.searchsorted(row_start[1:].long(), r, right=True)
    return s, r - row_start.long()[s]


def _ancestors(row_start, parent, total, m):
    """[n][m][m]: row t sees row j, for rows that are there (m >= every window)."""
    n = row_start.shape[0] - 1
    s, t = _owners(row_start, total)
    up = torch.zeros((n, m, m + 1), device=row_start.device)
    up[s, t, torch.where(parent < 0, m, parent).long()] = 1.0
    a = torch.eye(m, device=row_start.device) + up[:, :, :m]
    a = a @ a          # after four squarings: every chain of up to 16 parents
    a = (a @ a).clamp(max=1.0)
    a = (a @ a).clamp(max=1.0)
    a = (a @ a).clamp(max=1.0)
    return a > 0


def _plain_tables(s):
    page = s["c"]["page"]
    kv, have, table, free = s["kv_len"].long(), s["page_count"].long(), s["block_table"], s["free_pages"]
    start, total = s["row_start"], s["slots"].shape[0]
    rows = (start[1:] - start[:-1]).long()
    want = torch.where(kv < 0, 0, (kv + rows + page - 1) // page)
    drop, grow = (have - want).clamp(min=0), (want - have).clamp(min=0)
    drop_at, grow_at = drop.cumsum(0) - drop, grow.cumsum(0) - grow
    avail = s["free_count"].long() + drop.sum()
    ok = (grow_at + grow <= avail) & (kv >= 0)
    j = torch.arange(table.shape[1], device=table.device)[None]
    # released pages go on top of the free list, in stream order
    out = (j >= want[:, None]) & (j < have[:, None])
    dest = torch.where(out, s["free_count"].long() + drop_at[:, None] + j - want[:, None], free.shape[0])
    longer = torch.cat([free, free[:1]])
    longer[dest.reshape(-1)] = table.reshape(-1)
    free.copy_(longer[:-1])
    # then each stream that grows takes its pages from the top
    inn = (j >= have[:, None]) & (j < want[:, None]) & ok[:, None]
    src = torch.where(inn, avail - 1 - grow_at[:, None] - (j - have[:, None]), 0)
    table.copy_(torch.where(inn, free[src], table))
    s["page_count_out"].copy_(torch.where((grow > 0) & ~ok, have, want))
    s["free_count_out"].copy_(avail - torch.where(ok, grow, 0).sum())
    st, t = _owners(start, total)
    at = kv[st] + t
    slot = table.long()[st, at // page] * page + at % page
    s["slots"].copy_(torch.where(ok[st], slot, -1))
    if s["parent"] is not None:
        t = _ancestors(start, s["parent"], total, MAX_ROWS)[st, t].sum(-1) - 1
    s["positions"].copy_(torch.where(ok[st], kv[st] + t, -1))


def _rotate(x, cos, sin, inter):
    r = 2 * cos.shape[-1]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if inter else (x[..., :r // 2], x[..., r // 2:r])
    p, q = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([p, q], -1).flatten(-2) if inter else torch.cat([p, q], -1)
    return torch.cat([y, x[..., r:]], -1)


def _plain_prep(s):
    c, m = s["c"], s["cache"]
    angle = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()

    def normed(x, w):
        x = x.float()
        return _rotate(x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w, cos, sin, c["inter"])

    s["q_out"].copy_(normed(s["q"], s["q_norm"]))
    page, off = s["slots"].long() // c["page"], s["slots"].long() % c["page"]
    for pool, scale, x in ((m["k"], m["k_scale"], normed(s["k"], s["k_norm"])), (m["v"], m["v_scale"], s["v"].float())):
        if c["e4m3"]:
            x, row = _quantise(x)
            scale[page, :, off] = row
            pool.view(torch.uint8)[page, :, off] = x.view(torch.uint8)
        else:
            pool[page, :, off] = x.to(torch.bfloat16)


def _gathered(pool, scale, table):
    """[n][hkv][blocks * page][d] in fp32: every stream's pages side by side."""
    t = table.long().clamp(min=0)
    x = pool.view(torch.uint8)[t].view(pool.dtype).float() if scale is not None else pool[t].float()
    if scale is not None:
        x = x * scale[t][..., None]
    n, b, h, p, d = x.shape
    return x.transpose(1, 2).reshape(n, h, b * p, d)


def _plain_attn(s):
    c, m = s["c"], s["cache"]
    n, R, hq, hkv, d = c["n"], c["rows"], c["hq"], c["hkv"], c["d"]
    total = s["q"].shape[0]
    K, V = (_gathered(m[x], m[x + "_scale"], s["block_table"]) for x in "kv")
    T = K.shape[2]
    st, t = _owners(s["row_start"], total)
    q = torch.zeros((n, R, hq, d), device=K.device)
    q[st, t] = s["q"].float()
    q = q.view(n, R, hkv, hq // hkv, d).transpose(1, 2).reshape(n, hkv, -1, d)
    score = (q @ K.transpose(-1, -2)) * (d ** -0.5)
    del K
    if s["parent"] is None:
        seen = torch.ones((R, R), dtype=torch.bool, device=q.device).tril()[None].expand(n, R, R)
    else:
        seen = _ancestors(s["row_start"], s["parent"], total, R)
    j = torch.arange(T, device=q.device)[None] - s["kv_len"].long()[:, None]      # place in the window, < 0 before it
    rows = (s["row_start"][1:] - s["row_start"][:-1]).long()
    inside = ((j >= 0) & (j < rows[:, None]))[:, None, :]
    mask = (j < 0)[:, None, :] | (inside & seen.gather(2, j.clamp(0, R - 1)[:, None, :].expand(n, R, T)))
    mask = mask[:, None, :, None, :].expand(n, hkv, R, hq // hkv, T).reshape(n, hkv, -1, T)
    score = score.masked_fill(~mask, -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-1e30))
    o = (p @ V) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.view(n, hkv, R, hq // hkv, d).transpose(1, 2).reshape(n, R, hq, d)[st, t]
    if s["gate"] is not None:
        o = o / (1.0 + torch.exp(-s["gate"].float()))
    s["out"].copy_(o)


def _plain_commit(s):
    c, m = s["c"], s["cache"]
    n, R, page, kv = c["n"], c["rows"], c["page"], s["kv_len"].long()
    start, total = s["row_start"].long(), s["parent"].shape[0]
    path = _ancestors(s["row_start"], s["parent"], total, R)[torch.arange(n, device=kv.device), s["accept"].long() - start[:-1]]
    length = path.sum(-1)
    order = torch.argsort((~path).to(torch.int8), dim=1, stable=True)              # the path's rows, root first
    k = torch.minimum(torch.arange(R, device=kv.device)[None], length[:, None] - 1)  # past its end: its last row again
    src, dst = kv[:, None] + order.gather(1, k), kv[:, None] + k
    table = s["block_table"].long()
    sp, dp = table.gather(1, src // page), table.gather(1, dst // page)
    for x in (m["k"], m["v"], m["k_scale"], m["v_scale"]):
        if x is not None:
            x = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
            x[dp, :, dst % page] = x[sp, :, src % page]
    s["kv_len_out"].copy_(kv + length)


# ---- the definitions, in 64 bits ---------------------------------------------------

def exact(case, seed):
    c = case
    if c["op"] in ("tables", "commit"):
        return None                     # whole numbers and copies
    s = prepare(c, seed)
    if c["op"] == "prep":
        return _exact_prep(s)
    return _exact_attn(s)


def _exact_prep(s):
    c = s["c"]
    R, half = c["rows"], c["rot"] // 2
    first = [2 * i if c["inter"] else i for i in range(half)]
    second = [2 * i + 1 if c["inter"] else half + i for i in range(half)]
    theta = torch.outer(s["positions"].to(torch.float64), s["inv_freq"].to(torch.float64))
    turn = torch.polar(torch.ones_like(theta), theta)[:, None, :]

    def of(x, w):
        x = x.to(torch.float64)
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / c["d"] + 1e-6) * w.to(torch.float64)
        z = torch.complex(x[:, :, first], x[:, :, second]) * turn
        x[:, :, first], x[:, :, second] = z.real.contiguous(), z.imag.contiguous()
        return x

    out = dict(q=of(s["q"], s["q_norm"]))
    slots = s["slots"].tolist()
    pages = torch.tensor([x // c["page"] for x in slots], device=DEV)
    offs = torch.tensor([x % c["page"] for x in slots], device=DEV)
    for name, x in (("k", of(s["k"], s["k_norm"])), ("v", s["v"].to(torch.float64))):
        pool, scale = s["cache"][name].to(torch.float64), s["cache"][name + "_scale"]
        if scale is not None:
            step = x.abs().amax(-1) / 448.0
            scale = scale.to(torch.float64)
            scale[pages, :, offs] = step
            x = x / step[:, :, None]
        pool[pages, :, offs] = x
        out[name], out[name + "_scale"] = pool, scale
    return out


def _exact_attn(s):
    c, m = s["c"], s["cache"]
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    start, lens = s["row_start"].tolist(), s["kv_len"].tolist()
    parent = None if s["parent"] is None else s["parent"].tolist()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    for i, ln in enumerate(lens):
        a, b = start[i], start[i + 1]
        keys = ln + b - a
        ids = s["block_table"][i, :-(-keys // page)].long()
        sees = torch.zeros((b - a, keys), dtype=torch.bool, device=DEV)
        for t in range(b - a):
            sees[t, :ln] = True
            u = t
            while u >= 0:
                sees[t, ln + u] = True
                u = u - 1 if parent is None else parent[a + u]
        for h in range(hkv):
            kv = []
            for name in "kv":
                x = m[name].view(torch.uint8)[ids, h].view(m[name].dtype) if c["e4m3"] else m[name][ids, h]
                x = x.to(torch.float64)
                if c["e4m3"]:
                    x = x * m[name + "_scale"][ids, h].to(torch.float64)[..., None]
                kv.append(x.reshape(-1, d)[:keys])
            for g in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                x = s["q"][a:b, g].to(torch.float64) @ kv[0].t() / math.sqrt(d)
                w = torch.softmax(x.masked_fill(~sees, -math.inf), dim=-1)
                out[a:b, g] = w @ kv[1]
    if s["gate"] is not None:
        out = out * torch.sigmoid(s["gate"].to(torch.float64))
    return out
