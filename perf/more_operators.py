"""Measured cases of attention over whole prompts and of the 4-bit key-value
cache: attention of packed prompts, fresh or resumed, over the paged cache
(``attn_prompt``); steps, windows and draft trees over a cache in MXFP4
(``attn_window``); rows quantised as they are written and read back
(``attn_prep`` and ``kv_read``); and cached rows read back by themselves.

``run`` computes them in elementary torch operations, or, where ``own`` is
true, through the framework's entry points.  ``exact`` computes the same from
the definitions in 64 bits.

Layouts: a cache is K and V of ``[pages][kv heads][page size][d]`` in bf16, in
e4m3 with one fp32 scale a row in ``[pages][kv heads][page size]``, or in MXFP4:
e2m1 codes, two a byte with the even channel in the low half, and for every 32
channels of a row an exponent byte e, so that a value is code * 2^(e - 127).
Stream s keeps its cache row i in page ``block_table[s][i // page size]``, row
``i % page size``; packed rows of stream s are ``row_start[s]`` up to
``row_start[s + 1]``, and row t of them is its cache row ``kv_len[s] + t``.
"""
import math

import torch

own = False

DEV = "cuda"
MAX_ROWS = 16            # rows of a verify window
LEAST, MOST = 25, 252    # exponent bytes that the quantiser writes
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _gdn():
    from verify_causal_conv1d_amd import gdn
    return gdn


# ---- cases ------------------------------------------------------------------

def _text(values):
    return " ".join(str(int(v)) for v in values)


def _spread(n, lo, hi):
    """n lengths over lo..hi, evenly by their logarithm, in a mixed order."""
    if n == 1:
        return [hi]
    r = [int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)]
    step = next(k for k in range(max(1, n // 3), n + 1) if math.gcd(k, n) == 1)
    return [r[(i * step) % n] for i in range(n)]


def _windows(n, m):
    """Rows of n windows, ragged up to m; the first has them all."""
    return [m if i == 0 else 1 + (7 * i + 3) % m for i in range(n)]


def listed():
    wide = dict(hq=24, hkv=4, d=256, page=64)
    return [
        # The prompt of one small request: latency.
        dict(name="prompt 100", op="prompt", rows="100", cached="0", hq=4, hkv=2, d=64, page=16, fmt="bf16", gate=False),
        # The packed prompt pass of the 27B-like layer: four fresh prompts on its gated attention heads.
        dict(name="prompts 8306", op="prompt", rows="512 1024 2048 4722", cached="0 0 0 0", fmt="bf16", gate=True, **wide),
        # A piece of a long prompt, resumed over an e4m3 cache, beside three short prompts that arrived with it.
        dict(name="prompt resumed e4m3", op="prompt", rows="1873 64 1 211", cached="30111 0 517 9000", hq=32, hkv=8, d=128, page=16,
             fmt="e4m3", gate=False),
        # The last rows of a long document (a question about it) over its 4-bit cache: few rows, a long axis.
        dict(name="prompt tail 128K mxfp4", op="prompt", rows="65", cached="131000", fmt="mxfp4", gate=True, **wide),
        # One small request's next token over a 4-bit cache.
        dict(name="step 1 mxfp4", op="window", rows="1", cached="100", hq=4, hkv=2, d=64, page=16, fmt="mxfp4", gate=False, tree=False),
        # Decode of 16 ragged streams on the 27B-like layer's heads.
        dict(name="step 16 mxfp4", op="window", rows=_text([1] * 16), cached=_text(_spread(16, 1000, 16384)), fmt="mxfp4", gate=True,
             tree=False, **wide),
        # One stream at the end of a 256K context: what a 4-bit cache is for.
        dict(name="step 256K mxfp4", op="window", rows="1", cached="262143", hq=24, hkv=4, d=256, page=256, fmt="mxfp4", gate=True,
             tree=False),
        # 16 ragged streams' draft trees of up to 16 rows, the verify round.
        dict(name="tree 16 mxfp4", op="window", rows=_text(_windows(16, 16)), cached=_text(_spread(16, 700, 8191)), fmt="mxfp4",
             gate=True, tree=True, **wide),
        # One stream's next token: norms, rotation, quantised into the cache, and that row back.
        dict(name="store 1", op="store", rows="1", cached="5000", hq=24, hkv=4, d=256, page=64, rot=64, inter=False),
        # The packed prompt pass of the 27B-like layer quantised into the cache, and read back.
        dict(name="store 8306", op="store", rows="512 1024 2048 4722", cached="0 0 0 0", hq=24, hkv=4, d=256, page=64, rot=64, inter=False),
        # A short cached prompt taken out of the pool.
        dict(name="read 100", op="read", rows="100", cached="0", hkv=2, d=64, page=16, fmt="mxfp4"),
        # 16 streams' cached prompts taken out of the pool, to be kept elsewhere; some from a shared prefix on.
        dict(name="read 16", op="read", rows=_text(_spread(16, 1000, 16384)), cached=_text([0, 512, 0, 77] * 4), hkv=4, d=256, page=64,
             fmt="mxfp4"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "window", "window", "store", "read"])
    page = rng.choice([16, 32, 64, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 6, 8])
    d = rng.choice([64, 128, 256])
    fmt = rng.choice(["bf16", "e4m3", "mxfp4"])
    gate = rng.random() < 0.5
    if op == "prompt":
        n = _log(rng, 1, 12)
        top = _log(rng, 1, 6000)
        rows = [_log(rng, 1, top) for _ in range(n)]
        past = _log(rng, 1, 30000)
        cached = [0 if rng.random() < 0.5 else _log(rng, 1, past) for _ in range(n)]
        if n > 2 and rng.random() < 0.3:
            rows[rng.randrange(n)] = 0
        if sum(rows) == 0:
            rows[0] = 1
        # the plain form pads to the longest: its scores and its keys stay under the listed cases'
        while n * hq * max(rows) * max(a + b for a, b in zip(rows, cached)) * max(1, d // 64) > 4 << 30:
            rows, cached = [-(-a // 2) for a in rows], [b // 2 for b in cached]
        return dict(op=op, rows=_text(rows), cached=_text(cached), hq=hq, hkv=hkv, d=d, page=page, fmt=fmt, gate=gate)
    if op == "window":
        n = _log(rng, 1, 64)
        m = rng.choice([1, 1, rng.randint(2, MAX_ROWS), MAX_ROWS])
        hi = _log(rng, 1, min(200000, (1 << 28) // (n * hkv * d), (24 << 20) * 2 // (n * m * hq)))
        return dict(op=op, rows=_text(_windows(n, m)), cached=_text(_spread(n, _log(rng, 1, hi), hi)), hq=hq, hkv=hkv, d=d, page=page,
                    fmt="mxfp4", gate=gate, tree=m > 1 and rng.random() < 0.5)
    n = _log(rng, 1, 16)
    if op == "store":
        top = _log(rng, 1, max(1, 8306 * 32 * 256 // ((hq + 2 * hkv) * d) // n))
        return dict(op=op, rows=_text(_log(rng, 1, top) for _ in range(n)), cached=_text(_log(rng, 1, 250000) // n for _ in range(n)), hq=hq,
                    hkv=hkv, d=d, page=page, rot=2 * rng.randint(1, d // 2), inter=rng.random() < 0.5)
    top = _log(rng, 1, (1 << 26) // (hkv * d) // n)
    return dict(op=op, rows=_text(_log(rng, 1, top) for _ in range(n)), cached=_text(rng.choice([0, _log(rng, 1, 1000)]) for _ in range(n)),
                hkv=hkv, d=d, page=page, fmt=fmt)


# ---- sizes that follow from a case alone --------------------------------------

def _ints(text):
    return [int(x) for x in text.split()]


def _row_bytes(fmt, d):
    return {"bf16": 2 * d, "e4m3": d + 4, "mxfp4": d // 2 + d // 32}[fmt]


def work(case):
    c = case
    rows, cached, d, hkv = _ints(c["rows"]), _ints(c["cached"]), c["d"], c["hkv"]
    total = sum(rows)
    if c["op"] == "read":
        return {"bytes": float(2 * total * hkv * (_row_bytes(c["fmt"], d) + 2 * d)), "flops": 0.0}
    hq = c["hq"]
    if c["op"] == "store":
        # q, k and v in, q out, the quantised rows out, then read, then in bf16
        per = 2 * d * (2 * hq + 2 * hkv) + 2 * hkv * (2 * _row_bytes("mxfp4", d) + 2 * d) + 8
        return {"bytes": float(total * per), "flops": float(total * (hq + hkv) * (4 * d + 3 * c["rot"]))}
    keys = sum(a + b for a, b in zip(rows, cached) if a)
    pairs = sum(m * ln + m * (m + 1) // 2 for m, ln in zip(rows, cached))
    return {"bytes": 2.0 * keys * hkv * _row_bytes(c["fmt"], d) + total * hq * d * 2.0 * (3 if c["gate"] else 2), "flops": 4.0 * hq * d * pairs}


# ---- inputs -------------------------------------------------------------------

def _int(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _starts(rows):
    s = [0]
    for m in rows:
        s.append(s[-1] + m)
    return s


def _parents(rows, host):
    """Draft trees: row 0 follows the cache, row t a row drawn from the four before it."""
    p = []
    for m in rows:
        for t in range(m):
            p.append(-1 if t == 0 else t - 1 - int(torch.randint(0, min(t, 4), (1,), generator=host)))
    return _int(p)


def _cache(c, fmt, pages, g):
    """K and V pools with values as the norm and the projection leave them."""
    shape = (pages, c["hkv"], c["page"], c["d"])
    got = {}
    for name in "kv":
        x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
        scale = None
        if fmt == "e4m3":
            scale = x.float().abs().amax(-1) / 448.0
            x = (x.float() / scale[..., None]).to(torch.float8_e4m3fn)
        elif fmt == "mxfp4":
            # the values above as their quantiser would leave them, made page by page to save memory
            y = torch.empty(shape[:3] + (c["d"] // 2,), dtype=torch.uint8, device=DEV)
            scale = torch.empty(shape[:3] + (c["d"] // 32,), dtype=torch.uint8, device=DEV)
            step = max(1, (1 << 26) // (c["hkv"] * c["page"] * c["d"]))
            for i in range(0, pages, step):
                y[i:i + step], scale[i:i + step] = _quantise(x[i:i + step].float())
            x = y
        got[name], got[name + "_scale"] = x, scale
    return got


def _paged(c, lens, g, spare=5):
    """A block table over shuffled pages with room for lens rows of every stream."""
    need = [-(-ln // c["page"]) for ln in lens]
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
    rows, cached = _ints(c["rows"]), _ints(c["cached"])
    total, d, hkv = sum(rows), c["d"], c["hkv"]
    lens = [a + b for a, b in zip(rows, cached)]
    table, pages = _paged(c, lens, g)
    s = dict(c=c, row_start=_int(_starts(rows)), kv_len=_int(cached), block_table=table, most=max(rows),
             cache=_cache(c, c.get("fmt", "mxfp4"), pages, g))
    if c["op"] in ("read", "store"):
        s["k_out"], s["v_out"] = (torch.zeros((total, hkv, d), dtype=torch.bfloat16, device=DEV) for _ in "kv")
    if c["op"] == "read":
        return s
    hq = c["hq"]
    if c["op"] == "store":
        # the projection's output: each query head beside its gate, then the keys, then the values
        x = torch.randn((total, (2 * hq + 2 * hkv) * d), generator=g, device=DEV, dtype=torch.bfloat16)
        s["q"] = x[:, :2 * hq * d].view(total, hq, 2 * d)[:, :, :d]
        s["k"] = x[:, 2 * hq * d:(2 * hq + hkv) * d].view(total, hkv, d)
        s["v"] = x[:, (2 * hq + hkv) * d:].view(total, hkv, d)
        w = 1.0 + 0.2 * torch.randn((2, d), generator=g, device=DEV)
        s["q_norm"], s["k_norm"] = w[0].contiguous(), w[1].contiguous()
        s["inv_freq"] = (1e7 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])).to(torch.float32).to(DEV)
        st, at = _places(s["row_start"], s["kv_len"], total)
        s["slots"] = (table.long()[st, at // c["page"]] * c["page"] + at % c["page"]).to(torch.int32)
        s["positions"] = at.to(torch.int32)
        s["q_out"] = torch.zeros((total, hq, d), dtype=torch.bfloat16, device=DEV)
        return s
    # queries a little larger than unit norm: softmax rows with a few leading keys
    s["q"] = (1.5 * torch.randn((total, hq, d), generator=g, device=DEV)).to(torch.bfloat16)
    s["gate"] = torch.randn((total, hq, 2 * d), generator=g, device=DEV, dtype=torch.bfloat16)[:, :, d:] if c["gate"] else None
    s["parent"] = _parents(rows, host) if c.get("tree") else None
    s["out"] = torch.zeros((total, hq, d), dtype=torch.bfloat16, device=DEV)
    s["max_kv"] = max(lens)
    if own:  # the memory for partial results that a program allocates once for its largest call
        if c["op"] == "prompt":
            b = _gdn().attn_prompt_workspace_bytes(hq, hkv, d, len(rows), total, s["max_kv"])
        else:
            b = _gdn().attn_workspace_bytes(hq, hkv, d, len(rows), total, s["most"], s["max_kv"])
        s["workspace"] = torch.empty(max(b, 16), dtype=torch.uint8, device=DEV)
    return s


# ---- one pass -------------------------------------------------------------------

def run(state):
    s = state
    return {"prompt": _prompt, "window": _window, "store": _store, "read": _read}[s["c"]["op"]](s)


def _prompt(s):
    m = s["cache"]
    if own:
        _gdn().attn_prompt(s["row_start"], s["kv_len"], s["block_table"], s["q"], m["k"], m["v"], s["out"], s["workspace"],
                           max_kv=s["max_kv"], gate=s["gate"], k_scale=m["k_scale"], v_scale=m["v_scale"])
    else:
        _plain_attention(s)
    return s["out"]


def _window(s):
    m = s["cache"]
    if own:
        _gdn().attn_window(s["row_start"], s["kv_len"], s["block_table"], s["q"], m["k"], m["v"], s["out"], s["workspace"],
                           max_kv=s["max_kv"], max_rows=s["most"], parent=s["parent"], gate=s["gate"],
                           k_scale=m["k_scale"], v_scale=m["v_scale"])
    else:
        _plain_attention(s)
    return s["out"]


def _store(s):
    c, m = s["c"], s["cache"]
    if own:
        _gdn().attn_prep(s["q"], s["k"], s["v"], s["q_norm"], s["k_norm"], s["inv_freq"], s["positions"], s["slots"],
                         s["q_out"], m["k"], m["v"], m["k_scale"], m["v_scale"], eps=1e-6, interleaved=c["inter"])
        _gdn().kv_read(s["row_start"], s["kv_len"], s["block_table"], m["k"], m["v"], s["k_out"], s["v_out"],
                       k_scale=m["k_scale"], v_scale=m["v_scale"])
    else:
        _plain_store(s)
        _plain_read(s)
    return dict(q=s["q_out"], k=s["k_out"], v=s["v_out"])


def _read(s):
    m = s["cache"]
    if own:
        _gdn().kv_read(s["row_start"], s["kv_len"], s["block_table"], m["k"], m["v"], s["k_out"], s["v_out"],
                       k_scale=m["k_scale"], v_scale=m["v_scale"])
    else:
        _plain_read(s)
    return dict(k=s["k_out"], v=s["v_out"])


# ---- the plain forms ---------------------------------------------------------------

def _owners(row_start, total):
    """Stream and place among its rows of each packed row."""
    r = torch.arange(total, device=row_start.device)
    s = torch.searchsorted(row_start[1:].long(), r, right=True)
    return s, r - row_start.long()[s]


def _places(row_start, first, total):
    """Stream and cache row of each packed row."""
    s, t = _owners(row_start, total)
    return s, first.long()[s] + t


def _quantise(y):
    """fp32 [..][d] in MXFP4: codes [..][d / 2] and exponent bytes [..][d / 32].
    A block's largest magnitude lands in [3.5, 7) steps of 2^(e - 127): a quarter
    of a power of two added to its bits carries from 1.75 on."""
    y = y.unflatten(-1, (-1, 32))
    top = y.abs().amax(-1)
    e = ((top.view(torch.int32) + (1 << 21)) >> 23) - 2
    e = e.clamp(LEAST, MOST)
    x = y * torch.exp2((127 - e).float())[..., None]
    a = x.abs()
    # to the nearest code, ties to the even one
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
            + 8 * (torch.signbit(x)).to(torch.uint8)).to(torch.uint8)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), e.to(torch.uint8)


def _values(x, scale):
    """What a pool's rows hold, in fp32."""
    if x.dtype == torch.uint8:
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=x.device)
        y = table[torch.stack([x & 15, x >> 4], -1).flatten(-2).int()]
        return (y.unflatten(-1, (-1, 32)) * torch.exp2(scale.float() - 127.0)[..., None]).flatten(-2)
    return x.float() if scale is None else x.float() * scale[..., None]


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


def _gathered(pool, scale, table):
    """[n][hkv][blocks * page][d] in fp32: every stream's pages side by side."""
    t = table.long().clamp(min=0)
    x = pool.view(torch.uint8)[t].view(pool.dtype) if pool.dtype == torch.float8_e4m3fn else pool[t]
    x = _values(x, None if scale is None else scale[t])
    n, b, h, p, d = x.shape
    return x.transpose(1, 2).reshape(n, h, b * p, d)


def _plain_attention(s):
    c, m = s["c"], s["cache"]
    n, R, hq, hkv, d = s["block_table"].shape[0], s["most"], c["hq"], c["hkv"], c["d"]
    G, total = hq // hkv, s["q"].shape[0]
    K = _gathered(m["k"], m["k_scale"], s["block_table"])
    T = K.shape[2]
    st, t = _owners(s["row_start"], total)
    q = torch.zeros((n, R, hq, d), device=K.device)
    q[st, t] = s["q"].float()
    q = q.view(n, R, hkv, G, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, G * R, d)
    score = (q @ K.transpose(-1, -2)).mul_(d ** -0.5).view(n, hkv, G, R, T)
    del K
    j = torch.arange(T, device=q.device)[None] - s["kv_len"].long()[:, None]      # place in the pass, < 0 before it
    if s["parent"] is None:
        hidden = j[:, None, :] > torch.arange(R, device=q.device)[None, :, None]
    else:
        rows = (s["row_start"][1:] - s["row_start"][:-1]).long()
        inside = ((j >= 0) & (j < rows[:, None]))[:, None, :]
        seen = _ancestors(s["row_start"], s["parent"], total, R)
        hidden = ~((j < 0)[:, None, :] | (inside & seen.gather(2, j.clamp(0, R - 1)[:, None, :].expand(n, R, T))))
    score.masked_fill_(hidden[:, None, None], -math.inf)
    score.sub_(score.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    norm = score.sum(-1, keepdim=True).clamp(min=1e-30)
    V = _gathered(m["v"], m["v_scale"], s["block_table"])
    o = (score.view(n, hkv, G * R, T) @ V).view(n, hkv, G, R, d) / norm
    del score, V
    o = o.permute(0, 3, 1, 2, 4).reshape(n, R, hq, d)[st, t]
    if s["gate"] is not None:
        o = o / (1.0 + torch.exp(-s["gate"].float()))
    s["out"].copy_(o)


def _rotate(x, cos, sin, inter):
    r = 2 * cos.shape[-1]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if inter else (x[..., :r // 2], x[..., r // 2:r])
    p, q = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([p, q], -1).flatten(-2) if inter else torch.cat([p, q], -1)
    return torch.cat([y, x[..., r:]], -1)


def _plain_store(s):
    c, m = s["c"], s["cache"]
    angle = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    cos, sin = angle.cos(), angle.sin()

    def normed(x, w, cos, sin):
        return _rotate(x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w, cos, sin, c["inter"])

    s["q_out"].copy_(normed(s["q"].float(), s["q_norm"], cos.float(), sin.float()))
    # keys in 64 bits up to the one rounding before the quantiser: a value next to
    # the border of two codes decides which of them is stored
    key = normed(s["k"].double(), s["k_norm"].double(), cos, sin).float()
    page, off = s["slots"].long() // c["page"], s["slots"].long() % c["page"]
    for name, y in (("k", key), ("v", s["v"].float())):
        m[name][page, :, off], m[name + "_scale"][page, :, off] = _quantise(y)


def _plain_read(s):
    c, m, table = s["c"], s["cache"], s["block_table"].long()
    st, at = _places(s["row_start"], s["kv_len"], s["k_out"].shape[0])
    page, off = table[st, at // c["page"]], at % c["page"]
    for name in "kv":
        x, scale = m[name], m[name + "_scale"]
        x = x.view(torch.uint8)[page, :, off].view(x.dtype) if x.dtype == torch.float8_e4m3fn else x[page, :, off]
        s[name + "_out"].copy_(_values(x, None if scale is None else scale[page, :, off]))


# ---- the definitions, in 64 bits ---------------------------------------------------

def _decoded(x, scale):
    """A pool's rows by the formats' bits, in fp64."""
    if scale is None:
        return x.to(torch.float64)
    if x.dtype == torch.float8_e4m3fn:
        return x.to(torch.float64) * scale.to(torch.float64).unsqueeze(-1)
    y = torch.empty(x.shape[:-1] + (2 * x.shape[-1],), dtype=torch.float64, device=x.device)
    for half in (0, 1):
        c = (x >> (4 * half)).to(torch.int64) & 15
        exponent, mantissa = (c >> 1) & 3, (c & 1).to(torch.float64)
        size = torch.where(exponent == 0, 0.5 * mantissa, torch.ldexp(1.0 + 0.5 * mantissa, exponent - 1))
        y[..., half::2] = torch.where(c >= 8, -size, size)
    return torch.ldexp(y, scale.to(torch.int64).repeat_interleave(32, dim=-1) - 127)


def _rows_of(s, name, i, ln, h=None):
    """Cache rows 0 .. ln - 1 of stream i, of kv head h or of all: [hkv][ln][d]."""
    page = s["c"]["page"]
    ids = s["block_table"][i, :-(-ln // page)].long()
    x, scale = s["cache"][name], s["cache"][name + "_scale"]
    x = x.view(torch.uint8)[ids].view(x.dtype) if x.dtype == torch.float8_e4m3fn else x[ids]
    scale = None if scale is None else scale[ids]
    if h is not None:
        x, scale = x[:, h:h + 1], None if scale is None else scale[:, h:h + 1]
    y = _decoded(x, scale)
    return y.transpose(0, 1).reshape(y.shape[1], -1, s["c"]["d"])[:, :ln]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("prompt", "window"):
        return _exact_attention(s)
    if case["op"] == "store":
        return _exact_store(s)
    start, first = s["row_start"].tolist(), s["kv_len"].tolist()
    return {name: torch.cat([_rows_of(s, name, i, f + b - a)[:, f:].transpose(0, 1)
                             for i, (a, b, f) in enumerate(zip(start, start[1:], first))]) for name in "kv"}


def _exact_attention(s):
    c = s["c"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    start, lens = s["row_start"].tolist(), s["kv_len"].tolist()
    parent = None if s["parent"] is None else s["parent"].tolist()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    for i, ln in enumerate(lens):
        a, b = start[i], start[i + 1]
        keys = ln + b - a
        if a == b:
            continue
        if parent is None:
            sees = torch.arange(keys, device=DEV) <= ln + torch.arange(b - a, device=DEV).unsqueeze(1)
        else:
            sees = torch.zeros((b - a, keys), dtype=torch.bool, device=DEV)
            sees[:, :ln] = True
            for t in range(b - a):
                u = t
                while u >= 0:
                    sees[t, ln + u] = True
                    u = parent[a + u]
        for h in range(hkv):
            key, value = _rows_of(s, "k", i, keys, h)[0], _rows_of(s, "v", i, keys, h)[0]
            for g in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                x = s["q"][a:b, g].to(torch.float64) @ key.t() / math.sqrt(d)
                out[a:b, g] = torch.softmax(x.masked_fill_(~sees, -math.inf), dim=-1) @ value
    if s["gate"] is not None:
        out *= torch.sigmoid(s["gate"].to(torch.float64))
    return out


def _exact_store(s):
    c = s["c"]
    half = c["rot"] // 2
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

    def stored(x):
        """x, rounded to fp32, as the 4-bit rows stand for it: block by block, to
        the nearest multiple of the step that its magnitude has (ties to even)."""
        x = x.to(torch.float32).to(torch.float64).unflatten(-1, (-1, 32))
        m, e = torch.frexp(x.abs().amax(-1, keepdim=True))           # m in [0.5, 1)
        e = torch.where(m >= 0.875, e - 2, e - 3).clamp(LEAST - 127, MOST - 127)
        y = torch.ldexp(x, -e)
        step = torch.where(y.abs() < 2.0, 0.5, torch.where(y.abs() < 4.0, 1.0, 2.0))
        y = (torch.round(y / step) * step).clamp(-6.0, 6.0)
        return torch.ldexp(y, e).flatten(-2)

    return dict(q=of(s["q"], s["q_norm"]), k=stored(of(s["k"], s["k_norm"])), v=stored(s["v"].to(torch.float64)))
