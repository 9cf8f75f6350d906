"""Attention of whole prompts over bf16, e4m3 and 4-bit caches against the fp64
oracle: packed, resumed, cut along the keys, with rows that must not be seen,
broken layouts, captured rounds."""
import numpy as np
import pytest
import torch

from oracle import attn as ref
from verify_causal_conv1d_amd import gdn
from verify_causal_conv1d_amd import inputs as gi

from gpu_util import announce

pytestmark = pytest.mark.gpu

BF16, I32, F8, U8 = torch.bfloat16, torch.int32, torch.float8_e4m3fn, torch.uint8
FMTS = ("bf16", "e4m3", "mxfp4")


def i32(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def f64(t):
    return t.detach().cpu().double().numpy()


def cu(t):
    return None if t is None else t.cuda()


def made(x, fmt):
    """A pool's rows from fp32 values: (rows, scales)."""
    if fmt == "bf16":
        return x.to(BF16), None
    if fmt == "e4m3":
        s = x.abs().amax(-1) / 448.0
        return (x / s[..., None]).to(F8), s
    codes, exps = ref.mx_quantise(x.numpy())
    return torch.from_numpy(codes), torch.from_numpy(exps)


def values(pool, scale):
    """The values that a pool holds, in fp64."""
    if pool.dtype == U8:
        return ref.mx_values(pool.cpu().numpy(), scale.cpu().numpy())
    x = pool.cpu().float().double()
    return (x if scale is None else x * scale.cpu().double()[..., None]).numpy()


class Case:
    """Streams over a paged cache: every row that no stream holds is NaN."""

    def __init__(self, lens, rows, hq, hkv, d, page, fmt="bf16", gate=False, seed=0, amp=1.5, spare=3, gap=0, v_amp=1.0):
        g = self.g = torch.Generator().manual_seed(seed)
        self.lens, self.rows, self.hq, self.hkv, self.d, self.page, self.fmt = lens, rows, hq, hkv, d, page, fmt
        self.row_start = gi.starts_from_lengths(rows) + gap
        self.total = int(self.row_start[-1]) + gap
        need = [-(-(a + b) // page) for a, b in zip(lens, rows)]
        self.pages = sum(need) + spare
        perm = torch.randperm(self.pages, generator=g).to(I32)
        self.table = torch.full((len(lens), max(need) + 1), -1, dtype=I32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = perm[at:at + n]
            at += n
        held = torch.zeros((self.pages, 1, page), dtype=torch.bool)
        for s, n in enumerate(need):
            for j in range(n):
                held[self.table[s, j], 0, :max(0, min(page, lens[s] + rows[s] - j * page))] = True
        held = held.expand(self.pages, hkv, page)
        for name in "kv":
            x, sc = made(torch.randn((self.pages, hkv, page, d), generator=g) * (v_amp if name == "v" else 1.0), fmt)
            if fmt == "bf16":
                x[~held] = float("nan")
            elif fmt == "e4m3":
                x.view(U8)[~held] = 0x7F
                sc[~held] = float("nan")
            else:
                sc[~held] = 255
            setattr(self, name, x)
            setattr(self, name + "s", sc)
        self.q = (torch.randn((self.total, hq, d), generator=g) * amp).to(BF16)
        self.gate = (torch.randn((self.total, hq, 2 * d), generator=g) * 2).to(BF16) if gate else None
        self.kv_len = torch.tensor(lens, dtype=I32)

    def run(self, max_kv=None, out=None, table=None, row_start=None, kv_len=None, scale=None):
        max_kv = max_kv or max(a + b for a, b in zip(self.lens, self.rows))
        out = torch.full((self.total, self.hq, self.d), float("nan"), dtype=BF16, device="cuda") if out is None else out
        size = gdn.attn_prompt_workspace_bytes(self.hq, self.hkv, self.d, len(self.lens), self.total, max_kv)
        ws = torch.full((size,), 0xFF, dtype=U8, device="cuda")
        gate = self.gate.cuda()[:, :, self.d:] if self.gate is not None else None
        pick = lambda a, b: (b if a is None else a).cuda()  # noqa: E731
        gdn.attn_prompt(pick(row_start, self.row_start), pick(kv_len, self.kv_len), pick(table, self.table), self.q.cuda(), cu(self.k),
                        cu(self.v), out, ws, max_kv=max_kv, gate=gate, k_scale=cu(self.ks), v_scale=cu(self.vs), scale=scale)
        torch.cuda.synchronize()
        return out

    def oracle(self, scale=None):
        gate = None if self.gate is None else f64(self.gate[:, :, self.d:])
        rows = self.row_start.tolist()
        with np.errstate(invalid="ignore"):
            out, mag, reach = ref.prompt(self.page, rows, self.lens, self.table.numpy(), f64(self.q), values(self.k, self.ks),
                                         values(self.v, self.vs), ref.default_scale(self.d) if scale is None else scale, gate)
        return out, ref.window_bound(out, mag, reach, self.d) + self.underflow()

    def underflow(self):
        """What weights below fp32's (and bf16's) least normal number can add up to.  A
        column's base lies at most 2^8 above its maximum, so the sum of its weights is
        2^-8 at least, and a weight that comes out as 0 is less than 2^-126: 2^-118 of
        its value for each key.  It shows where larger weights meet values that are
        exactly 0, as 4-bit values often are."""
        top = float(np.nanmax(np.abs(values(self.v, self.vs))))
        return 2.0 ** -118 * (max(self.lens) + max(self.rows)) * top

    def inside(self):
        return slice(int(self.row_start[0]), int(self.row_start[-1]))


def close(got, want, bound, what=""):
    got = f64(got)
    assert np.all(np.isfinite(got)), what
    worst = float(np.max(np.abs(got - want) / bound)) if got.size else 0.0
    print(f"{what} worst error {worst:.3f} of its bound")
    assert worst <= 1.0, (what, worst)


PROMPTS = [
    # one row and one key; lengths around the tiles of 32 and 64 keys, streams without rows
    dict(lens=[0], rows=[1], hq=1, hkv=1, d=64, page=16),
    dict(lens=[0] * 10, rows=[1, 0, 15, 16, 17, 31, 32, 33, 64, 65], hq=4, hkv=2, d=64, page=16),
    dict(lens=[1, 0, 63, 64, 65, 127, 128, 200], rows=[1, 0, 15, 63, 64, 65, 2, 130], hq=4, hkv=2, d=128, page=32, gate=True),
    dict(lens=[14, 30, 62, 126, 127, 0, 129, 255], rows=[2, 3, 40, 3, 100, 77, 16, 1], hq=6, hkv=1, d=256, page=16, gate=True),
    # (row, head) pairs around a workgroup's 256: 6 heads a group, then groups that cut rows, then more than a tile
    dict(lens=[0, 5, 9, 130], rows=[42, 43, 85, 86], hq=24, hkv=4, d=256, page=64, gate=True),
    dict(lens=[70, 0], rows=[13, 33], hq=40, hkv=1, d=64, page=128),
    dict(lens=[20, 100], rows=[9, 5], hq=300, hkv=1, d=128, page=256),
    dict(lens=[33, 0], rows=[3, 40], hq=1024, hkv=1, d=64, page=16),
    dict(lens=[17], rows=[70], hq=256, hkv=256, d=64, page=16, spare=1),
    dict(lens=[0, 300, 40], rows=[300, 129, 1], hq=3, hkv=3, d=128, page=16, gap=5),
    dict(lens=[1000, 0], rows=[257, 700], hq=2, hkv=2, d=256, page=64),
    # mostly cached rows, in one chunk
    dict(lens=[300, 17, 399, 0], rows=[100, 3, 1, 0], hq=6, hkv=1, d=256, page=32, gate=True),
    dict(lens=[350, 200], rows=[60, 90], hq=12, hkv=2, d=256, page=128),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("i", range(len(PROMPTS)))
def test_prompts_match_oracle(i, fmt):
    kw = PROMPTS[i]
    announce(f"prompts {kw} {fmt}")
    c = Case(fmt=fmt, seed=40 + i, **kw)
    out, (want, bound) = c.run(), c.oracle()
    a = c.inside()
    close(out[a], want[a], bound[a])
    assert torch.isnan(out[:a.start]).all() and torch.isnan(out[a.stop:]).all()      # rows of no stream


@pytest.mark.parametrize("lens,rows,hq,hkv,d,page", [
    ([1200], [65], 6, 1, 256, 64),                      # two chunks, none of them at the rows' border
    ([4090, 3], [70, 5], 4, 2, 64, 16),                 # 8 chunks beside a stream that needs one
    ([9000, 0, 2000, 511], [1, 600, 3, 1], 2, 1, 128, 32),      # a fresh prompt whose first rows see one chunk
    ([33000], [17], 12, 2, 128, 256),
    ([40000, 17], [300, 2], 1, 1, 64, 128),
    ([0], [1500], 1, 1, 256, 64),                       # a single prompt of few pairs
])
@pytest.mark.parametrize("fmt", FMTS)
def test_calls_cut_along_the_keys(lens, rows, hq, hkv, d, page, fmt):
    announce(f"prompts cut along the keys: {lens} {rows} {hq}/{hkv} d {d} {fmt}")
    c = Case(lens, rows, hq, hkv, d, page, fmt=fmt, seed=7, gate=len(lens) > 1)
    assert gdn.attn_prompt_workspace_bytes(hq, hkv, d, len(lens), c.total, max(a + b for a, b in zip(lens, rows))) > 0
    close(c.run(), *c.oracle())


@pytest.mark.parametrize("fmt", FMTS)
def test_parts_of_many_bytes(fmt):
    """As above, with parts of more than 16 MB, which the join asks for once it knows the stream."""
    announce(f"prompts with many parts, {fmt}")
    c = Case([12000, 30, 2500, 0], [250, 20, 130, 9], 16, 1, 128, 64, fmt=fmt, seed=8, gate=True)
    close(c.run(), *c.oracle())


def test_peaked_scores_and_scales():
    for d, fmt in ((64, "bf16"), (256, "mxfp4"), (128, "e4m3")):
        announce(f"prompts, peaked rows, given scales, d {d} {fmt}")
        c = Case([200, 0], [60, 90], 4, 2, d, 32, fmt=fmt, seed=13, amp=30.0)
        close(c.run(), *c.oracle())
        for scale in (0.0, -0.02, 0.3):
            close(c.run(scale=scale), *c.oracle(scale=scale))


@pytest.mark.parametrize("fmt", FMTS)
def test_scores_that_rise_and_fall(fmt):
    """Each column's base has to move at every stage of keys, or never again after the first."""
    for d, rising in ((64, True), (128, True), (256, True), (256, False)):
        announce(f"scores that {'rise' if rising else 'fall'} along the keys, {fmt}, d {d}")
        c = Case([700], [90], 4, 2, d, 64, fmt=fmt, seed=16)
        x = 0.1 * torch.randn((c.pages, 2, 64, d), generator=c.g)
        for j in range(-(-790 // 64)):
            at = torch.arange(64 * j, 64 * j + 64) / 790.0
            x[c.table[0, j]] += 8.0 * (at if rising else 1 - at)[None, :, None]
        c.k, c.ks = made(x, fmt)
        c.q = c.q.abs()
        close(c.run(), *c.oracle())
        close(c.run(scale=-0.05), *c.oracle(scale=-0.05))


def test_values_near_the_types_largest():
    """Sums of weighted values overflow no sooner than the result does."""
    announce("prompts, values near the largest")
    c = Case([100], [60], 2, 1, 128, 16, seed=14)
    c.v = torch.where(torch.isnan(c.v), c.v, torch.full_like(c.v, 3.0e38))
    got = c.run().float()
    assert ((got / 3.0e38 - 1).abs() <= 2.0 ** -6).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_that_are_not_seen_change_nothing(fmt):
    """Infinities and NaN in K, in V and in scales reach the rows that see them and no others, bit for bit."""
    for d, lens, rows in ((64, [70, 0], [50, 90]), (256, [1300, 3], [45, 9])):       # the second pair is cut along the keys
        announce(f"unseen rows, {fmt}, d {d}, {lens}")
        c = Case(lens, rows, 6, 2, d, 16, fmt=fmt, seed=15)
        clean = c.run()
        for st, bad in ((0, 7), (0, rows[0] - 1), (1, 0), (1, 8)):
            at = lens[st] + bad
            page, off = int(c.table[st, at // 16]), at % 16
            tries = [(c.k, float("nan")), (c.v, float("nan"))]
            if fmt == "bf16":
                tries += [(c.v, float("inf")), (c.k, float("-inf")), (c.v, float("-inf"))]
            if fmt == "mxfp4":
                tries = [(c.ks, 255), (c.vs, 255), (c.vs, 253)]
            if fmt == "e4m3":
                tries += [(c.ks, float("nan")), (c.vs, float("nan")), (c.vs, float("inf"))]
            for pool, value in tries:
                keep = pool[page, :, off].clone()
                pool[page, :, off] = torch.full(keep.shape, value).to(pool.dtype)
                got = c.run()
                pool[page, :, off] = keep
                a = int(c.row_start[st]) + bad
                hit = torch.zeros(c.total, dtype=torch.bool)
                hit[a:int(c.row_start[st + 1])] = True
                assert torch.equal(got[~hit], clean[~hit]), (st, bad, value)
                if pool is c.v and abs(value) == float("inf"):
                    assert (got[hit].float() == value).all(), (st, bad, value)
                elif value != value or fmt == "mxfp4":
                    assert torch.isnan(got[hit]).all(), (st, bad, value)
                else:
                    assert not torch.isfinite(got[hit]).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_cached_rows_that_are_not_finite_reach_all_rows(fmt):
    c = Case([70, 333], [40, 9], 6, 2, 128, 16, fmt=fmt, seed=30)
    clean = c.run()
    announce(f"cached rows that are not finite, {fmt}")
    for s, key in ((0, 69), (0, 64), (0, 63), (0, 0), (1, 332), (1, 320), (1, 319)):
        page, off = int(c.table[s, key // 16]), key % 16
        pool, value = (c.vs, 255) if fmt == "mxfp4" else (c.v, float("nan"))
        keep = pool[page, :, off].clone()
        pool[page, :, off] = torch.full(keep.shape, value).to(pool.dtype)
        got = c.run()
        pool[page, :, off] = keep
        a, b = int(c.row_start[s]), int(c.row_start[s + 1])
        hit = torch.zeros(c.total, dtype=torch.bool)
        hit[a:b] = True
        assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], clean[~hit]), (s, key)


@pytest.mark.parametrize("fmt", FMTS)
def test_streams_do_not_depend_on_each_other(fmt):
    """With the same total_rows and max_kv a stream's bits are its own, wherever it is packed and whatever lies beside it."""
    for lens, rows in (([300, 0, 77], [50, 200, 3]), ([5000, 3, 900], [20, 9, 1])):
        announce(f"prompts in another order, {fmt}, {lens}")
        c = Case(lens, rows, 4, 2, 128, 32, fmt=fmt, seed=16)
        want = c.run()
        order = [2, 0, 1]
        rs = gi.starts_from_lengths([rows[s] for s in order])
        one = Case.__new__(Case)
        one.__dict__.update(c.__dict__)
        at = [slice(int(c.row_start[s]), int(c.row_start[s + 1])) for s in order]
        one.q = torch.cat([c.q[a] for a in at])
        one.row_start, one.kv_len, one.table = rs, c.kv_len[order], c.table[order].contiguous()
        assert torch.equal(one.run(), torch.cat([want[a] for a in at]))
        # the others skipped: their lengths are out of range
        for s in range(3):
            kv = c.kv_len.clone()
            kv[[x for x in range(3) if x != s]] = -1
            got = c.run(kv_len=kv)
            a = slice(int(c.row_start[s]), int(c.row_start[s + 1]))
            assert torch.equal(got[a], want[a])
            assert torch.isnan(got).sum() == want.numel() - want[a].numel()


@pytest.mark.parametrize("lens,rows", [([300, 70, 900, 40], [60, 100, 4, 4]), ([3000, 70, 2900, 40], [6, 10, 4, 4])])
def test_broken_streams_are_skipped(lens, rows):
    c = Case(lens, rows, 4, 2, 128, 16, seed=17)
    good = c.run()
    announce(f"skipped streams {lens}")

    def same_but(got, streams):
        for s in range(4):
            a, b = int(c.row_start[s]), int(c.row_start[s + 1])
            if s in streams:
                assert torch.isnan(got[a:b]).all(), s
            else:
                assert torch.equal(got[a:b], good[a:b]), s
    last = [(a + b - 1) // 16 for a, b in zip(lens, rows)]
    for s, j in ((0, 3), (0, last[0]), (1, 0), (2, last[2]), (3, last[3])):
        for page in (-1, c.pages, 1 << 30):
            t = c.table.clone()
            t[s, j] = page
            same_but(c.run(table=t), {s})
    for value in (-1, 10 ** 6, 2 ** 31 - 1):
        kv = c.kv_len.clone()
        kv[1] = value
        same_but(c.run(kv_len=kv), {1})
    top = max(a + b for a, b in zip(lens, rows))
    for value in (-5, c.total + 1, 2 ** 31 - 1):
        rs = c.row_start.clone()
        rs[4] = value
        same_but(c.run(row_start=rs, max_kv=top), {3})
        rs = c.row_start.clone()
        rs[2] = value
        same_but(c.run(row_start=rs, max_kv=top), {1, 2})
    # a bound that a stream passes
    short = sorted(a + b for a, b in zip(lens, rows))[2]
    got = c.run(max_kv=short)
    longest = max(range(4), key=lambda s: lens[s] + rows[s])
    for s in range(4):
        a = slice(int(c.row_start[s]), int(c.row_start[s + 1]))
        assert torch.isnan(got[a]).all() if s == longest else torch.isfinite(got[a]).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows", [[300, 50, 150], [300, 0, 150]])
def test_finished_streams_of_any_length(rows, fmt):
    """A kv_len below 0 marks a finished stream, with rows or without, down to the type's
    lowest value: the streams beside it keep their bits.  (Not cut along the keys, so that
    tiles go by length over all streams.)"""
    announce(f"finished prompts {rows} {fmt}")
    c = Case([0, 30, 20], rows, 6, 2, 64, 16, fmt=fmt, seed=40)
    good = c.run()
    a, b = int(c.row_start[1]), int(c.row_start[2])
    for value in (-1, -1000, -2 ** 30, -2 ** 31 + 470, -2 ** 31 + 5, -2 ** 31):
        kv = c.kv_len.clone()
        kv[1] = value
        got = c.run(kv_len=kv)
        assert torch.equal(got[:a], good[:a]) and torch.equal(got[b:], good[b:]), value
        assert torch.isnan(got[a:b]).all(), value


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("scale", [0.0, 0.1, -0.1])
def test_queries_that_are_not_finite(fmt, scale):
    """They make their row and head NaN under any scale, 0 too (0 * infinity), and no other."""
    announce(f"queries that are not finite, {fmt}, scale {scale}")
    for d in (64, 128, 256):
        c = Case([70, 1300], [5, 9], 6, 2, d, 16, fmt=fmt, seed=42)
        clean = c.run(scale=scale)
        close(clean, *c.oracle(scale=scale))
        for value in (float("nan"), float("inf"), float("-inf")):
            keep = c.q.clone()
            c.q[1, 3, 5] = c.q[7, 0, d - 1] = value
            got = c.run(scale=scale)
            c.q = keep
            hit = torch.zeros((c.total, 6), dtype=torch.bool)
            hit[1, 3] = hit[7, 0] = True
            assert torch.equal(got[~hit], clean[~hit]), (d, value)
            if scale == 0.0 or value != value:
                assert torch.isnan(got[hit]).all(), (d, value)
            else:
                assert not torch.isfinite(got[hit]).any(), (d, value)


def test_many_streams():
    """More streams than a wave looks at together, among them some without rows."""
    g = torch.Generator().manual_seed(25)
    for n, fmt in ((70, "bf16"), (200, "mxfp4"), (130, "e4m3")):
        lens = torch.randint(0, 300, (n,), generator=g).tolist()
        rows = [0 if i % 7 == 3 else 1 + (i * i) % 40 for i in range(n)]
        announce(f"prompts of {n} streams {fmt}")
        c = Case(lens, rows, 4, 2, 64, 32, fmt=fmt, seed=26)
        close(c.run(), *c.oracle())


def test_longest_bound():
    """The largest max_kv: a call that is not cut by it gives the same bits, one that is stays within the bound."""
    announce("prompts under the largest max_kv")
    c = Case([600, 70], [30, 40], 8, 2, 256, 64, seed=27)
    close(c.run(max_kv=1 << 21), *c.oracle())
    c = Case([60, 7], [2800, 400], 24, 4, 64, 64, seed=28)
    many = c.run(max_kv=1 << 21)
    assert torch.isfinite(many).all()
    close(c.run()[:50], *(x[:50] for x in _some(c, 50)))


@pytest.mark.parametrize("fmt", FMTS)
def test_loose_bounds(fmt):
    """Under bounds far above all lengths every stream has one chunk: every row within the oracle's bound, and the same bits under another such bound."""
    for d, lens, rows, hq, hkv in ((64, [60, 7], [1400, 200], 8, 2), (256, [600, 70, 0], [30, 40, 500], 8, 2), (128, [900], [300], 6, 1),
                                   (256, [3000], [65], 6, 1)):
        announce(f"prompts under loose bounds, {fmt}, d {d}, {lens} {rows}")
        c = Case(lens, rows, hq, hkv, d, 64, fmt=fmt, seed=43, gate=d == 128)
        want, bound = c.oracle()
        loose = c.run(max_kv=1 << 21)
        close(loose, want, bound)
        assert torch.equal(loose, c.run(max_kv=1 << 20))
        close(c.run(), want, bound)


def _some(c, rows):
    """The oracle of a case's first rows."""
    one = Case.__new__(Case)
    one.__dict__.update(c.__dict__)
    one.row_start, one.lens, one.q = torch.tensor([0, rows], dtype=I32), c.lens[:1], c.q[:rows]
    return one.oracle()


def test_pieces_of_a_prompt():
    """A prompt in pieces over what the earlier ones stored, against the whole prompt's oracle."""
    for fmt in FMTS:
        announce(f"a prompt in pieces {fmt}")
        c = Case([0], [400], 6, 2, 128, 32, fmt=fmt, seed=18)
        want, bound = c.oracle()
        for a, b in ((0, 1), (1, 130), (130, 399), (399, 400)):
            one = Case.__new__(Case)
            one.__dict__.update(c.__dict__)
            one.lens, one.rows, one.q, one.total = [a], [b - a], c.q[a:b].contiguous(), b - a
            one.kv_len, one.row_start = torch.tensor([a], dtype=I32), torch.tensor([0, b - a], dtype=I32)
            close(one.run(), want[a:b], bound[a:b])


def test_streams_that_share_pages():
    announce("prompts over shared pages")
    c = Case([640, 700], [30, 9], 6, 2, 128, 64, seed=33)
    for j in range(10):
        for pool in (c.k, c.v):
            pool[c.table[1, j]] = pool[c.table[0, j]]
    want = c.run()
    table = c.table.clone()
    table[1, :10] = table[0, :10]
    assert torch.equal(c.run(table=table), want)


@pytest.mark.parametrize("fmt", FMTS)
def test_offsets_past_32_bits(fmt):
    """Pools of more than 4 GiB, the streams' pages at the far end; and back into packed rows."""
    announce(f"prompts, 5 GiB pools, {fmt}")
    c = Case([130, 700], [3, 40], 4, 2, 256, 64, fmt=fmt, seed=17)
    row = {"bf16": 512, "e4m3": 256, "mxfp4": 128}[fmt]
    pages = (5 << 30) // (2 * 64 * row)
    first = pages - c.pages
    want = c.run()
    big = []
    for pool, scale in ((c.k, c.ks), (c.v, c.vs)):
        p = torch.empty((pages,) + tuple(pool.shape[1:]), dtype=pool.dtype, device="cuda")
        s = None if scale is None else torch.empty((pages,) + tuple(scale.shape[1:]), dtype=scale.dtype, device="cuda")
        p[first:] = pool.cuda()
        if s is not None:
            s[first:] = scale.cuda()
        big.append((p, s))
    table = torch.where(c.table >= 0, c.table + first, c.table).cuda()
    out = torch.zeros_like(want)
    ws = torch.empty(gdn.attn_prompt_workspace_bytes(4, 2, 256, 2, 43, 740), dtype=U8, device="cuda")
    (k, ks), (v, vs) = big
    gdn.attn_prompt(c.row_start.cuda(), c.kv_len.cuda(), table, c.q.cuda(), k, v, out, ws, max_kv=740, k_scale=ks, v_scale=vs)
    assert torch.equal(out, want)
    ko, vo = (torch.zeros((43, 2, 256), dtype=BF16, device="cuda") for _ in "kv")
    gdn.kv_read(c.row_start.cuda(), c.kv_len.cuda(), table, k, v, ko, vo, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    for got, pool, scale in ((ko, c.k, c.ks), (vo, c.v, c.vs)):
        exact = ref.read(64, c.row_start.tolist(), c.lens, c.table.numpy(), values(pool, scale), np.zeros((43, 2, 256)))
        assert np.all(np.abs(f64(got) - exact) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(exact) * (fmt == "e4m3"))


def test_on_another_stream_and_two_at_once():
    """Two calls in flight on two streams, each with its own workspace, give what they give alone."""
    announce("prompts on two streams")
    cases = [Case([5000], [40], 4, 2, 128, 64, seed=41), Case([3000, 9], [20, 100], 4, 2, 256, 32, fmt="mxfp4", seed=42)]
    want = [c.run() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    args = []
    for c in cases:
        top = max(a + b for a, b in zip(c.lens, c.rows))
        args.append(dict(row_start=c.row_start.cuda(), kv_len=c.kv_len.cuda(), block_table=c.table.cuda(), q=c.q.cuda(), k_cache=cu(c.k),
                         v_cache=cu(c.v), out=torch.zeros((c.total, c.hq, c.d), dtype=BF16, device="cuda"), max_kv=top, k_scale=cu(c.ks),
                         v_scale=cu(c.vs), workspace=torch.empty(gdn.attn_prompt_workspace_bytes(c.hq, c.hkv, c.d, 2, c.total, top),
                                                                 dtype=U8, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(3):
        for s, a in zip(streams, args):
            a["out"].zero_()
        torch.cuda.synchronize()
        for s, a in zip(streams, args):
            with torch.cuda.stream(s):
                gdn.attn_prompt(**a)
        torch.cuda.synchronize()
        for a, w in zip(args, want):
            assert torch.equal(a["out"], w)


@pytest.mark.parametrize("fmt", FMTS)
def test_captured_round_of_prompts(fmt):
    """Tables, prep, attention and read of a prompt pass, captured once: replays with
    other layouts of the same sizes give what the same calls give run eagerly."""
    announce(f"a captured prompt round {fmt}")
    g = torch.Generator().manual_seed(50)
    n, total, hq, hkv, d, page, pages, blocks = 3, 150, 4, 2, 128, 16, 200, 64
    codes, exps = {"bf16": (BF16, None), "e4m3": (F8, torch.float32), "mxfp4": (U8, U8)}[fmt]
    width = d // 2 if fmt == "mxfp4" else d
    x = torch.randn((total, (hq + 2 * hkv) * d), generator=g).to(BF16).cuda()
    q, k, v = x[:, :hq * d].view(total, hq, d), x[:, hq * d:(hq + hkv) * d].view(total, hkv, d), x[:, (hq + hkv) * d:].view(total, hkv, d)
    w = torch.ones(d, device="cuda")
    freq = (1e4 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float().cuda()

    def state():
        s = dict(row_start=i32([0, 0, 0, 0]), kv_len=i32([0] * n), page_count=i32([0] * n), free_count=i32([pages]),
                 free_pages=torch.arange(pages, dtype=I32, device="cuda"), block_table=torch.full((n, blocks), -1, dtype=I32, device="cuda"),
                 slots=i32([-1] * total), positions=i32([0] * total))
        s["k"], s["v"] = (torch.zeros((pages, hkv, page, width), device="cuda").to(codes) for _ in "kv")
        scale = (pages, hkv, page, d // 32) if fmt == "mxfp4" else (pages, hkv, page)
        s["ks"], s["vs"] = (None, None) if exps is None else (torch.zeros(scale, dtype=exps, device="cuda") for _ in "kv")
        s["qo"], s["out"] = (torch.zeros((total, hq, d), dtype=BF16, device="cuda") for _ in "qo")
        s["ko"], s["vo"] = (torch.zeros((total, hkv, d), dtype=BF16, device="cuda") for _ in "kv")
        s["ws"] = torch.zeros(gdn.attn_prompt_workspace_bytes(hq, hkv, d, n, total, 1000), dtype=U8, device="cuda")
        return s

    def round_(s):
        gdn.kv_tables(s["row_start"], s["kv_len"], s["page_count"], s["free_count"], s["free_pages"], s["block_table"], s["slots"],
                      s["positions"], page_size=page)
        gdn.attn_prep(q, k, v, w, w, freq, s["positions"], s["slots"], s["qo"], s["k"], s["v"], s["ks"], s["vs"])
        gdn.attn_prompt(s["row_start"], s["kv_len"], s["block_table"], s["qo"], s["k"], s["v"], s["out"], s["ws"], max_kv=1000,
                        k_scale=s["ks"], v_scale=s["vs"])
        gdn.kv_read(s["row_start"], s["kv_len"], s["block_table"], s["k"], s["v"], s["ko"], s["vo"], k_scale=s["ks"], v_scale=s["vs"])

    a, b = state(), state()
    round_(state())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        round_(a)
    lens = [0] * n
    for rows in ([50, 50, 50], [150, 0, 0], [1, 17, 100], [0, 149, 1], [30, 30, 30]):
        for s in (a, b):
            s["row_start"].copy_(gi.starts_from_lengths(rows))
            s["kv_len"].copy_(torch.tensor(lens, dtype=I32))
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        round_(b)
        torch.cuda.synchronize()
        for name in ("out", "ko", "vo", "qo", "k", "v", "slots", "block_table"):
            assert torch.equal(a[name].view(U8), b[name].view(U8)), (rows, name)
        # and the definition: keys are normed and rotated, so the cache is taken as it stands
        rs = gi.starts_from_lengths(rows).tolist()
        out, mag, reach = ref.prompt(page, rs, lens, b["block_table"].cpu().numpy(), f64(b["qo"]), values(b["k"].cpu(), cpu(b["ks"])),
                                     values(b["v"].cpu(), cpu(b["vs"])), ref.default_scale(d))
        end = rs[-1]
        close(b["out"][:end], out[:end], ref.window_bound(out, mag, reach, d)[:end])
        lens = [p + m for p, m in zip(lens, rows)]


def cpu(t):
    return None if t is None else t.cpu()
