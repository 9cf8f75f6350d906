"""The attention-layer calls against the fp64 oracle: block tables, norms with
rotation and cache writes, attention of steps, windows and trees over the paged
cache, commits, and rounds of them together."""
import numpy as np
import pytest
import torch

from oracle import attn as ref
from verify_causal_conv1d_amd import gdn
from verify_causal_conv1d_amd import inputs as gi

from gpu_util import announce

pytestmark = pytest.mark.gpu

BF16, I32, F32, F8 = torch.bfloat16, torch.int32, torch.float32, torch.float8_e4m3fn


def i32(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def f64(t):
    return t.detach().cpu().double().numpy()


def values(pool, scale):
    """The values a cache holds, in fp64."""
    x = pool.cpu().float().double()
    return (x if scale is None else x * scale.cpu().double()[..., None]).numpy()


class Case:
    """Streams over a paged cache: every row that no stream holds is NaN."""

    def __init__(self, lens, rows, hq, hkv, d, page, e4m3=False, tree=False, gate=False, seed=0, amp=1.5, spare=3):
        g = self.g = torch.Generator().manual_seed(seed)
        self.lens, self.rows, self.hq, self.hkv, self.d, self.page = lens, rows, hq, hkv, d, page
        self.row_start = gi.starts_from_lengths(rows)
        self.total = int(self.row_start[-1])
        self.parent = gi.random_tree_parents(rows, g) if tree else None
        need = [-(-(a + b) // page) for a, b in zip(lens, rows)]
        self.pages = sum(need) + spare
        perm = torch.randperm(self.pages, generator=g).to(I32)
        self.table = torch.full((len(lens), max(need) + 1), -1, dtype=I32)
        self.free = perm[sum(need):]
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = perm[at:at + n]
            at += n
        shape = (self.pages, hkv, page, d)
        held = torch.zeros((self.pages, 1, page, 1), dtype=torch.bool)
        for s, n in enumerate(need):
            for j in range(n):
                held[self.table[s, j], 0, :max(0, min(page, lens[s] + rows[s] - j * page))] = True
        self.k, self.v, self.ks, self.vs = None, None, None, None
        for name in "kv":
            x = torch.randn(shape, generator=g)
            if e4m3:
                sc = x.abs().amax(-1) / 448.0
                x = (x / sc[..., None]).to(F8).view(torch.uint8)
                x = torch.where(held, x, torch.tensor(0x7F, dtype=torch.uint8)).view(F8)
                setattr(self, name + "s", torch.where(held[..., 0], sc, torch.tensor(float("nan"))))
            else:
                x = torch.where(held, x, torch.tensor(float("nan"))).to(BF16)
            setattr(self, name, x)
        self.q = (torch.randn((self.total, hq, d), generator=g) * amp).to(BF16)
        self.gate = (torch.randn((self.total, hq, 2 * d), generator=g) * 2).to(BF16) if gate else None
        self.kv_len = torch.tensor(lens, dtype=I32)

    def run(self, max_kv=None, max_rows=None, out=None, table=None, row_start=None, kv_len=None, parent=None, scale=None):
        cu = lambda t: None if t is None else t.cuda()  # noqa: E731
        max_kv = max_kv or max(a + b for a, b in zip(self.lens, self.rows))
        max_rows = max_rows or max(max(self.rows), 1)
        n = len(self.lens)
        out = torch.full((self.total, self.hq, self.d), float("nan"), dtype=BF16, device="cuda") if out is None else out
        ws = torch.full((gdn.attn_workspace_bytes(self.hq, self.hkv, self.d, n, self.total, max_rows, max_kv),), 0xFF,
                        dtype=torch.uint8, device="cuda")
        gate = self.gate.cuda()[:, :, self.d:] if self.gate is not None else None
        par = self.parent if parent is None else parent
        gdn.attn_window(cu(self.row_start if row_start is None else row_start), cu(self.kv_len if kv_len is None else kv_len),
                        cu(self.table if table is None else table), self.q.cuda(), cu(self.k), cu(self.v), out, ws,
                        max_kv=max_kv, max_rows=max_rows, parent=cu(par), gate=gate, k_scale=cu(self.ks), v_scale=cu(self.vs),
                        scale=scale)
        torch.cuda.synchronize()
        return out

    def oracle(self, scale=None):
        gate = None if self.gate is None else f64(self.gate[:, :, self.d:])
        out, mag, reach = ref.window(self.page, self.row_start.tolist(), None if self.parent is None else self.parent.tolist(),
                                     self.lens, self.table.numpy(), f64(self.q), values(self.k, self.ks),
                                     values(self.v, self.vs), ref.default_scale(self.d) if scale is None else scale, gate)
        return out, ref.window_bound(out, mag, reach, self.d)


def close(got, want, bound, what=""):
    got = f64(got)
    assert np.all(np.isfinite(got)), what
    worst = float(np.max(np.abs(got - want) / bound)) if got.size else 0.0
    print(f"{what} worst error {worst:.3f} of its bound")
    assert worst <= 1.0, (what, worst)


WINDOWS = [
    # one key, one row; then lengths around the tiles of 16 and 32 keys
    dict(lens=[0], rows=[1], hq=1, hkv=1, d=64, page=16),
    dict(lens=[0, 1, 15, 16, 17, 31, 32, 33], rows=[1] * 8, hq=4, hkv=2, d=64, page=16),
    dict(lens=[0, 1, 15, 16, 17, 31, 32, 33], rows=[1] * 8, hq=4, hkv=2, d=128, page=32, e4m3=True),
    dict(lens=[14, 30, 62, 126, 127, 128, 129, 255], rows=[2, 3, 4, 3, 1, 2, 16, 1], hq=6, hkv=1, d=256, page=16, gate=True),
    dict(lens=[14, 30, 62, 126, 127, 128, 129, 255], rows=[2, 3, 4, 3, 1, 2, 16, 1], hq=6, hkv=1, d=256, page=16, e4m3=True, gate=True),
    # windows and trees over chunks, streams without rows, pages that end inside a tile
    dict(lens=[300, 40, 511, 700, 0, 383], rows=[16, 0, 7, 1, 16, 2], hq=6, hkv=2, d=128, page=64, tree=True),
    dict(lens=[300, 40, 511, 700, 0, 383], rows=[16, 0, 7, 1, 16, 2], hq=6, hkv=2, d=128, page=16, tree=True, e4m3=True),
    dict(lens=[520, 0, 17], rows=[16, 16, 5], hq=24, hkv=4, d=256, page=64, tree=True, gate=True),
    dict(lens=[520, 0, 17], rows=[16, 16, 5], hq=24, hkv=4, d=256, page=256, tree=True, e4m3=True),
    dict(lens=[200, 90], rows=[16, 16], hq=16, hkv=1, d=64, page=128, gate=True),
    dict(lens=[77], rows=[3], hq=40, hkv=2, d=128, page=32),           # 20 heads a group: tiles that cut rows
    dict(lens=[1000, 1500], rows=[9, 12], hq=8, hkv=8, d=64, page=32, tree=True, e4m3=True),
    dict(lens=[2000, 5], rows=[4, 4], hq=8, hkv=2, d=256, page=32),
    dict(lens=[3000, 50, 1023], rows=[11, 5, 6], hq=9, hkv=3, d=128, page=128, gate=True),
    dict(lens=[250], rows=[16], hq=64, hkv=2, d=64, page=64, tree=True),
]


@pytest.mark.parametrize("kw", WINDOWS, ids=range(len(WINDOWS)))
def test_window_matches_oracle(kw):
    announce(f"attention {kw}")
    c = Case(seed=11, **kw)
    out, (want, bound) = c.run(), c.oracle()
    close(out, want, bound)


@pytest.mark.parametrize("n,e4m3,d", [(16384 - 3, False, 64), (16384 + 5, True, 64), (33000, False, 128), (40001, True, 256)])
def test_long_streams_beside_short_ones(n, e4m3, d):
    announce(f"attention over {n} keys, d {d}, e4m3 {e4m3}")
    c = Case([n, 3, 900], [2, 1, 3], 2, 1, d, 256, e4m3=e4m3, seed=12)
    close(c.run(), *c.oracle())


def test_many_streams_and_pieces():
    """More streams than a wave looks at together, and more pieces of work than workgroups."""
    g = torch.Generator().manual_seed(25)
    lens = torch.randint(0, 1400, (70,), generator=g).tolist()
    for rows, hq, e4m3, tree in (([1] * 70, 16, False, False), ([1 + i % 3 for i in range(70)], 32, True, True),
                                 ([(5 * i) % 9 for i in range(70)], 16, False, True)):
        announce(f"attention of 70 streams, up to {max(rows)} rows, {hq} heads, e4m3 {e4m3}")
        c = Case(lens, rows, hq, 4, 64, 32, e4m3=e4m3, tree=tree, seed=26, spare=9)
        close(c.run(), *c.oracle())


def test_longest_bound():
    """The largest max_kv: short streams under it give the same bits as under their own bound."""
    announce("attention under the largest max_kv")
    for rows in ([1, 2], [16, 9]):
        c = Case([600, 70], rows, 8, 2, 256, 64, seed=27)
        assert torch.equal(c.run(max_kv=1 << 21), c.run())


@pytest.mark.parametrize("hq,hkv,rows", [(1024, 1, 16), (1024, 1024, 2), (1024, 512, 9)])
def test_the_most_heads(hq, hkv, rows):
    announce(f"attention, {hq} heads over {hkv}")
    c = Case([40, 150], [rows, 1], hq, hkv, 64, 16, seed=32)
    close(c.run(), *c.oracle())


def test_streams_that_share_pages():
    """Two streams and a third that begin with the same pages: as if each had its own copy."""
    announce("attention over shared pages")
    for rows in (1, 9):
        c = Case([640, 700, 655], [rows] * 3, 6, 2, 128, 64, tree=rows > 1, seed=33)
        for s in (1, 2):
            for j in range(10):
                for pool in (c.k, c.v):
                    pool[c.table[s, j]] = pool[c.table[0, j]]
        want = c.run()
        table = c.table.clone()
        table[1:, :10] = table[0, :10]
        assert torch.equal(c.run(table=table), want)


def test_peaked_scores_and_scales():
    announce("attention, peaked rows, given scale")
    c = Case([500, 80], [5, 1], 4, 2, 128, 32, seed=13, amp=30.0)
    close(c.run(), *c.oracle())
    close(c.run(scale=0.0), *c.oracle(scale=0.0))
    close(c.run(scale=-0.02), *c.oracle(scale=-0.02))


def test_values_of_unseen_rows_reach_nobody():
    """Window rows that hold infinities or NaN, in K and in V, change only the rows that see them."""
    for e4m3 in (False, True):
        for d in (64, 256):
            announce(f"unseen rows, e4m3 {e4m3}, d {d}")
            c = Case([70, 130], [9, 9], 6, 2, d, 16, e4m3=e4m3, seed=14)
            c.parent = torch.tensor([-1, 0, 0, 2, 1, 3, 5, 4, 0] * 2, dtype=I32)
            clean = c.run()
            par = c.parent[:9].tolist()
            sees = [[u in ref.ancestors(par, t) for u in range(9)] for t in range(9)]
            bad = 3
            for s, (pool, value) in enumerate(((c.v, float("nan")), (c.v, float("inf")), (c.k, float("nan")), (c.k, float("-inf")))):
                if e4m3 and not np.isnan(value):
                    continue
                for st in range(2):
                    at = c.lens[st] + bad
                    page = int(c.table[st, at // 16])
                    keep = pool[page, :, at % 16].clone()
                    pool[page, :, at % 16] = torch.full((2, d), value).to(pool.dtype)
                    got = c.run()
                    pool[page, :, at % 16] = keep
                    for t in range(18):
                        hit = t // 9 == st and sees[t % 9][bad]
                        if not hit:
                            assert torch.equal(got[t], clean[t]), (s, st, t)
                        elif pool is c.v and value == float("inf"):
                            assert torch.isinf(got[t]).all() and (got[t] > 0).all(), (s, st, t)
                        elif value != value:
                            assert torch.isnan(got[t]).all(), (s, st, t)
            if e4m3:       # a scale that is not finite is its row's alone, too
                for pool in (c.ks, c.vs):
                    at = c.lens[0] + bad
                    page = int(c.table[0, at // 16])
                    keep = pool[page, :, at % 16].clone()
                    pool[page, :, at % 16] = float("nan")
                    got = c.run()
                    pool[page, :, at % 16] = keep
                    for t in range(18):
                        if t < 9 and sees[t][bad]:
                            assert torch.isnan(got[t]).all()
                        else:
                            assert torch.equal(got[t], clean[t]), t


def test_cached_rows_that_are_not_finite_reach_all_rows():
    """An infinite or NaN value of a cached row, in the window's tile of keys or before it, is seen by every row of its stream."""
    for e4m3, rows, d in ((False, 2, 64), (False, 9, 128), (False, 9, 256), (True, 2, 256), (True, 9, 64), (True, 9, 256)):
        announce(f"cached rows that are not finite, e4m3 {e4m3}, {rows} rows, d {d}")
        c = Case([70, 333], [rows, rows], 6, 2, d, 16, e4m3=e4m3, seed=30)
        clean = c.run()
        for value in (float("nan"),) if e4m3 else (float("nan"), float("inf"), float("-inf")):
            for s, key in ((0, 69), (0, 64), (0, 63), (0, 0), (1, 332), (1, 320), (1, 319)):
                page = int(c.table[s, key // 16])
                keep = c.v[page, :, key % 16].clone()
                c.v[page, :, key % 16] = torch.full((2, d), value).to(c.v.dtype)
                got = c.run()
                c.v[page, :, key % 16] = keep
                hit, other = (got[:rows], got[rows:]) if s == 0 else (got[rows:], got[:rows])
                assert torch.equal(other, clean[rows:] if s == 0 else clean[:rows]), (value, s, key)
                assert torch.isnan(hit).all() if value != value else (hit == value).all(), (value, s, key)


def test_streams_do_not_depend_on_each_other():
    """Each stream alone gives the bits it gives in the batch, wherever it is packed."""
    for tree in (False, True):
        announce(f"attention, batch against single streams, tree {tree}")
        lens, rows = [700, 3, 5000, 130], [5, 16, 9, 1]
        c = Case(lens, rows, 12, 2, 128, 32, tree=tree, seed=15)
        whole = c.run(max_rows=16)
        back = c.run(max_rows=16, max_kv=1 << 20)
        assert torch.equal(whole, back)
        for s in range(4):
            a, b = int(c.row_start[s]), int(c.row_start[s + 1])
            one = Case.__new__(Case)
            one.__dict__.update(c.__dict__)
            one.lens, one.rows, one.row_start, one.total = [lens[s]], [rows[s]], torch.tensor([0, b - a], dtype=I32), b - a
            one.table, one.kv_len, one.q = c.table[s:s + 1].contiguous(), c.kv_len[s:s + 1], c.q[a:b].contiguous()
            one.parent = None if c.parent is None else c.parent[a:b].contiguous()
            assert torch.equal(one.run(max_rows=16), whole[a:b]), s


def test_broken_streams_are_skipped():
    lens, rows = [300, 70, 900, 40], [4, 4, 4, 4]
    for tree in (False, True):
        c = Case(lens, rows, 4, 2, 128, 16, tree=tree, seed=16)
        good = c.run()
        announce(f"skipped streams, tree {tree}")

        def same_but(got, streams):
            for s in range(4):
                a, b = int(c.row_start[s]), int(c.row_start[s + 1])
                if s in streams:
                    assert torch.isnan(got[a:b]).all(), s
                else:
                    assert torch.equal(got[a:b], good[a:b]), s
        for s, j in ((0, 3), (1, 0), (2, 56), (3, 2)):      # a page outside the cache, in the first, a middle and the last block
            for page in (-1, c.pages, 1 << 30):
                t = c.table.clone()
                t[s, j] = page
                same_but(c.run(table=t), {s})
        kv = c.kv_len.clone()
        kv[1] = -1
        same_but(c.run(kv_len=kv), {1})
        kv[1] = 10 ** 6
        same_but(c.run(kv_len=kv), {1})
        kv[1] = 2 ** 31 - 1
        same_but(c.run(kv_len=kv), {1})
        same_but(c.run(max_kv=500), {2})
        rs = c.row_start.clone()
        rs[4] = 14                                          # the last window ends early: its last two rows belong to nobody
        got = c.run(row_start=rs)
        assert torch.equal(got[:12], good[:12]) and torch.isnan(got[14:]).all()
        rs[4] = 17
        same_but(c.run(row_start=rs), {3})                  # past the packed rows
        rs[4] = -5
        same_but(c.run(row_start=rs), {3})
        if tree:
            for bad in (2, -2, 9):
                p = c.parent.clone()
                p[4 + 2] = bad
                same_but(c.run(parent=p), {1})
                p = c.parent.clone()
                p[8] = bad
                same_but(c.run(parent=p), {2})


def test_a_falling_row_start_skips_its_two_streams_only():
    announce("attention of 70 streams, one falling row_start")
    rows = [2] * 70
    c = Case([300 + 7 * s for s in range(70)], rows, 4, 2, 64, 32, seed=31)
    good = c.run()
    for at in (64, 3):
        for value in (-5, 0, 10 ** 6):
            rs = c.row_start.clone()
            rs[at] = value
            got = c.run(row_start=rs)
            for s in range(70):
                if s in (at - 1, at):
                    assert torch.isnan(got[2 * s:2 * s + 2]).all(), (at, value, s)
                else:
                    assert torch.equal(got[2 * s:2 * s + 2], good[2 * s:2 * s + 2]), (at, value, s)


def test_offsets_past_32_bits():
    """A cache of more than 4 GiB, its pages at the far end."""
    announce("attention, 6 GiB pools")
    c = Case([130, 700], [3, 1], 4, 2, 128, 64, seed=17)
    pages = (6 << 30) // (2 * 64 * 128 * 2)
    first = pages - c.pages
    want = c.run()
    k, v = (torch.empty((pages, 2, 64, 128), dtype=BF16, device="cuda") for _ in range(2))
    k[first:], v[first:] = c.k.cuda(), c.v.cuda()
    table = torch.where(c.table >= 0, c.table + first, c.table).cuda()
    out = torch.zeros_like(want)
    ws = torch.empty(gdn.attn_workspace_bytes(4, 2, 128, 2, 4, 3, 701), dtype=torch.uint8, device="cuda")
    gdn.attn_window(c.row_start.cuda(), c.kv_len.cuda(), table, c.q.cuda(), k, v, out, ws, max_kv=701, max_rows=3)
    assert torch.equal(out, want)
    # a row written and moved there
    slots = i32([(pages - 1) * 64 + 63])
    x = torch.randn((1, 2, 128), device="cuda").to(BF16)
    qo = torch.zeros((1, 4, 128), dtype=BF16, device="cuda")
    gdn.attn_prep(torch.zeros((1, 4, 128), dtype=BF16, device="cuda"), x, x, None, None, torch.zeros(0, device="cuda"), i32([0]), slots,
                  qo, k, v)
    assert torch.equal(k[pages - 1, :, 63], x[0]) and torch.equal(v[pages - 1, :, 63], x[0])
    length = i32([62])
    gdn.attn_commit(i32([0, 2]), i32([1]), length, i32([[pages - 1]]), k, v, parent=i32([-1, -1]))
    torch.cuda.synchronize()
    assert torch.equal(k[pages - 1, :, 62], x[0]) and torch.equal(v[pages - 1, :, 62], x[0]) and length.item() == 63


# ---- norms, rotation, cache writes ------------------------------------------

PREPS = [(R, hq, hkv, d, rot, page, e4m3, inter, norm)
         for R, hq, hkv, d, rot, page, e4m3, inter, norm in [
             (1, 1, 1, 64, 0, 16, False, False, True), (5, 4, 2, 64, 64, 16, False, False, True),
             (5, 4, 2, 64, 64, 16, True, True, True), (33, 24, 4, 256, 64, 64, False, False, True),
             (33, 24, 4, 256, 64, 64, True, True, False), (7, 6, 2, 128, 50, 32, False, False, True),
             (7, 6, 2, 128, 50, 32, True, True, True), (7, 3, 3, 128, 2, 256, False, False, False),
             (7, 9, 3, 128, 126, 128, True, False, True), (64, 8, 1, 256, 256, 16, False, False, True),
             (64, 7, 7, 256, 256, 16, True, True, True), (300, 2, 1, 64, 22, 16, False, True, True)]]


@pytest.mark.parametrize("R,hq,hkv,d,rot,page,e4m3,inter,norm", PREPS)
def test_prep_matches_oracle(R, hq, hkv, d, rot, page, e4m3, inter, norm):
    announce(f"prep rows {R} heads {hq}/{hkv} d {d} rot {rot} page {page} e4m3 {e4m3} interleaved {inter} norm {norm}")
    g = torch.Generator().manual_seed(R + d + rot)
    x = (torch.randn((R, (2 * hq + 2 * hkv) * d + 8), generator=g) * 3).to(BF16)
    x[R // 2, :2 * hq * d] = 0                                      # a row of zero queries
    xc = x.cuda()
    q = xc[:, :2 * hq * d].view(R, hq, 2 * d)[:, :, :d]
    k = xc[:, 2 * hq * d:(2 * hq + hkv) * d].view(R, hkv, d)
    v = xc[:, (2 * hq + hkv) * d:(2 * hq + 2 * hkv) * d].view(R, hkv, d)
    w = [1 + 0.3 * torch.randn(d, generator=g) for _ in range(2)] if norm else [None, None]
    freq = (5e5 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float()
    pos = torch.randint(0, 1 << 18, (R,), generator=g).to(I32)
    pos[0] = (1 << 24) - 1
    pages = R // page + 2
    slots = torch.randperm(pages * page, generator=g)[:R].to(I32)
    skip = R // 3 if R > 3 else None                                # rows without a slot store nothing
    if skip is not None:
        slots[skip], slots[skip + 1] = -1, pages * page
    shape = (pages, hkv, page, d)
    fill = torch.full(shape, 3.0).to(F8 if e4m3 else BF16).cuda()
    kc, vc = fill.clone(), fill.clone()
    ks, vs = ((torch.full(shape[:3], 7.0, device="cuda") for _ in range(2)) if e4m3 else (None, None))
    qo = torch.full((R, hq, d), float("nan"), dtype=BF16, device="cuda")
    rs = 1.25 if inter else 1.0
    gdn.attn_prep(q, k, v, *[None if t is None else t.cuda() for t in w], freq.cuda(), pos.cuda(), slots.cuda(), qo, kc, vc, ks, vs,
                  eps=1e-5, interleaved=inter, rot_scale=rs)
    torch.cuda.synchronize()

    def want(t, weight):
        n = ref.normed(f64(t), None if weight is None else weight.double().numpy(), 1e-5)
        return ref.rotated(n, pos.numpy(), freq.double().numpy(), inter, rs)
    # half a bf16 step of the result, and 2^-20 of its terms: fp32 norm, angle, products and sum
    y, mag = want(q, w[0])
    assert np.all(np.abs(f64(qo) - y) <= 2.0 ** -8 * np.abs(y) + 2.0 ** -19 * mag + 1e-38)
    kw, kmag = want(k, w[1])
    kc_, vc_, kref = f64(kc.float()), f64(vc.float()), f64(fill.float())
    written = np.zeros(shape[:3], bool)
    for r in range(R):
        s = int(slots[r])
        if s < 0 or s >= pages * page:
            continue
        p, o = s // page, s % page
        written[p, :, o] = True
        for pool, sc, ref_, m in ((kc_, ks, kw, kmag), (vc_, vs, f64(v), np.abs(f64(v)))):
            if not e4m3:
                assert np.all(np.abs(pool[p, :, o] - ref_[r]) <= 2.0 ** -8 * np.abs(ref_[r]) + 2.0 ** -19 * m[r] + 1e-38), r
                continue
            top = np.abs(ref_[r]).max(-1)
            scale = f64(sc)[p, :, o]
            assert np.all(np.abs(scale * 448 - np.maximum(top, 2.0 ** -100)) <= 2.0 ** -18 * m[r].max(-1) + 1e-40), r
            got = pool[p, :, o] * scale[:, None]
            # half an e4m3 step: 2^-4 of the value, or half the smallest step (2^-9 of the scale)
            assert np.all(np.abs(got - ref_[r]) <= 2.0 ** -4 * np.abs(ref_[r]) + 2.0 ** -10 * scale[:, None] + 2.0 ** -18 * m[r]), r
    for pool in (kc_, vc_):
        assert np.array_equal(pool[~written], kref[~written])       # nothing else is touched
    if e4m3:
        assert np.all(f64(ks)[~written] == 7.0) and np.all(f64(vs)[~written] == 7.0)


def test_e4m3_rows_of_zeros_and_extremes():
    announce("e4m3 rows: zeros, tiny, huge, infinite")
    d, R = 64, 5
    x = torch.zeros((R, 1, d))
    x[1] = torch.randn((1, d), generator=torch.Generator().manual_seed(1)) * 2.0 ** -126
    x[2, 0, 5], x[2, 0, 6] = 3.3e38, -1e30
    x[3, 0, 5], x[3, 0, 6] = 448.0, 0.25
    x[4, 0, 5] = float("inf")
    x = x.to(BF16).cuda()
    kc, vc = (torch.zeros((1, 1, 16, d), device="cuda").to(F8) for _ in range(2))
    ks, vs = (torch.zeros((1, 1, 16), device="cuda") for _ in range(2))
    qo = torch.zeros((R, 1, d), dtype=BF16, device="cuda")
    gdn.attn_prep(x, x, x, None, None, torch.zeros(0, device="cuda"), i32([0] * R), i32(list(range(R))), qo, kc, vc, ks, vs)
    torch.cuda.synchronize()
    got = values(vc, vs)[0, 0]
    assert np.all(got[0] == 0) and float(vs[0, 0, 0]) > 0
    assert np.all(np.abs(got[1] - f64(x)[1, 0]) < 2.0 ** -100)          # below the least maximum: within the zero of its step
    assert abs(got[2, 5] / f64(x)[2, 0, 5] - 1) <= 2.0 ** -4 and got[2, 6] == 0
    assert got[3, 5] == 448 and got[3, 6] == 0.25
    assert not np.isfinite(got[4]).any()
    assert torch.equal(qo, x)


# ---- block tables --------------------------------------------------------------

def tables_case(n, page, seed, tree=False, free=50, max_len=300, prompt=0, gap=0):
    g = np.random.default_rng(seed)
    kv = g.integers(0, max_len, n)
    rows = g.integers(0, 17, n) if not prompt else np.where(g.random(n) < 0.3, g.integers(0, prompt, n), g.integers(0, 4, n))
    kv[g.random(n) < 0.2] = -1
    have = np.maximum(0, -(-np.maximum(kv, 0) // page) + g.integers(-1, 3, n))
    have[kv < 0] = g.integers(0, max_len // page + 1, int((kv < 0).sum()))
    total_held = int(have.sum())
    perm = g.permutation(total_held + free).astype(np.int32)
    blocks = max(int(have.max()), int((-(-(np.maximum(kv, 0) + rows) // page)).max())) + 1
    table = np.full((n, blocks), -7, np.int32)
    at = 0
    for s in range(n):
        table[s, :have[s]] = perm[at:at + have[s]]
        at += have[s]
    stack = np.full(total_held + free, -3, np.int32)
    stack[:free] = perm[at:]
    rs = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32) + gap
    parent = gi.random_tree_parents(rows.tolist(), torch.Generator().manual_seed(seed)).numpy() if tree else None
    if parent is not None:
        parent = np.concatenate([np.zeros(gap, np.int32), parent, np.zeros(gap, np.int32)]).astype(np.int32)
    total = int(rs[-1]) + gap
    return dict(row_start=rs, parent=parent, kv_len=kv.astype(np.int32), page_count=have.astype(np.int32),
                free_count=np.array([free], np.int32), free_pages=stack, block_table=table,
                slots=np.full(total, -9, np.int32), positions=np.full(total, -9, np.int32))


def run_tables(c, page, in_place):
    d = {k: None if v is None else torch.from_numpy(v.copy()).cuda() for k, v in c.items()}
    pc, fc = (d["page_count"], d["free_count"]) if in_place else (torch.full_like(d["page_count"], -5), torch.full_like(d["free_count"], -5))
    gdn.kv_tables(d["row_start"], d["kv_len"], d["page_count"], d["free_count"], d["free_pages"], d["block_table"], d["slots"],
                  d["positions"], page_size=page, parent=d["parent"], page_count_out=None if in_place else pc,
                  free_count_out=None if in_place else fc)
    torch.cuda.synchronize()
    if not in_place:
        assert np.array_equal(d["page_count"].cpu().numpy(), c["page_count"])
    return dict(block_table=d["block_table"], free_pages=d["free_pages"], page_count=pc, free_count=fc, slots=d["slots"],
                positions=d["positions"])


def check_tables(c, page):
    want = ref.tables(page, c["row_start"], c["parent"], c["kv_len"], c["page_count"], c["free_count"][0], c["free_pages"],
                      c["block_table"], c["slots"], c["positions"])
    for in_place in (False, True):
        got = run_tables(c, page, in_place)
        for k, w in want.items():
            assert np.array_equal(got[k].cpu().numpy().reshape(-1), np.asarray(w).reshape(-1)), (k, in_place)


@pytest.mark.parametrize("n,page,tree,free,max_len,prompt,gap", [
    (1, 16, False, 50, 100, 0, 0), (7, 16, True, 50, 100, 0, 3), (16, 64, True, 100, 5000, 0, 0), (64, 32, False, 60, 300, 0, 5),
    (65, 32, False, 200, 300, 0, 0), (200, 16, True, 500, 2000, 0, 2), (16, 16, False, 3, 200, 0, 0), (300, 128, False, 40, 3000, 0, 0),
    (20, 16, False, 400, 500, 900, 0), (1500, 16, False, 3000, 200, 40, 0), (4096, 256, True, 4000, 1000, 0, 0), (3, 16, False, 0, 50, 0, 0)])
def test_tables_match_oracle(n, page, tree, free, max_len, prompt, gap):
    announce(f"tables n {n} page {page} tree {tree} free {free} len {max_len} prompt {prompt}")
    for seed in range(3):
        check_tables(tables_case(n, page, 100 * seed + n, tree, free, max_len, prompt, gap), page)


def test_tables_edges():
    announce("tables: no streams, all finished, a table that is too short, broken counts and windows")
    c = tables_case(5, 16, 7)
    empty = dict(c, row_start=c["row_start"][:1], kv_len=c["kv_len"][:0], page_count=c["page_count"][:0],
                 block_table=c["block_table"][:0], slots=c["slots"][:0], positions=c["positions"][:0])
    d = {k: None if v is None else torch.from_numpy(v.copy()).cuda() for k, v in empty.items()}
    out = i32([-1])
    gdn.kv_tables(d["row_start"], d["kv_len"], d["page_count"], d["free_count"], d["free_pages"], d["block_table"], d["slots"],
                  d["positions"], page_size=16, free_count_out=out)
    assert out.item() == 50
    done = dict(c, kv_len=np.full(5, -1, np.int32))
    check_tables(done, 16)
    short = dict(c, kv_len=np.array([3, 10 ** 6, 5, -1, 2], np.int32))     # stream 1 does not fit its table
    check_tables(short, 16)
    got = run_tables(dict(c, kv_len=np.array([3, 2 ** 31 - 1, 5, -1, 2], np.int32)), 16, False)
    a, b = c["row_start"][1:3]
    assert (got["slots"][a:b] == -1).all()
    # broken counts and windows: that stream keeps what it has and gets no slots, nothing faults
    for key, s, value in (("page_count", 1, -4), ("page_count", 1, 10 ** 6), ("row_start", 2, -3), ("row_start", 2, 10 ** 6)):
        x = c[key].copy()
        x[s] = value
        got = run_tables(dict(c, **{key: x}), 16, False)
        assert torch.equal(got["block_table"][1].cpu(), torch.from_numpy(c["block_table"][1]))
        lo, hi = max(0, int(c["row_start"][1])), int(c["row_start"][2])
        assert (got["slots"][lo:hi] <= -1).all()
    for fc in (-1, 10 ** 6):
        got = run_tables(dict(c, free_count=np.array([fc], np.int32)), 16, False)
        assert 0 <= got["free_count"].item() <= c["free_pages"].shape[0]


@pytest.mark.parametrize("n", [5, 70])
def test_tables_with_a_falling_row_start(n):
    """Its two streams keep their pages and get no slots; the others are served as ever."""
    announce(f"tables of {n} streams, one falling row_start")
    c = tables_case(n, 16, 8, free=400)
    c["kv_len"] = np.maximum(c["kv_len"], 0)
    at = n // 2
    # the oracle's two streams do not fit their tables instead: the same outputs
    kv = c["kv_len"].copy()
    kv[at - 1:at + 1] = 10 ** 6
    want = ref.tables(16, c["row_start"], None, kv, c["page_count"], 400, c["free_pages"], c["block_table"], c["slots"], c["positions"])
    for value in (-5, 10 ** 6, 2 ** 31 - 1):
        rs = c["row_start"].copy()
        rs[at] = value
        for in_place in (False, True):
            got = run_tables(dict(c, row_start=rs), 16, in_place)
            for k, w in want.items():
                assert np.array_equal(got[k].cpu().numpy().reshape(-1), np.asarray(w).reshape(-1)), (k, value, in_place)


# ---- commits --------------------------------------------------------------------

@pytest.mark.parametrize("e4m3,d,page,hkv", [(False, 64, 16, 1), (True, 64, 16, 3), (False, 256, 64, 4), (True, 256, 32, 2), (False, 128, 256, 9)])
def test_commit_matches_oracle(e4m3, d, page, hkv):
    announce(f"commit e4m3 {e4m3} d {d} page {page} hkv {hkv}")
    lens, rows = [0, 14, 250, 63, 5, 40, 31], [16, 16, 9, 1, 0, 12, 16]
    c = Case(lens, rows, hkv, hkv, d, page, e4m3=e4m3, tree=True, seed=18)
    rs = c.row_start.tolist()
    accept = [rs[0] + 15, rs[1] + 11, rs[2] + 8, rs[3], -1, rs[5] + 6, rs[6] + 13]
    # several roots: the first kept row moves, too
    c.parent[rs[5]:rs[6]] = torch.tensor([-1, 0, -1, 2, 2, 3, 4, 4, -1, 8, 8, 10], dtype=I32)
    for chain in (False, True):
        parent = None if chain else c.parent
        pools = [t for t in (c.k, c.v, c.ks, c.vs) if t is not None]
        raw = [t.view(torch.uint8).numpy() if t.dtype in (F8,) else t.view(torch.int16).numpy() if t.dtype == BF16 else t.view(I32).numpy()
               for t in pools]
        want, length = ref.commit(page, rs, None if chain else c.parent.tolist(), accept, lens, c.table.numpy(), *raw)
        for in_place in (False, True):
            dev = [t.cuda().clone() for t in pools]
            kv = c.kv_len.cuda().clone()
            out = kv if in_place else torch.full_like(kv, -1)
            gdn.attn_commit(c.row_start.cuda(), i32(accept), kv, c.table.cuda(), dev[0], dev[1], *(dev[2:] or (None, None)),
                            parent=None if chain else parent.cuda(), kv_len_out=None if in_place else out)
            torch.cuda.synchronize()
            assert out.cpu().tolist() == length.tolist()
            for got, w, t in zip(dev, want, pools):
                view = torch.uint8 if t.dtype == F8 else torch.int16 if t.dtype == BF16 else I32
                assert np.array_equal(got.cpu().view(view).numpy(), w)


def test_commit_skips_what_breaks_the_rules():
    announce("commit, broken streams")
    c = Case([20, 30], [6, 6], 1, 1, 64, 16, tree=True, seed=19)
    c.parent = torch.tensor([-1, 0, 0, 2, 2, 4] * 2, dtype=I32)

    def go(accept=(5, 11), parent=None, table=None, kv=None, rs=None):
        k, v, length = c.k.cuda(), c.v.cuda(), (c.kv_len if kv is None else kv).cuda().clone()
        gdn.attn_commit((c.row_start if rs is None else rs).cuda(), i32(list(accept)), length, (c.table if table is None else table).cuda(),
                        k, v, parent=(c.parent if parent is None else parent).cuda())
        torch.cuda.synchronize()
        return k.cpu(), length.cpu().tolist()
    good, length = go()
    assert length == [24, 34]
    only_second, _ = go(accept=(-1, 11))
    no_page = c.table.clone()
    no_page[0, 1] = c.pages
    for kw in (dict(accept=(6, 11)), dict(accept=(12, 11)), dict(accept=(-3, 11)),
               dict(parent=torch.tensor([-1, 0, 2, 2, 2, 4] + [-1, 0, 0, 2, 2, 4], dtype=I32)),
               dict(parent=torch.tensor([-1, 0, -2, 2, 2, 4] + [-1, 0, 0, 2, 2, 4], dtype=I32)),
               dict(rs=torch.tensor([-1, 6, 12], dtype=I32)), dict(table=no_page)):
        k, length = go(**kw)
        assert length == [20, 34], kw
        assert torch.equal(k.view(torch.int16), only_second.view(torch.int16)), kw
    k, length = go(kv=torch.tensor([-1, 30], dtype=I32))
    assert length == [-1, 34] and torch.equal(k.view(torch.int16), only_second.view(torch.int16))


# ---- together ---------------------------------------------------------------------

class Server:
    """Streams of one attention layer: every count on the device, buffers made once."""

    def __init__(self, n, hq, hkv, d, page, e4m3, pages, blocks, rows, max_kv, rot, seed):
        g = self.g = torch.Generator().manual_seed(seed)
        self.n, self.hq, self.hkv, self.d, self.page, self.rows, self.max_kv = n, hq, hkv, d, page, rows, max_kv
        shape = (pages, hkv, page, d)
        nan = torch.full(shape, float("nan"), device="cuda")
        self.k, self.v = nan.to(F8 if e4m3 else BF16), nan.to(F8 if e4m3 else BF16)
        self.ks, self.vs = (torch.full(shape[:3], float("nan"), device="cuda") for _ in range(2)) if e4m3 else (None, None)
        self.kv_len, self.page_count = i32([0] * n), i32([0] * n)
        self.free_pages, self.free_count = torch.randperm(pages, generator=g).to(I32).cuda(), i32([pages])
        self.table = torch.full((n, blocks), -1, dtype=I32, device="cuda")
        total = n * rows
        self.row_start, self.parent, self.accept = i32([0] * (n + 1)), i32([-1] * total), i32([-1] * n)
        self.slots, self.positions = i32([-1] * total), i32([0] * total)
        self.x = torch.zeros((total, 2 * hq + 2 * hkv, d), dtype=BF16, device="cuda")
        self.q = torch.zeros((total, hq, d), dtype=BF16, device="cuda")
        self.out = torch.zeros((total, hq, d), dtype=BF16, device="cuda")
        self.w = (1 + 0.2 * torch.randn((2, d), generator=g)).cuda()
        self.freq = (1e4 ** (-torch.arange(0, rot, 2).double() / rot)).float().cuda()
        self.ws = torch.empty(gdn.attn_workspace_bytes(hq, hkv, d, n, total, rows, max_kv), dtype=torch.uint8, device="cuda")

    def forward(self):
        hq, hkv = self.hq, self.hkv
        gdn.kv_tables(self.row_start, self.kv_len, self.page_count, self.free_count, self.free_pages, self.table, self.slots,
                      self.positions, page_size=self.page, parent=self.parent)
        gdn.attn_prep(self.x[:, :hq], self.x[:, 2 * hq:2 * hq + hkv], self.x[:, 2 * hq + hkv:], self.w[0], self.w[1], self.freq,
                      self.positions, self.slots, self.q, self.k, self.v, self.ks, self.vs)
        gdn.attn_window(self.row_start, self.kv_len, self.table, self.q, self.k, self.v, self.out, self.ws, max_kv=self.max_kv,
                        max_rows=self.rows, parent=self.parent, gate=self.x[:, hq:2 * hq], k_scale=self.ks, v_scale=self.vs)

    def commit(self):
        gdn.attn_commit(self.row_start, self.accept, self.kv_len, self.table, self.k, self.v, self.ks, self.vs, parent=self.parent,
                        max_rows=self.rows)

    def draw(self, lens):
        rows = gi.starts_from_lengths(lens)
        R = int(rows[-1])
        self.row_start.copy_(rows)
        parent = torch.full((self.n * self.rows,), -1, dtype=I32)
        parent[:R] = gi.random_tree_parents(lens, self.g)
        self.parent.copy_(parent)
        self.accept.copy_(torch.tensor([int(a) + int(torch.randint(0, m, (1,), generator=self.g)) if m else -1
                                        for a, m in zip(rows, lens)], dtype=I32))
        self.x.copy_((torch.randn(self.x.shape, generator=self.g) * 1.5).to(BF16))
        return R


@pytest.mark.parametrize("e4m3,d,rot,page", [(False, 128, 32, 16), (True, 64, 64, 16), (False, 256, 64, 32)])
def test_rounds_of_all_calls(e4m3, d, rot, page):
    """Draft trees of three streams, round after round: tables, norms and cache
    writes, attention, commit; against dense histories kept by the oracle."""
    n, rows = 3, 12
    announce(f"rounds of all calls, e4m3 {e4m3}, d {d}")
    sv = Server(n, 6, 2, d, page, e4m3, 40, 12, rows, 160, rot, seed=20)
    hist = [([], []) for _ in range(n)]                  # each stream's kept (pre-norm k, v) rows
    w = f64(sv.w)
    for rnd in range(9):
        lens = [[12, 1, 7], [3, 12, 0], [12, 12, 12]][rnd % 3]
        R = sv.draw(lens)
        if rnd == 5:                                     # the second stream ends, and its place is taken by a new one
            sv.kv_len[1] = -1
            gdn.kv_tables(i32([0] * 4), sv.kv_len, sv.page_count, sv.free_count, sv.free_pages, sv.table, i32([]), i32([]), page_size=page)
            sv.kv_len[1] = 0
            hist[1] = ([], [])
        before = sv.kv_len.cpu().tolist()
        assert before == [len(h[0]) for h in hist]
        sv.out.fill_(float("nan"))
        sv.forward()
        torch.cuda.synchronize()
        x, rs, parent, out = f64(sv.x), sv.row_start.cpu().tolist(), sv.parent.cpu().tolist(), f64(sv.out)
        assert np.isnan(out[R:]).all()
        hq, hkv = sv.hq, sv.hkv
        kcache, vcache = values(sv.k, sv.ks), values(sv.v, sv.vs)
        for s in range(n):
            par = parent[rs[s]:rs[s + 1]]
            for t in range(len(par)):
                r = rs[s] + t
                path = ref.ancestors(par, t)
                pos = before[s] + len(path) - 1
                assert sv.positions[r].item() == pos
                ks = hist[s][0] + [x[rs[s] + u, 2 * hq:2 * hq + hkv] for u in path]
                vs = hist[s][1] + [x[rs[s] + u, 2 * hq + hkv:] for u in path]
                q, _ = ref.rotated(ref.normed(x[r:r + 1, :hq], w[0], 1e-6), [pos], f64(sv.freq), False)
                kk, _ = ref.rotated(ref.normed(np.array(ks), w[1], 1e-6), range(len(ks)), f64(sv.freq), False)
                vv = np.array(vs)
                for h in range(hq):
                    lo = kk[:, h // (hq // hkv)] @ q[0, h] * d ** -0.5
                    # q and k are stored in bf16 (2^-8 each), or k in e4m3 (2^-4): an error of the
                    # scores of e of their terms' size moves each weight by a factor of at most e^{2e}
                    e = np.max(np.abs(kk[:, h // (hq // hkv)]) @ np.abs(q[0, h])) * d ** -0.5 * (2.0 ** -8 + (2.0 ** -4 if e4m3 else 2.0 ** -8))
                    p = np.exp(lo - lo.max())
                    p /= p.sum()
                    gate = 1 / (1 + np.exp(-x[r, hq + h]))
                    want, mag = p @ vv[:, h // (hq // hkv)] * gate, p @ np.abs(vv[:, h // (hq // hkv)]) * gate
                    bound = 2.0 ** -8 * np.abs(want) + mag * (np.expm1(2 * e) + 2.0 ** -7 + (2.0 ** -4 if e4m3 else 0.0))
                    assert np.all(np.abs(out[r, h] - want) <= bound), (rnd, s, t, h)
        # the exact form of the check above: the cache's own values and the stored queries
        table = sv.table.cpu().numpy()
        o, m, reach = ref.window(page, rs, parent, before, table, f64(sv.q)[:R], kcache, vcache, d ** -0.5, x[:R, hq:2 * hq])
        close(torch.from_numpy(out[:R]), o, ref.window_bound(o, m, reach, d), f"round {rnd}")
        sv.commit()
        torch.cuda.synchronize()
        acc = sv.accept.cpu().tolist()
        for s in range(n):
            par = parent[rs[s]:rs[s + 1]]
            if par:
                for u in ref.ancestors(par, acc[s] - rs[s]):
                    hist[s][0].append(x[rs[s] + u, 2 * hq:2 * hq + hkv])
                    hist[s][1].append(x[rs[s] + u, 2 * hq + hkv:])
    held = sv.page_count.cpu().tolist()
    used = [int(sv.table[s, j]) for s in range(n) for j in range(held[s])] + sv.free_pages[:sv.free_count.item()].cpu().tolist()
    assert sorted(used) == list(range(40))               # no page is lost or held twice


def test_captured_rounds_equal_eager_rounds():
    """A round captured once and replayed on new trees, with eager work between the replays."""
    announce("graph capture of attention rounds")
    args = dict(n=3, hq=6, hkv=2, d=128, page=16, e4m3=False, pages=64, blocks=20, rows=8, max_kv=300, rot=32, seed=21)
    a, b = Server(**args), Server(**args)

    def rnd(s):
        s.forward()
        s.commit()
    a.draw([8, 8, 8])
    b.draw([8, 8, 8])
    rnd(a)                                     # an eager round first, on both
    rnd(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rnd(a)
    torch.cuda.synchronize()
    for i, lens in enumerate(([8, 3, 8], [1, 1, 1], [8, 0, 5], [8, 8, 8], [2, 8, 8])):
        a.draw(lens)
        b.draw(lens)
        graph.replay()
        torch.cuda.synchronize()
        rnd(b)
        torch.cuda.synchronize()
        R = sum(lens)
        assert torch.equal(a.out[:R], b.out[:R]) and not torch.isnan(a.out[:R]).any(), i
        for name in ("kv_len", "page_count", "free_count", "table", "slots", "positions"):
            assert torch.equal(getattr(a, name), getattr(b, name)), (i, name)
        assert torch.equal(a.k.view(torch.int16), b.k.view(torch.int16)) and torch.equal(a.v.view(torch.int16), b.v.view(torch.int16)), i


def test_captured_rounds_of_many_streams():
    """40 streams of e4m3 rows, counts in place, captured and replayed on a HIP stream that is not the default one."""
    announce("graph capture of attention rounds, 40 streams")
    args = dict(n=40, hq=8, hkv=2, d=256, page=16, e4m3=True, pages=300, blocks=12, rows=6, max_kv=180, rot=64, seed=34)
    a, b = Server(**args), Server(**args)
    side = torch.cuda.Stream()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    a.draw([6] * 40)
    b.draw([6] * 40)
    a.forward(), a.commit(), b.forward(), b.commit()
    torch.cuda.synchronize()
    for graph, part in zip(graphs, (a.forward, a.commit)):
        with torch.cuda.graph(graph):
            part()
    torch.cuda.synchronize()
    for i in range(6):
        lens = [(3 * s + 5 * i) % 7 for s in range(40)]
        a.draw(lens)
        b.draw(lens)
        if i == 3:
            a.kv_len[7:20] = -1                 # they end: their pages go to the others
            b.kv_len[7:20] = -1
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for graph in graphs:
                graph.replay()
            b.forward()
            b.commit()
        torch.cuda.synchronize()
        rs = a.row_start.cpu().tolist()
        for s in range(40):
            if a.kv_len[s].item() >= 0:
                out = a.out[rs[s]:rs[s + 1]]
                assert torch.equal(out, b.out[rs[s]:rs[s + 1]]) and not torch.isnan(out).any(), (i, s)
        for name in ("kv_len", "page_count", "free_count", "table", "slots", "positions", "ks", "vs"):
            assert torch.equal(torch.nan_to_num(getattr(a, name)), torch.nan_to_num(getattr(b, name))), (i, name)
        assert torch.equal(a.k.view(torch.uint8), b.k.view(torch.uint8)) and torch.equal(a.v.view(torch.uint8), b.v.view(torch.uint8)), i
        held = a.page_count.cpu().tolist()
        used = [int(x) for s in range(40) for x in a.table[s, :held[s]].tolist()] + a.free_pages[:a.free_count.item()].cpu().tolist()
        assert sorted(used) == list(range(300)), i


def test_two_streams_at_once():
    """Calls on two HIP streams, each with its own workspace, and on a stream that is not the default one."""
    announce("attention on two streams")
    a, b = Case([900, 2000], [5, 16], 6, 2, 128, 32, tree=True, seed=22), Case([1500], [1], 6, 2, 128, 64, seed=23)
    want = [a.run(), b.run()]
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    dev = []
    for c in (a, b):
        mk, mr = max(x + y for x, y in zip(c.lens, c.rows)), max(c.rows)
        dev.append(dict(row_start=c.row_start.cuda(), kv_len=c.kv_len.cuda(), block_table=c.table.cuda(), q=c.q.cuda(), k_cache=c.k.cuda(),
                        v_cache=c.v.cuda(), out=torch.zeros((c.total, c.hq, c.d), dtype=BF16, device="cuda"), max_kv=mk, max_rows=mr,
                        parent=None if c.parent is None else c.parent.cuda(),
                        workspace=torch.empty(gdn.attn_workspace_bytes(c.hq, c.hkv, c.d, len(c.lens), c.total, mr, mk), dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(20):
        for st, kw in zip(streams, dev):
            with torch.cuda.stream(st):
                gdn.attn_window(**kw)
    torch.cuda.synchronize()
    got = [kw["out"] for kw in dev]
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_window_rows_against_steps():
    """A chain window's rows against one-row steps over the same cache: the same values within twice their bound."""
    announce("window against steps")
    c = Case([333], [9], 6, 2, 128, 32, seed=24, gate=True)
    out, (want, bound) = c.run(), c.oracle()
    for t in range(9):
        one = Case.__new__(Case)
        one.__dict__.update(c.__dict__)
        one.lens, one.rows, one.row_start, one.total = [333 + t], [1], torch.tensor([0, 1], dtype=I32), 1
        one.kv_len, one.q, one.gate = torch.tensor([333 + t], dtype=I32), c.q[t:t + 1].contiguous(), c.gate[t:t + 1].contiguous()
        step = one.run()
        assert np.all(np.abs(f64(step[0]) - want[t]) <= bound[t])
        assert np.all(np.abs(f64(step[0]) - f64(out[t])) <= 2 * bound[t])
