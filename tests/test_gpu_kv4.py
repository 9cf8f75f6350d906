"""The 4-bit cache against the fp64 oracle: rows quantised as they are written,
attention of steps, windows and trees over them, commits, and cached rows of
every format read back."""
import numpy as np
import pytest
import torch

from oracle import attn as ref
from verify_causal_conv1d_amd import gdn
from verify_causal_conv1d_amd import inputs as gi

from gpu_util import announce
from test_gpu_prompt import BF16, FMTS, I32, U8, Case, close, cu, f64, i32, values

pytestmark = pytest.mark.gpu


class Windows(Case):
    """Steps, windows and trees over a 4-bit cache."""

    def __init__(self, lens, rows, hq, hkv, d, page, tree=False, fmt="mxfp4", **kw):
        super().__init__(lens, rows, hq, hkv, d, page, fmt=fmt, **kw)
        self.parent = gi.random_tree_parents(rows, self.g) if tree else None

    def run(self, max_kv=None, max_rows=None, out=None, table=None, row_start=None, kv_len=None, parent=None, scale=None):
        max_kv = max_kv or max(a + b for a, b in zip(self.lens, self.rows))
        max_rows = max_rows or max(max(self.rows), 1)
        out = torch.full((self.total, self.hq, self.d), float("nan"), dtype=BF16, device="cuda") if out is None else out
        ws = torch.full((gdn.attn_workspace_bytes(self.hq, self.hkv, self.d, len(self.lens), self.total, max_rows, max_kv),), 0xFF,
                        dtype=U8, device="cuda")
        gate = self.gate.cuda()[:, :, self.d:] if self.gate is not None else None
        pick = lambda a, b: cu(b if a is None else a)  # noqa: E731
        gdn.attn_window(pick(row_start, self.row_start), pick(kv_len, self.kv_len), pick(table, self.table), self.q.cuda(), cu(self.k),
                        cu(self.v), out, ws, max_kv=max_kv, max_rows=max_rows, parent=pick(parent, self.parent), gate=gate,
                        k_scale=cu(self.ks), v_scale=cu(self.vs), scale=scale)
        torch.cuda.synchronize()
        return out

    def oracle(self, scale=None):
        gate = None if self.gate is None else f64(self.gate[:, :, self.d:])
        out, mag, reach = ref.window(self.page, self.row_start.tolist(), None if self.parent is None else self.parent.tolist(),
                                     self.lens, self.table.numpy(), f64(self.q), values(self.k, self.ks),
                                     values(self.v, self.vs), ref.default_scale(self.d) if scale is None else scale, gate)
        return out, ref.window_bound(out, mag, reach, self.d) + self.underflow()


WINDOWS = [
    dict(lens=[0], rows=[1], hq=1, hkv=1, d=64, page=16),
    dict(lens=[0, 1, 15, 16, 17, 31, 32, 33], rows=[1] * 8, hq=4, hkv=2, d=64, page=16),
    dict(lens=[0, 1, 15, 16, 17, 31, 32, 33], rows=[1] * 8, hq=4, hkv=2, d=128, page=32, gate=True),
    dict(lens=[0, 63, 64, 65, 127, 128, 500], rows=[1] * 7, hq=6, hkv=1, d=256, page=64, gate=True),
    dict(lens=[14, 30, 62, 126, 127, 128, 129, 255], rows=[2, 3, 4, 3, 1, 2, 16, 1], hq=6, hkv=1, d=256, page=16, gate=True),
    dict(lens=[300, 40, 511, 700, 0, 383], rows=[16, 0, 7, 1, 16, 2], hq=6, hkv=2, d=128, page=64, tree=True),
    dict(lens=[520, 0, 17], rows=[16, 16, 5], hq=24, hkv=4, d=256, page=256, tree=True, gate=True),
    dict(lens=[200, 90], rows=[16, 16], hq=16, hkv=1, d=64, page=128, gate=True),
    dict(lens=[77], rows=[3], hq=40, hkv=2, d=128, page=32),
    dict(lens=[1000, 1500], rows=[9, 12], hq=8, hkv=8, d=64, page=32, tree=True),
    dict(lens=[2000, 5], rows=[4, 4], hq=8, hkv=2, d=256, page=32),
    dict(lens=[3000, 50, 1023], rows=[11, 5, 6], hq=9, hkv=3, d=128, page=128, gate=True),
    dict(lens=[16384 - 3, 3, 900], rows=[2, 1, 3], hq=2, hkv=1, d=64, page=256),
    dict(lens=[40001], rows=[1], hq=2, hkv=1, d=256, page=256),
    dict(lens=[33000, 17], rows=[16, 3], hq=6, hkv=1, d=128, page=128, tree=True),
    dict(lens=[40, 150], rows=[16, 1], hq=1024, hkv=1, d=64, page=16),
    dict(lens=[40, 150], rows=[9, 1], hq=1024, hkv=512, d=64, page=16),
]


@pytest.mark.parametrize("kw", WINDOWS, ids=range(len(WINDOWS)))
def test_windows_match_oracle(kw):
    announce(f"attention over 4 bits {kw}")
    c = Windows(seed=11, **kw)
    close(c.run(), *c.oracle())


def test_few_columns_keep_the_weights_bits():
    """Up to 16 columns weights count to 2^-15: the result is its own rounding away, and little more."""
    for d in (64, 128, 256):
        announce(f"weights over 4 bits, d {d}")
        c = Windows([700, 90], [1, 2], 6, 1, d, 32, seed=12)
        (want, bound), out = c.oracle(), f64(c.run())
        gate = None
        _, mag, reach = ref.window(c.page, c.row_start.tolist(), None, c.lens, c.table.numpy(), f64(c.q), values(c.k, c.ks),
                                   values(c.v, c.vs), ref.default_scale(d), gate)
        fine = 2.0 ** -8 * np.abs(want) + (2.0 ** -15 + 2.0 ** -18 + 2.0 * (d + 8) * 2.0 ** -24 * reach[..., None]) * 1.01 * mag + 1e-37
        assert np.all(np.abs(out - want) <= fine)


def test_scales_and_peaked_scores():
    announce("windows over 4 bits, peaked rows, given scales")
    for rows in ([1, 1], [9, 16]):
        c = Windows([500, 80], rows, 4, 2, 128, 32, seed=13, amp=30.0)
        close(c.run(), *c.oracle())
        for scale in (0.0, -0.02):
            close(c.run(scale=scale), *c.oracle(scale=scale))


def test_blocks_that_are_not_seen_change_nothing():
    for hq, d in ((1, 64), (1, 256), (6, 64), (6, 128), (6, 256)):        # 9 columns, and 54
        announce(f"unseen blocks, {hq} heads, d {d}")
        c = Windows([70, 130], [9, 9], 2 * hq, 2, d, 16, seed=14)
        c.parent = torch.tensor([-1, 0, 0, 2, 1, 3, 5, 4, 0] * 2, dtype=I32)
        clean = c.run()
        par = c.parent[:9].tolist()
        sees = [[u in ref.ancestors(par, t) for u in range(9)] for t in range(9)]
        for bad in (3, 0, 8):
            for pool, e in ((c.ks, 255), (c.vs, 255), (c.vs, 254), (c.ks, 253)):
                for st in range(2):
                    at = c.lens[st] + bad
                    page = int(c.table[st, at // 16])
                    keep = pool[page, :, at % 16].clone()
                    pool[page, :, at % 16] = e
                    got = c.run()
                    pool[page, :, at % 16] = keep
                    for t in range(18):
                        if t // 9 == st and sees[t % 9][bad]:
                            assert torch.isnan(got[t]).all(), (bad, e, st, t)
                        else:
                            assert torch.equal(got[t], clean[t]), (bad, e, st, t)


def test_cached_blocks_of_nan_reach_their_channels():
    """One block of a cached row's values: its 32 channels are NaN for every row of the stream, the others keep their bits."""
    for rows, key in ((1, 0), (1, 69), (9, 64), (9, 10), (9, 69)):
        announce(f"a NaN block at key {key}, {rows} rows")
        c = Windows([70, 333], [rows, rows], 6, 2, 128, 16, seed=30)
        clean = c.run()
        page = int(c.table[0, key // 16])
        c.vs[page, :, key % 16, 2] = 255
        got = c.run()
        hit = torch.zeros_like(got, dtype=torch.bool)
        hit[:rows, :, 64:96] = True
        assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], clean[~hit])


def test_streams_do_not_depend_on_each_other():
    for hq in (2, 12):
        for tree in (False, True):
            announce(f"windows over 4 bits, batch against single streams, {hq} heads, tree {tree}")
            lens, rows = [700, 3, 5000, 130], [5, 8, 7, 1]
            c = Windows(lens, rows, hq, 2, 128, 32, tree=tree, seed=15)
            whole = c.run(max_rows=8)
            assert torch.equal(whole, c.run(max_rows=8, max_kv=1 << 20))
            for s in range(4):
                a, b = int(c.row_start[s]), int(c.row_start[s + 1])
                one = Windows.__new__(Windows)
                one.__dict__.update(c.__dict__)
                one.lens, one.rows, one.row_start, one.total = [lens[s]], [rows[s]], torch.tensor([0, b - a], dtype=I32), b - a
                one.table, one.kv_len, one.q = c.table[s:s + 1].contiguous(), c.kv_len[s:s + 1], c.q[a:b].contiguous()
                one.parent = None if c.parent is None else c.parent[a:b].contiguous()
                assert torch.equal(one.run(max_rows=8), whole[a:b]), s


@pytest.mark.parametrize("hq,tree", [(2, False), (2, True), (16, False), (16, True)])
def test_broken_streams_are_skipped(hq, tree):
    c = Windows([300, 70, 900, 40], [4, 4, 4, 4], hq, 2, 128, 16, tree=tree, seed=16)
    good = c.run()
    announce(f"skipped streams over 4 bits, {hq} heads, tree {tree}")

    def same_but(got, streams):
        for s in range(4):
            a, b = 4 * s, 4 * s + 4
            if s in streams:
                assert torch.isnan(got[a:b]).all(), s
            else:
                assert torch.equal(got[a:b], good[a:b]), s
    for s, j in ((0, 3), (1, 0), (2, 56), (3, 2)):
        for page in (-1, c.pages, 1 << 30):
            t = c.table.clone()
            t[s, j] = page
            same_but(c.run(table=t), {s})
    for value in (-1, 10 ** 6, 2 ** 31 - 1):
        kv = c.kv_len.clone()
        kv[1] = value
        same_but(c.run(kv_len=kv), {1})
    same_but(c.run(max_kv=500), {2})
    for value in (17, -5):
        rs = c.row_start.clone()
        rs[4] = value
        same_but(c.run(row_start=rs), {3})
    if tree:
        for bad in (2, -2, 9):
            p = c.parent.clone()
            p[6] = bad
            same_but(c.run(parent=p), {1})


def test_many_streams():
    g = torch.Generator().manual_seed(25)
    lens = torch.randint(0, 1400, (70,), generator=g).tolist()
    for rows, hq, tree in (([1] * 70, 16, False), ([1 + i % 3 for i in range(70)], 32, True), ([(5 * i) % 9 for i in range(70)], 16, True)):
        announce(f"70 streams over 4 bits, up to {max(rows)} rows, {hq} heads")
        c = Windows(lens, rows, hq, 4, 64, 32, tree=tree, seed=26, spare=9)
        close(c.run(), *c.oracle())


def test_parts_of_many_bytes():
    """More than 16 MB of parts, which the join asks for once it knows each stream's chunks: one to seven of them."""
    announce("24 trees over 4 bits, 19 MB of parts")
    lens = [3 + 137 * s for s in range(24)]
    c = Windows(lens, [16 - s % 3 for s in range(24)], 16, 1, 128, 64, tree=True, gate=True, seed=27)
    close(c.run(), *c.oracle())


def test_offsets_past_32_bits():
    announce("windows and a commit over 4 bits, 5 GiB pools")
    pages = (5 << 30) // (2 * 64 * 128)
    for rows in ([1, 1], [3, 9]):
        c = Windows([130, 700], rows, 12, 2, 256, 64, seed=17)
        want, first = c.run(), pages - c.pages
        k, v = (torch.empty((pages, 2, 64, 128), dtype=U8, device="cuda") for _ in "kv")
        ks, vs = (torch.empty((pages, 2, 64, 8), dtype=U8, device="cuda") for _ in "kv")
        k[first:], v[first:], ks[first:], vs[first:] = c.k.cuda(), c.v.cuda(), c.ks.cuda(), c.vs.cuda()
        table = torch.where(c.table >= 0, c.table + first, c.table).cuda()
        out = torch.zeros_like(want)
        ws = torch.empty(gdn.attn_workspace_bytes(12, 2, 256, 2, c.total, max(rows), 709), dtype=U8, device="cuda")
        gdn.attn_window(c.row_start.cuda(), c.kv_len.cuda(), table, c.q.cuda(), k, v, out, ws, max_kv=709, max_rows=max(rows), k_scale=ks,
                        v_scale=vs)
        assert torch.equal(out, want)
    slots = i32([(pages - 1) * 64 + 63])
    x = torch.randn((1, 2, 256), device="cuda").to(BF16)
    gdn.attn_prep(torch.zeros((1, 4, 256), dtype=BF16, device="cuda"), x, x, None, None, torch.zeros(0, device="cuda"), i32([0]), slots,
                  torch.zeros((1, 4, 256), dtype=BF16, device="cuda"), k, v, ks, vs)
    codes, exps = ref.mx_quantise(f64(x)[0])
    length = i32([62])
    gdn.attn_commit(i32([0, 2]), i32([1]), length, i32([[pages - 1]]), k, v, k_scale=ks, v_scale=vs, parent=i32([-1, -1]))
    torch.cuda.synchronize()
    for at in (63, 62):
        for p, e in ((k, ks), (v, vs)):
            assert np.array_equal(p[pages - 1, :, at].cpu().numpy(), codes) and np.array_equal(e[pages - 1, :, at].cpu().numpy(), exps)
    assert length.item() == 63


# ---- rows quantised as they are written -------------------------------------------

@pytest.mark.parametrize("R,hq,hkv,d,rot,page,inter,norm", [
    (1, 1, 1, 64, 0, 16, False, True), (5, 4, 2, 64, 64, 16, False, True), (5, 4, 2, 64, 64, 16, True, True),
    (33, 24, 4, 256, 64, 64, False, True), (33, 24, 4, 256, 64, 64, True, False), (7, 6, 2, 128, 50, 32, False, True),
    (7, 3, 3, 128, 2, 256, True, False), (7, 9, 3, 128, 126, 128, False, True), (64, 8, 1, 256, 256, 16, False, True),
    (64, 7, 7, 256, 256, 16, True, True), (300, 2, 1, 64, 22, 16, True, True), (700, 3, 3, 128, 128, 64, False, False),
    (700, 3, 3, 64, 20, 64, False, True), (601, 4, 1, 256, 2, 16, True, True), (520, 2, 2, 128, 126, 32, False, True),
    (513, 1, 1, 64, 0, 16, False, True), (900, 20, 5, 64, 60, 16, True, True)])
def test_prep_writes_the_oracles_codes(R, hq, hkv, d, rot, page, inter, norm):
    """Every code and every exponent, of keys and of values."""
    announce(f"prep into 4 bits, rows {R} heads {hq}/{hkv} d {d} rot {rot} page {page} interleaved {inter} norm {norm}")
    g = torch.Generator().manual_seed(R + d + rot)
    x = (torch.randn((R, (2 * hq + 2 * hkv) * d + 8), generator=g) * 3).to(BF16)
    x[R // 2] = 0
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
    if R > 3:
        slots[R // 3], slots[R // 3 + 1] = -1, pages * page
    kc, vc = (torch.full((pages, hkv, page, d // 2), 0x5A, dtype=U8, device="cuda") for _ in "kv")
    ks, vs = (torch.full((pages, hkv, page, d // 32), 99, dtype=U8, device="cuda") for _ in "kv")
    qo = torch.full((R, hq, d), float("nan"), dtype=BF16, device="cuda")
    rs, eps = (1.25, 2.0 ** -17) if inter else (1.0, 2.0 ** -20)
    gdn.attn_prep(q, k, v, *[cu(t) for t in w], freq.cuda(), pos.cuda(), slots.cuda(), qo, kc, vc, ks, vs, eps=eps, interleaved=inter,
                  rot_scale=rs)
    torch.cuda.synchronize()

    def want(t, weight):
        n = ref.normed(f64(t), None if weight is None else weight.double().numpy(), eps)
        return ref.rotated(n, pos.numpy(), freq.double().numpy(), inter, rs)
    y, mag = want(q, w[0])
    assert np.all(np.abs(f64(qo) - y) <= 2.0 ** -8 * np.abs(y) + 2.0 ** -19 * mag + 1e-38)
    for pool, exps, y in ((kc, ks, want(k, w[1])[0]), (vc, vs, f64(v))):
        codes, e = ref.mx_quantise(y)
        wc, we = (np.full(t.shape, fill, np.uint8) for t, fill in ((pool, 0x5A), (exps, 99)))
        for r in range(R):
            s = int(slots[r])
            if 0 <= s < pages * page:
                wc[s // page, :, s % page], we[s // page, :, s % page] = codes[r], e[r]
        assert np.array_equal(exps.cpu().numpy(), we)
        got = pool.cpu().numpy()
        # a value of 0 may have either sign (0 * -1 in one order of the rotation's terms)
        plain = lambda c: np.stack([np.where((c & 7) == 0, 0, c & 15), np.where((c >> 4 & 7) == 0, 0, c >> 4)])  # noqa: E731
        assert np.array_equal(plain(got), plain(wc))


def test_blocks_at_the_ends_of_the_range():
    """Ties, zeros, tiny and huge values, infinities and NaN: as the oracle quantises them, and read back as it reads them."""
    announce("4-bit blocks at the ends of the range")
    d, R = 64, 12
    x = torch.zeros((R, 1, d))
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    x[1, 0, :8], x[1, 0, 8:16] = ties, -ties
    x[1, 0, 32:40] = ties * 2.0 ** 90
    x[2, 0, 0], x[2, 0, 1] = 7.0, 3.5                                     # the first that goes a power of two up
    x[2, 0, 32], x[2, 0, 33] = 6.96875, 5.03125
    x[3] = torch.randn((1, d), generator=torch.Generator().manual_seed(1)) * 2.0 ** -126
    x[4, 0, 5], x[4, 0, 6] = 3.3e38, -1e30
    x[5, 0, 5] = float("inf")
    x[6, 0, 40] = float("nan")
    x[7, 0, 5], x[7, 0, 6] = float("-inf"), float("nan")
    x[8, 0, 1], x[8, 0, 2] = 2.0 ** -101, -2.0 ** -103
    x[9, 0, :] = -0.0
    x[10, 0, 3], x[10, 0, 35] = 1.7e38, 1.6e38
    x[11] = torch.randn((1, d), generator=torch.Generator().manual_seed(2)) * torch.logspace(-20, 20, d)
    x = x.to(BF16).cuda()
    kc, vc = (torch.zeros((1, 1, 16, d // 2), dtype=U8, device="cuda") for _ in "kv")
    ks, vs = (torch.zeros((1, 1, 16, 2), dtype=U8, device="cuda") for _ in "kv")
    qo = torch.zeros((R, 1, d), dtype=BF16, device="cuda")
    gdn.attn_prep(x, x, x, None, None, torch.zeros(0, device="cuda"), i32([0] * R), i32(list(range(R))), qo, kc, vc, ks, vs)
    codes, exps = ref.mx_quantise(f64(x.float()))
    ko, vo = (torch.zeros((R, 1, d), dtype=BF16, device="cuda") for _ in "kv")
    gdn.kv_read(i32([0, R]), i32([0]), i32([[0]]), kc, vc, ko, vo, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    for p, e, out in ((kc, ks, ko), (vc, vs, vo)):
        assert np.array_equal(e[0, 0, :R].cpu().numpy(), exps[:, 0])
        assert np.array_equal(p[0, 0, :R].cpu().numpy(), codes[:, 0])
        assert np.array_equal(f64(out), ref.mx_values(codes, exps), equal_nan=True)


def test_every_code_under_every_exponent():
    announce("all 4-bit codes under all exponents")
    e = torch.arange(256, dtype=U8).view(16, 1, 16, 1).expand(16, 1, 16, 2).contiguous().cuda()
    k = torch.arange(256, dtype=U8).view(8, 32)
    ko, vo = (torch.zeros((256, 1, 64), dtype=BF16, device="cuda") for _ in "kv")
    table = torch.arange(16, dtype=I32).view(1, 16).cuda()
    for i in range(0, 8, 2):
        kc, vc = (k[i + j].view(1, 1, 1, 32).expand(16, 1, 16, 32).contiguous().cuda() for j in (0, 1))
        gdn.kv_read(i32([0, 256]), i32([0]), table, kc, vc, ko, vo, k_scale=e, v_scale=e)
        torch.cuda.synchronize()
        for pool, out in ((kc, ko), (vc, vo)):
            want = ref.mx_values(pool.cpu().numpy(), e.cpu().numpy()).reshape(256, 1, 64)
            # exponents from 2^-126 on: all of a block's values are normal or 0
            assert np.array_equal(f64(out)[2:], want[2:], equal_nan=True)


def test_the_least_exponent_reads_exactly():
    """Under e = 1 the code of 0.5 is 2^-127, below the least normal number and a bf16 number all the same."""
    announce("4-bit codes under the least exponent")
    e = torch.ones((1, 1, 16, 2), dtype=U8, device="cuda")
    k = torch.arange(256, dtype=U8).view(1, 1, 8, 32)
    kc, vc = (torch.cat([x, x], 2).cuda() for x in (k, k.flip(3)))
    ko, vo = (torch.zeros((16, 1, 64), dtype=BF16, device="cuda") for _ in "kv")
    gdn.kv_read(i32([0, 16]), i32([0]), i32([[0]]), kc, vc, ko, vo, k_scale=e, v_scale=e)
    torch.cuda.synchronize()
    for pool, out in ((kc, ko), (vc, vo)):
        assert np.array_equal(f64(out)[:, 0], ref.mx_values(pool.cpu().numpy(), e.cpu().numpy())[0, 0])


@pytest.mark.parametrize("d", [64, 128, 256])
def test_keys_under_the_least_exponent(d):
    """Keys of 0 and +-2^-127 only, and queries large enough that they decide the weights."""
    for kind, rows, hq in ((Windows, [1, 2], 4), (Windows, [9, 16], 12), (Case, [40, 3], 6)):
        announce(f"keys of 2^-127, d {d}, rows {rows}")
        c = kind([70, 333], rows, hq, 2, d, 16, fmt="mxfp4", seed=41)
        code = torch.tensor([0x0, 0x1, 0x9])[torch.randint(0, 3, (*c.k.shape[:3], d), generator=c.g)]
        c.k = (code[..., 0::2] | code[..., 1::2] << 4).to(U8)
        c.ks = torch.where(c.ks == 255, 255, 1).to(U8)
        c.q = (torch.randn(c.q.shape, generator=c.g).clamp(-3.5, 3.5) * 2.0 ** 125).to(BF16)
        scale = 8.0 * d ** -0.5
        want, bound = c.oracle(scale=scale)
        close(c.run(scale=scale), want, bound)
        c.q = torch.zeros_like(c.q)           # and not within the bound of what they are without them
        flat, _ = c.oracle(scale=scale)
        assert (np.abs(want - flat) > 2 * bound).mean() > 0.5


# ---- commits -----------------------------------------------------------------------

def test_commit_moves_rows_and_exponents():
    for d, page in ((64, 16), (128, 64), (256, 32)):
        announce(f"commit over 4 bits, d {d}")
        lens, rows = [30, 7, 500, 0, 64], [16, 5, 9, 3, 1]
        c = Windows(lens, rows, 4, 2, d, page, tree=True, seed=19)
        rs, par = c.row_start.tolist(), c.parent.tolist()
        accept = [rs[0] + 13, rs[1] + 4, -1, rs[3] + 2, rs[4]]
        pools = [t.cuda() for t in (c.k, c.v, c.ks, c.vs)]
        out = i32([-9] * 5)
        gdn.attn_commit(c.row_start.cuda(), i32(accept), c.kv_len.cuda(), c.table.cuda(), *pools[:2], k_scale=pools[2], v_scale=pools[3],
                        parent=c.parent.cuda(), kv_len_out=out)
        torch.cuda.synchronize()
        want, length = ref.commit(page, rs, par, accept, lens, c.table.numpy(), *(t.numpy() for t in (c.k, c.v, c.ks, c.vs)))
        for got, w in zip(pools, want):
            assert np.array_equal(got.cpu().numpy(), w)
        assert out.tolist() == length.tolist()


# ---- cached rows read back ---------------------------------------------------------

@pytest.mark.parametrize("fmt", FMTS)
def test_read_matches_oracle(fmt):
    for lens, rows, hkv, d, page, gap in (([0], [1], 1, 64, 16, 0), ([3, 0, 77, 500, 16], [40, 1, 0, 123, 16], 2, 128, 16, 3),
                                          ([5, 600], [1000, 17], 3, 256, 256, 0), ([9] * 150, [1 + i % 5 for i in range(150)], 1, 64, 32, 2)):
        announce(f"read {lens[:5]} {rows[:5]} {hkv} heads d {d} page {page} {fmt}")
        c = Case(lens, rows, hkv, hkv, d, page, fmt=fmt, seed=20, gap=gap)
        ko, vo = (torch.full((c.total, hkv, d), 7.0, dtype=BF16, device="cuda") for _ in "kv")
        gdn.kv_read(c.row_start.cuda(), c.kv_len.cuda(), c.table.cuda(), cu(c.k), cu(c.v), ko, vo, k_scale=cu(c.ks), v_scale=cu(c.vs))
        torch.cuda.synchronize()
        for out, pool, scale in ((ko, c.k, c.ks), (vo, c.v, c.vs)):
            want = ref.read(page, c.row_start.tolist(), lens, c.table.numpy(), values(pool, scale), np.full((c.total, hkv, d), 7.0))
            if fmt == "e4m3":       # the fp32 product (2^-24), then bf16 (2^-8)
                assert np.all(np.abs(f64(out) - want) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(want))
            else:
                assert np.array_equal(f64(out), want)


def test_read_leaves_out_what_is_broken():
    announce("read, broken layouts")
    c = Case([30, 5, 100], [20, 7, 40], 2, 2, 64, 16, seed=21)
    args = dict(row_start=c.row_start, first=c.kv_len, block_table=c.table)

    def read(**kw):
        ko, vo = (torch.full((c.total, 2, 64), 7.0, dtype=BF16, device="cuda") for _ in "kv")
        a = {k: kw.get(k, v).cuda() for k, v in args.items()}
        gdn.kv_read(a["row_start"], a["first"], a["block_table"], c.k.cuda(), c.v.cuda(), ko, vo)
        torch.cuda.synchronize()
        return ko, vo
    good = read()

    def same_but(got, rows):
        keep = torch.ones(c.total, dtype=torch.bool)
        keep[rows] = False
        for a, b in zip(got, good):
            assert torch.equal(a[keep], b[keep]) and (a[~keep] == 7.0).all()
    for bad in (-1, c.pages, 1 << 30):
        t = c.table.clone()
        t[0, 2] = bad                               # cache rows 32 .. 47: packed rows 2 .. 17
        same_but(read(block_table=t), list(range(2, 18)))
    for bad in (-1, 2 ** 31 - 1, 16 * c.table.shape[1]):
        f = c.kv_len.clone()
        f[1] = bad
        same_but(read(first=f), list(range(20, 27)))
    for bad in (-5, c.total + 1, 2 ** 31 - 1):
        rs = c.row_start.clone()
        rs[3] = bad
        same_but(read(row_start=rs), list(range(27, 67)))
    rs = c.row_start.clone()
    rs[3] = 50
    same_but(read(row_start=rs), list(range(50, 67)))


def test_rows_come_back_bit_for_bit():
    """Read from a bf16 cache and written again, without norm and rotation, rows are the same bits; read
    from a 4-bit cache and written again, the same codes and exponents."""
    for fmt in ("bf16", "mxfp4"):
        announce(f"read and written again, {fmt}")
        c = Case([0, 33], [100, 60], 2, 2, 128, 16, fmt=fmt, seed=22)
        ko, vo = (torch.zeros((160, 2, 128), dtype=BF16, device="cuda") for _ in "kv")
        k, v, ks, vs = cu(c.k), cu(c.v), cu(c.ks), cu(c.vs)
        gdn.kv_read(c.row_start.cuda(), c.kv_len.cuda(), c.table.cuda(), k, v, ko, vo, k_scale=ks, v_scale=vs)
        slots = torch.cat([torch.tensor([int(c.table[s, (c.lens[s] + t) // 16]) * 16 + (c.lens[s] + t) % 16 for t in range(c.rows[s])])
                           for s in range(2)]).to(I32).cuda()
        again = [t if t is None else t.clone() for t in (k, v, ks, vs)]
        for t in again:
            if t is not None:
                t.view(U8)[c.table[0, :6].long()] = 1            # whole pages of the first stream
        q = torch.zeros((160, 2, 128), dtype=BF16, device="cuda")
        gdn.attn_prep(q, ko, vo, None, None, torch.zeros(0, device="cuda"), i32([0] * 160), slots, q.clone(), *again)
        torch.cuda.synchronize()
        for a, b in zip(again, (k, v, ks, vs)):
            if a is not None:
                assert torch.equal(a.view(U8), b.view(U8))


# ---- rounds ---------------------------------------------------------------------------

@pytest.mark.parametrize("hq", [2, 12])
def test_captured_rounds_of_trees(hq):
    """A prompt pass, then verify rounds (tables, prep, attention of trees, commit) over a 4-bit cache, captured
    once and replayed with the streams' own lengths: each round against the oracle and the eager run."""
    announce(f"captured rounds over 4 bits, {hq} heads")
    g = torch.Generator().manual_seed(60)
    n, hkv, d, page, pages, blocks, m = 4, 2, 128, 16, 120, 24, 8
    rows = [8, 3, 5, 1]
    total = sum(rows)
    freq = (1e4 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float().cuda()
    w = torch.ones(d, device="cuda")
    lens = [40, 100, 0, 17]
    parent = gi.random_tree_parents(rows, g)

    def state():
        s = dict(row_start=gi.starts_from_lengths(rows).cuda(), parent=parent.cuda(), kv_len=i32(lens), free_count=i32([pages]),
                 page_count=i32([0] * n), free_pages=torch.arange(pages, dtype=I32, device="cuda"), accept=i32([-1] * n),
                 block_table=torch.full((n, blocks), -1, dtype=I32, device="cuda"), slots=i32([-1] * total), positions=i32([0] * total))
        s["x"] = torch.zeros((total, (hq + 2 * hkv) * d), dtype=BF16, device="cuda")
        s["k"], s["v"] = (torch.zeros((pages, hkv, page, d // 2), dtype=U8, device="cuda") for _ in "kv")
        s["ks"], s["vs"] = (torch.full((pages, hkv, page, d // 32), 127, dtype=U8, device="cuda") for _ in "kv")
        s["qo"], s["out"] = (torch.zeros((total, hq, d), dtype=BF16, device="cuda") for _ in "qo")
        s["ws"] = torch.zeros(gdn.attn_workspace_bytes(hq, hkv, d, n, total, m, 300), dtype=U8, device="cuda")
        return s

    def heads(s, x):
        t = x.shape[0]
        return x[:, :hq * d].view(t, hq, d), x[:, hq * d:(hq + hkv) * d].view(t, hkv, d), x[:, (hq + hkv) * d:].view(t, hkv, d)

    def round_(s):
        gdn.kv_tables(s["row_start"], s["kv_len"], s["page_count"], s["free_count"], s["free_pages"], s["block_table"], s["slots"],
                      s["positions"], page_size=page, parent=s["parent"])
        gdn.attn_prep(*heads(s, s["x"]), w, w, freq, s["positions"], s["slots"], s["qo"], s["k"], s["v"], s["ks"], s["vs"])
        gdn.attn_window(s["row_start"], s["kv_len"], s["block_table"], s["qo"], s["k"], s["v"], s["out"], s["ws"], max_kv=300, max_rows=m,
                        parent=s["parent"], k_scale=s["ks"], v_scale=s["vs"])
        gdn.attn_commit(s["row_start"], s["accept"], s["kv_len"], s["block_table"], s["k"], s["v"], k_scale=s["ks"], v_scale=s["vs"],
                        parent=s["parent"], max_rows=m)

    a, b = state(), state()
    # the streams' first rows, by a prompt pass of their own
    px = torch.randn((sum(lens), (hq + 2 * hkv) * d), generator=g).to(BF16).cuda()
    for s in (a, b):
        rs, zero = gi.starts_from_lengths(lens).cuda(), i32([0] * n)
        slots, positions = i32([-1] * sum(lens)), i32([0] * sum(lens))
        gdn.kv_tables(rs, zero, s["page_count"], s["free_count"], s["free_pages"], s["block_table"], slots, positions, page_size=page)
        qo = torch.zeros((sum(lens), hq, d), dtype=BF16, device="cuda")
        gdn.attn_prep(*heads(s, px), w, w, freq, positions, slots, qo, s["k"], s["v"], s["ks"], s["vs"])
        gdn.attn_prompt(rs, zero, s["block_table"], qo, s["k"], s["v"], qo.clone(), None, max_kv=max(lens), k_scale=s["ks"], v_scale=s["vs"])
    round_(state())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        round_(a)
    for step in range(5):
        x = torch.randn((total, (hq + 2 * hkv) * d), generator=g).to(BF16)
        accept = [int(gi.starts_from_lengths(rows)[s]) + int(torch.randint(0, rows[s], (1,), generator=g)) for s in range(n)]
        if step == 2:
            accept[1] = -1
        for s in (a, b):
            s["x"].copy_(x)
            s["accept"].copy_(torch.tensor(accept, dtype=I32))
        torch.cuda.synchronize()
        before = b["kv_len"].tolist()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            graph.replay()
        # the window's result against the oracle, from the cache before the commit
        gdn.kv_tables(b["row_start"], b["kv_len"], b["page_count"], b["free_count"], b["free_pages"], b["block_table"], b["slots"],
                      b["positions"], page_size=page, parent=b["parent"])
        gdn.attn_prep(*heads(b, b["x"]), w, w, freq, b["positions"], b["slots"], b["qo"], b["k"], b["v"], b["ks"], b["vs"])
        kv = [values(b[p].cpu(), b[p + "s"].cpu()) for p in "kv"]
        out, mag, reach = ref.window(page, gi.starts_from_lengths(rows).tolist(), parent.tolist(), before, b["block_table"].cpu().numpy(),
                                     f64(b["qo"]), *kv, ref.default_scale(d))
        round_(b)                   # tables and prep again change nothing: the same pages, the same rows
        torch.cuda.synchronize()
        close(b["out"], out, ref.window_bound(out, mag, reach, d), f"round {step}")
        for name in ("out", "k", "v", "ks", "vs", "kv_len", "block_table", "slots", "page_count", "free_count"):
            assert torch.equal(a[name].view(U8), b[name].view(U8)), (step, name)
        depth = [len(ref.ancestors(ref.local_parents(gi.starts_from_lengths(rows).tolist(), parent.tolist(), s),
                                   accept[s] - int(gi.starts_from_lengths(rows)[s]))) if accept[s] >= 0 else 0 for s in range(n)]
        assert b["kv_len"].tolist() == [p + k for p, k in zip(before, depth)]
