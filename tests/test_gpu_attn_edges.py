"""The attention-layer calls where they can go wrong together or at the ends of
their ranges: pools that run out, long wide windows, prompts, extreme values,
broken layouts."""
import numpy as np
import pytest
import torch

from oracle import attn as ref
from verify_causal_conv1d_amd import gdn

from gpu_util import announce
from test_gpu_attn import BF16, F8, I32, Case, Server, check_tables, close, f64, i32, run_tables, tables_case, values
from test_gpu_attn import test_prep_matches_oracle as prep_matches_oracle

pytestmark = pytest.mark.gpu


# ---- pools that run out -----------------------------------------------------------

def bits(t):
    return t.view(torch.uint8).cpu()


def test_tables_of_a_stream_without_pages_name_no_page():
    """Entries that an unserved stream asked for and that still name a page become -1; others stay."""
    announce("tables, unserved streams with page numbers of earlier rounds")
    for n, tree in ((7, True), (16, False), (90, False)):
        for seed in range(3):
            c = tables_case(n, 16, 40 + seed, tree=tree, free=2)
            g = np.random.default_rng(seed)
            table, have = c["block_table"], c["page_count"]
            pool, blocks = c["free_pages"].shape[0], table.shape[1]
            # every stream grows by a page or more, where its table has room
            c["kv_len"] = np.minimum(np.maximum(c["kv_len"], 16 * have), 16 * blocks - 16).astype(np.int32)
            for s in range(n):      # what lies past a stream's pages: anything, of the pool and not
                past = table[s, have[s]:]
                past[:] = np.where(g.random(past.shape) < 0.7, g.integers(0, pool, past.shape), pool + 5)
            check_tables(c, 16)
            want = ref.tables(16, c["row_start"], c["parent"], c["kv_len"], have, 2, c["free_pages"], table, c["slots"], c["positions"])
            assert (want["block_table"] == -1).any()


@pytest.mark.parametrize("n", [3, 40])
def test_a_finished_stream_with_more_rows_than_its_table_holds(n):
    """It needs no room for them, and gives its pages back."""
    announce(f"tables of {n} streams, a finished one with many packed rows")
    c = tables_case(n, 16, 50, free=100)
    blocks, rows = c["block_table"].shape[1], np.diff(c["row_start"])
    c["kv_len"] = np.maximum(c["kv_len"], 0)
    c["kv_len"][1], rows[1] = -1, 16 * blocks + 1
    c["row_start"] = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    c["slots"], c["positions"] = (np.full(int(c["row_start"][-1]), -9, np.int32) for _ in range(2))
    assert c["page_count"][1] > 0
    check_tables(c, 16)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("e4m3,hq", [(False, 2), (True, 6), (False, 6)])
def test_a_round_in_which_the_pool_is_empty(captured, e4m3, hq):
    """A stream that gets no page: its results, rows and length stay, and no other
    stream's page is read or written for it, although its table still holds the
    number of a page that it gave back and another stream took."""
    announce(f"a round without pages, e4m3 {e4m3}, {hq} heads over 2, captured {captured}")
    sv = Server(3, hq, 2, 128, 16, e4m3, 4, 3, 12, 48, 32, seed=41)
    side, graphs = torch.cuda.Stream(), None

    def go(part):
        if graphs is None:
            part()
        else:
            with torch.cuda.stream(side):
                graphs[part.__name__].replay()
        torch.cuda.synchronize()

    def setup(lens, parents, accept):
        """Windows of these lengths; a stream's parents (None: a chain) and accepted local row."""
        R = sv.draw(lens)
        starts = sv.row_start.cpu().tolist()
        parent = sv.parent.cpu()
        for s, p in enumerate(parents):
            parent[starts[s]:starts[s + 1]] = torch.tensor(range(-1, lens[s] - 1) if p is None else p, dtype=I32)
        sv.parent.copy_(parent)
        sv.accept.copy_(torch.tensor([-1 if a is None else starts[s] + a for s, a in enumerate(accept)], dtype=I32))
        sv.out.fill_(float("nan"))
        return R, starts

    setup([12, 12, 12], [None] * 3, [11, 11, 0])
    go(sv.forward), go(sv.commit)
    if captured:
        graphs = {}
        sv.accept.fill_(-1)
        for part in (sv.forward, sv.commit):
            graphs[part.__name__] = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graphs[part.__name__]):
                part()
    assert sv.kv_len.tolist() == [12, 12, 1] and sv.free_count.item() == 1
    setup([12, 0, 0], [None] * 3, [None] * 3)               # the first stream takes the last page and keeps no row
    go(sv.forward), go(sv.commit)
    given = sv.table[0, 1].item()
    assert sv.kv_len.tolist() == [12, 12, 1] and sv.free_count.item() == 0
    setup([1, 12, 0], [None] * 3, [0, 11, None])            # it gives the page back, and the second stream takes it
    go(sv.forward), go(sv.commit)
    assert sv.kv_len.tolist() == [13, 24, 1] and sv.table[1, 1].item() == given and sv.page_count.tolist() == [1, 2, 1]

    tree = [-1, 0, 0, 2, 3, 4, 5, 6, 7, 8, 9, 10]
    for last in (11, 0):                                    # its path: rows past the page that it holds, or one within it
        R, rs = setup([12, 4, 3], [tree, None, None], [last, None, None])
        before = [t.clone() for t in (sv.k, sv.v, sv.ks, sv.vs) if t is not None]
        go(sv.forward)
        assert (sv.slots[:12] == -1).all() and (sv.slots[12:R] >= 0).all()
        assert sv.table[0, 1].item() == -1 and sv.page_count.tolist() == [1, 2, 1] and sv.free_count.item() == 0
        assert torch.isnan(sv.out[:12]).all() and torch.isnan(sv.out[R:]).all()
        # the others: against the oracle over the cache's own values
        kv, table = sv.kv_len.cpu().tolist(), sv.table.cpu().numpy()
        x = f64(sv.x)
        o, m, reach = ref.window(16, [0, 4, 7], None, kv[1:], table[1:], f64(sv.q)[12:R], values(sv.k, sv.ks), values(sv.v, sv.vs),
                                 128 ** -0.5, x[12:R, hq:2 * hq])
        close(sv.out[12:R], o, ref.window_bound(o, m, reach, 128))
        after = [t.clone() for t in (sv.k, sv.v, sv.ks, sv.vs) if t is not None]
        go(sv.commit)
        assert sv.kv_len.tolist() == [13, 24, 1]
        slots = sv.slots[12:R].long().cpu()
        for t, mid, old in zip((t for t in (sv.k, sv.v, sv.ks, sv.vs) if t is not None), after, before):
            assert torch.equal(bits(t), bits(mid))          # the commit moved nothing
            now, was = (y.view(torch.uint8 if y.dtype == F8 else torch.int16 if y.dtype == BF16 else I32).cpu() for y in (t, old))
            keep = torch.ones(4 * 16, dtype=torch.bool)     # cache rows that the two streams did not store
            keep[slots] = False
            assert torch.equal(now.transpose(1, 2).flatten(0, 1)[keep], was.transpose(1, 2).flatten(0, 1)[keep])

    sv.kv_len[1] = -1                                       # the second stream ends: the first is served again
    R, rs = setup([12, 0, 3], [tree, None, None], [11, None, None])
    go(sv.forward)
    assert (sv.slots[:R] >= 0).all() and sv.page_count.tolist() == [2, 0, 1] and not torch.isnan(sv.out[:R]).any()
    go(sv.commit)
    assert sv.kv_len.tolist() == [13 + 11, -1, 1]
    held = sv.page_count.tolist()
    used = [int(p) for s in range(3) for p in sv.table[s, :held[s]].tolist()] + sv.free_pages[:sv.free_count.item()].tolist()
    assert sorted(used) == list(range(4))


# ---- precision ------------------------------------------------------------------------

@pytest.mark.parametrize("kw", [
    dict(lens=[0, 5, 300, 700], rows=[1, 1, 1, 1], hq=8, hkv=2, d=256, page=64, gate=True),
    dict(lens=[17, 640], rows=[1, 1], hq=32, hkv=2, d=128, page=16, amp=6.0),
    dict(lens=[0, 5, 300, 700], rows=[1, 1, 1, 1], hq=8, hkv=2, d=256, page=64, e4m3=True),
    dict(lens=[260, 31], rows=[4, 3], hq=8, hkv=2, d=64, page=32, e4m3=True, tree=True, gate=True),
    dict(lens=[500, 3], rows=[8, 5], hq=4, hkv=2, d=128, page=32, tree=True)], ids=range(5))
def test_weights_of_few_columns_keep_more_than_bf16(kw):
    """Up to 16 columns: the only rounding to bf16 is the result's own."""
    announce(f"precision of the weights {kw}")
    c = Case(seed=44, **kw)
    gate = None if c.gate is None else f64(c.gate[:, :, c.d:])
    want, mag, reach = ref.window(c.page, c.row_start.tolist(), None if c.parent is None else c.parent.tolist(), c.lens, c.table.numpy(),
                                  f64(c.q), values(c.k, c.ks), values(c.v, c.vs), ref.default_scale(c.d), gate)
    # half a bf16 step of the result; of the terms 2^-15 from the weights' two bf16 parts (what the first
    # leaves, less than 2^-7 of the weight, is off by 2^-8 of itself), 2^-24 for each addition of a key, 2^-18 for the fp32 exponentials, sums and gate, and the scores' error (the oracle's window_bound)
    n = max(a + b for a, b in zip(c.lens, c.rows))
    bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -15 + 2.0 ** -18 + n * 2.0 ** -24 + 2 * (c.d + 8) * 2.0 ** -24 * reach[..., None]) * 1.01 * mag
    close(c.run(), want, bound)


# ---- extreme values -----------------------------------------------------------------

@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rows,hq,d", [(1, 2, 64), (9, 4, 64), (2, 2, 256), (16, 8, 128)])
def test_values_near_the_largest(rows, hq, d, e4m3):
    """Values of up to 2^126 under scores that rise from tile to tile: no sum of weighted values overflows that does not for weights of at most 1."""
    announce(f"values near the largest, {rows} rows, {hq} heads, d {d}, e4m3 {e4m3}")
    n = 2200
    c = Case([n], [rows], hq, 2, d, 64, seed=42)
    # base-2 scores of -120, but 0 and 7 for two keys of tiles that the same wave takes
    score = torch.full((n + rows,), -120.0)
    score[3], score[128 + 5], score[600], score[640 + 200] = 0.0, 7.0, 1.0, 6.0
    x = torch.randn((n + rows, 2, d), generator=c.g).clamp(-3, 3) * 2.0 ** 124
    at = torch.arange(n + rows)
    page, off = c.table[0, at // 64].long(), at % 64
    c.k[page, :, off] = 0
    c.k[page, :, off, 0] = score[:, None].to(BF16)
    c.v[page, :, off] = x.to(BF16)
    c.q = torch.zeros_like(c.q)
    c.q[:, :, 0] = 8
    if e4m3:
        for name in "kv":
            p = getattr(c, name).float()
            sc = p.abs().amax(-1).clamp(min=2.0 ** -100) / 448.0
            setattr(c, name, (p / sc[..., None]).to(F8))
            setattr(c, name + "s", sc)
    scale = np.log(2.0) / 8
    close(c.run(scale=scale), *c.oracle(scale=scale))


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("rows", [1, 2, 9])
def test_infinite_values_under_small_weights(rows, d):
    """An infinite value makes its channel infinite as long as its weight is a number above 0, a power of two among them."""
    announce(f"infinite values under small weights, {rows} rows, d {d}")
    n = 700
    c = Case([n], [rows], 4, 2, d, 64, seed=49)
    at = torch.arange(n + rows)
    page, off = c.table[0, at // 64].long(), at % 64
    c.k[page, :, off] = 0
    c.q = torch.zeros_like(c.q)
    c.q[:, :, 0] = 8
    scale = float(np.log(2.0) / 8)
    for key, score in ((130, -1.0), (131, -60.0), (400, -98.0), (401, -110.0)):
        for sign in (1.0, -1.0):
            k, v = c.k.clone(), c.v.clone()
            c.k[page[key], :, off[key], 0] = score
            c.v[page[key], :, off[key], 5] = sign * float("inf")
            got = f64(c.run(scale=scale))
            c.k, c.v = k, v
            assert np.all(got[:, :, 5] == sign * np.inf), (key, sign)
            assert np.all(np.isfinite(np.delete(got, 5, axis=2))), (key, sign)


@pytest.mark.parametrize("rows", [1, 2, 9])
def test_an_infinite_scale_makes_its_row_infinite(rows):
    """A cached e4m3 row of codes other than 0 under an infinite scale: infinities of the codes' signs."""
    announce(f"an infinite scale, {rows} rows")
    c = Case([300, 40], [rows, rows], 4, 2, 64, 16, e4m3=True, seed=51)
    clean = c.run()
    page, off = int(c.table[0, 70 // 16]), 70 % 16
    c.vs[page, :, off] = float("inf")
    codes = c.v.view(torch.uint8)
    codes[page, :, off] = torch.where(torch.arange(64) % 2 == 0, 0x38, 0xB8).to(torch.uint8)      # 1 and -1
    got = f64(c.run())
    assert np.all(got[:rows, :, 0::2] == np.inf) and np.all(got[:rows, :, 1::2] == -np.inf)
    assert np.array_equal(got[rows:], f64(clean)[rows:])


@pytest.mark.parametrize("rows,hq", [(1, 2), (9, 4)])
def test_e4m3_values_near_the_smallest(rows, hq):
    """Rows with the least scale: weights times scales lie near the least normal number."""
    announce(f"e4m3 values near the smallest, {rows} rows")
    c = Case([1500], [rows], hq, 2, 128, 32, e4m3=True, seed=43, amp=3.0)
    c.vs = torch.where(torch.isnan(c.vs), c.vs, torch.full_like(c.vs, 2.0 ** -100 / 448))
    close(c.run(), *c.oracle())


# ---- layouts ------------------------------------------------------------------------

def test_one_row_of_a_tensor_with_odd_rows():
    """One stream's step from a projection whose rows are no multiple of 16 bytes apart."""
    announce("prep and attention of one row with an odd stride")
    d, page = 64, 16
    x = torch.randn((1, 8 * d + 5), device="cuda", generator=torch.Generator("cuda").manual_seed(3)).to(BF16)
    views = [x[:, a * d:b * d].view(1, b - a, d) for a, b in ((0, 2), (2, 3), (3, 4), (4, 6))]
    res = []
    for q, k, v, gate in (views, [t.contiguous() for t in views]):
        kc, vc = (torch.zeros((1, 1, page, d), dtype=BF16, device="cuda") for _ in range(2))
        qo, out = (torch.zeros((1, 2, d), dtype=BF16, device="cuda") for _ in range(2))
        gdn.attn_prep(q, k, v, None, None, torch.ones(8, device="cuda"), i32([4]), i32([4]), qo, kc, vc)
        gdn.attn_window(i32([0, 1]), i32([4]), i32([[0]]), qo, kc, vc, out, None, max_kv=5, max_rows=1, gate=gate)
        res.append((qo, kc, vc, out))
    for a, b in zip(*res):
        assert torch.equal(a, b) and a.any()


def test_two_broken_entries_of_row_start_skip_their_streams_only():
    """The start of a block of 64 streams and the last entry at once."""
    announce("attention of 70 streams, two broken entries of row_start")
    c = Case([300 + 7 * s for s in range(70)], [2] * 70, 4, 2, 64, 32, seed=50)
    good = c.run()
    for first in (10 ** 6, -5):
        for last in (-5, 3, 10 ** 6):
            rs = c.row_start.clone()
            rs[64], rs[70] = first, last
            got = c.run(row_start=rs)
            for s in range(70):
                if s in (63, 64, 69):
                    assert torch.isnan(got[2 * s:2 * s + 2]).all(), (first, last, s)
                else:
                    assert torch.equal(got[2 * s:2 * s + 2], good[2 * s:2 * s + 2]), (first, last, s)


@pytest.mark.parametrize("by", [-3, -4, 3, 4])
def test_windows_that_overlap_touch_no_other_stream(by):
    """A small fall of row_start, after which two windows share rows: streams without shared rows get their pages and slots as ever."""
    announce(f"tables, overlapping windows, an entry off by {by}")
    n, at = 70, 33
    kv = np.arange(300, 300 + 7 * n, 7).astype(np.int32)
    rs = np.arange(0, 2 * n + 1, 2).astype(np.int32)
    rs[at] += by
    start = rs.tolist()
    window = {s: set(range(start[s], start[s + 1])) for s in range(n)}
    alone = [s for s in range(n) if s not in (at - 1, at) and not window[s] & (window[at - 1] | window[at])]
    assert n - 5 <= len(alone) < n - 2
    for tree in (False, True):
        d = tables_case(n, 16, 48, tree=False, free=300)
        d["kv_len"], d["slots"], d["positions"] = kv, np.full(2 * n, -9, np.int32), np.full(2 * n, -9, np.int32)
        d["block_table"] = np.concatenate([d["block_table"], np.full((n, 60), -7, np.int32)], 1)
        d["free_pages"] = np.concatenate([d["free_pages"], np.arange(d["free_pages"].shape[0], 5000)]).astype(np.int32)
        d["free_pages"][300:4000] = np.arange(1300, 5000)
        d["free_count"][:] = 4000
        d["row_start"], d["parent"] = rs, np.full(2 * n, -1, np.int32) if tree else None
        before = sorted(p for s in range(n) for p in d["block_table"][s, :d["page_count"][s]]) + sorted(d["free_pages"][:4000])
        out = {k: v.cpu().numpy() for k, v in run_tables(d, 16, False).items()}
        table, held = out["block_table"], out["page_count"]
        after = [p for s in range(n) for p in table[s, :held[s]]] + list(out["free_pages"][:out["free_count"][0]])
        assert sorted(after) == sorted(before)              # no page is lost or held twice
        for s in alone:
            for t in range(2):
                j = int(kv[s]) + t
                assert held[s] * 16 > j and out["slots"][2 * s + t] == table[s, j // 16] * 16 + j % 16, (s, t)


# ---- prompts ------------------------------------------------------------------------

# rows past those whose heads are spread over workgroups (512), where one workgroup goes through all of a row's heads:
# fewer than it holds at once, one batch of loads, several, a last one that is not full
@pytest.mark.parametrize("R,hq,hkv,d,rot,page,e4m3,inter,norm", [
    (513, 24, 4, 256, 64, 64, False, False, True), (700, 24, 4, 256, 64, 64, True, False, True),
    (530, 36, 9, 256, 256, 16, False, True, True), (530, 36, 9, 256, 256, 16, True, True, True),
    (515, 64, 8, 128, 100, 32, True, False, True), (515, 63, 9, 128, 128, 32, False, True, False),
    (600, 130, 10, 64, 64, 128, False, False, True), (600, 130, 10, 64, 22, 128, True, True, True),
    (1025, 3, 1, 64, 64, 256, True, False, False)])
def test_prep_of_prompts_matches_oracle(R, hq, hkv, d, rot, page, e4m3, inter, norm):
    prep_matches_oracle(R, hq, hkv, d, rot, page, e4m3, inter, norm)


def test_prep_of_prompts_equals_prep_in_pieces():
    """The rows of a long call have the bits that they have in calls of few rows."""
    announce("prep of 1,200 rows against pieces of 100")
    g = torch.Generator("cuda").manual_seed(45)
    R, hq, hkv, d, page = 1200, 30, 6, 128, 32
    x = torch.randn((R, hq + 2 * hkv, d), device="cuda", generator=g).to(BF16)
    w, freq = torch.rand((2, d), device="cuda", generator=g) + 0.5, 1e4 ** (-torch.arange(32, device="cuda") / 32)
    pos = torch.randint(0, 1 << 20, (R,), device="cuda", generator=g).to(I32)
    slots = torch.randperm(R + 80, device="cuda", generator=g)[:R].to(I32)
    for e4m3 in (False, True):
        res = []
        for step in (R, 100):
            kc, vc = (torch.zeros((40, hkv, page, d), device="cuda").to(F8 if e4m3 else BF16) for _ in range(2))
            sc = [torch.zeros((40, hkv, page), device="cuda") for _ in range(2)] if e4m3 else [None, None]
            qo = torch.zeros((R, hq, d), dtype=BF16, device="cuda")
            for a in range(0, R, step):
                p = x[a:a + step]
                gdn.attn_prep(p[:, :hq], p[:, hq:hq + hkv], p[:, hq + hkv:], w[0], w[1], freq, pos[a:a + step], slots[a:a + step],
                              qo[a:a + step], kc, vc, *sc)
            res.append([qo, kc.view(torch.uint8), vc.view(torch.uint8)] + (sc if e4m3 else []))
        for a, b in zip(*res):
            assert torch.equal(a, b) and a.any()


# ---- long streams ---------------------------------------------------------------------

@pytest.mark.parametrize("n,rows,hq,d,e4m3,tree", [
    (16384 - 8, 9, 2, 64, False, True), (16384 + 1, 12, 2, 64, True, False), (33000, 16, 2, 64, False, False),
    (40003, 9, 2, 128, True, True), (65536 - 9, 9, 2, 64, False, False), (65536 + 5, 16, 2, 64, True, True), (70001, 3, 8, 64, False, True)])
def test_wide_windows_over_long_streams(n, rows, hq, d, e4m3, tree):
    """More than 16 columns over streams whose chunks are longer than the usual 512 keys, up to 64 of them, beside short ones."""
    announce(f"{rows} rows of {hq} heads over {n} keys, d {d}, e4m3 {e4m3}, tree {tree}")
    c = Case([40, n, 700], [rows, rows, 2], hq, 1, d, 256, e4m3=e4m3, tree=tree, seed=46)
    out = c.run()
    close(out, *c.oracle())
    assert torch.equal(c.run(max_kv=1 << 18), out)
