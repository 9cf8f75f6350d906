"""The attention-layer calls without a GPU: every host-side refusal, at the C
boundary and in the binding, and the oracle's pins."""
import ctypes as C

import numpy as np
import pytest
import torch

from oracle import attn as ref
from verify_causal_conv1d_amd import gdn

P16 = C.c_void_p(0x10000)     # never dereferenced: every call below is refused first, or has nothing to do
P8 = C.c_void_p(0x10008)
P4 = C.c_void_p(0x10004)


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(gdn.LIB_PATH):
        from verify_causal_conv1d_amd import build
        build.build()
    return gdn.lib()


class _KvCache(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("n_pages", C.c_int32), ("page_size", C.c_int32), ("hkv", C.c_int32), ("d", C.c_int32),
                ("format", C.c_int32)]


class _Rope(C.Structure):
    _fields_ = [("inv_freq", C.c_void_p), ("rot_dim", C.c_int32), ("interleaved", C.c_int32), ("rot_scale", C.c_float)]


def cache(k=0x10000, v=0x10000, ks=None, vs=None, pages=100, page=64, hkv=4, d=256, fmt=0):
    return _KvCache(k, v, ks, vs, pages, page, hkv, d, fmt)


def test_packed_structs_are_the_headers():
    """The binding's packed bytes lie as the C structs do."""
    assert gdn._pack_cache(1, 2, 3, 4, 5, 6, 7, 8, 1) == bytes(_KvCache(1, 2, 3, 4, 5, 6, 7, 8, 1))
    assert gdn._pack_rope(1, 64, 1, 1.5) == bytes(_Rope(1, 64, 1, 1.5))


def refused(L, rc, code, needle):
    assert rc == code, (rc, L.gdn_last_error())
    assert needle in L.gdn_last_error().decode(), L.gdn_last_error()


BAD_CACHES = [
    (dict(pages=0), gdn.GDN_EINVAL, "positive"), (dict(hkv=-1), gdn.GDN_EINVAL, "positive"),
    (dict(page=48), gdn.GDN_EUNSUPPORTED, "page_size"), (dict(page=8), gdn.GDN_EUNSUPPORTED, "page_size"),
    (dict(page=512), gdn.GDN_EUNSUPPORTED, "page_size"), (dict(d=96), gdn.GDN_EUNSUPPORTED, "d 96"),
    (dict(fmt=2), gdn.GDN_EINVAL, "format"), (dict(pages=1 << 23, page=64, hkv=4), gdn.GDN_EUNSUPPORTED, "2^31"),
    (dict(k=None), gdn.GDN_EINVAL, "k is NULL"), (dict(v=0x10004), gdn.GDN_EINVAL, "v must be 16-byte"),
    (dict(fmt=1), gdn.GDN_EINVAL, "k_scale"), (dict(fmt=1, ks=0x10000), gdn.GDN_EINVAL, "v_scale"),
]


def window(L, c=None, n=16, total=256, max_rows=16, max_kv=4096, blocks=64, hq=24, rs=P16, kv=P16, tb=P16, q=P16, gate=None,
           gr=0, gh=0, scale=1.0, out=P16, ws=P16, wsb=1 << 50):
    c = c or cache()
    return L.gdn_attn_window(C.byref(c), n, total, max_rows, max_kv, blocks, hq, rs, None, kv, tb, q, gate, gr, gh, scale, out,
                             ws, wsb, None)


@pytest.mark.parametrize("kw,code,needle", BAD_CACHES)
def test_bad_caches_are_refused_everywhere(L, kw, code, needle):
    c = cache(**kw)
    refused(L, window(L, c=c, hq=24 if c.hkv > 0 else 1), code, needle)
    rope = _Rope(0x10000, 64, 0, 1.0)
    refused(L, L.gdn_attn_prep(C.byref(c), 3, 24, P16, 0, 0, P16, 0, 0, P16, 0, 0, None, None, 1e-6, C.byref(rope), P16, P16,
                               P16, None), code, needle)
    refused(L, L.gdn_attn_commit(C.byref(c), 2, 9, 16, 64, P16, None, P16, P16, P16, P16, None), code, needle)


@pytest.mark.parametrize("kw,code,needle", [
    (dict(n=-1), gdn.GDN_EINVAL, "negative"), (dict(total=-1), gdn.GDN_EINVAL, "negative"),
    (dict(max_rows=0), gdn.GDN_EINVAL, "max_rows"), (dict(max_rows=17), gdn.GDN_EINVAL, "max_rows"),
    (dict(total=257), gdn.GDN_EINVAL, "exceeds"), (dict(max_kv=0), gdn.GDN_EINVAL, "max_kv"),
    (dict(max_kv=(1 << 21) + 1), gdn.GDN_EUNSUPPORTED, "max_kv"), (dict(blocks=0), gdn.GDN_EINVAL, "max_blocks"),
    (dict(blocks=1 << 26), gdn.GDN_EUNSUPPORTED, "max_blocks"), (dict(hq=22), gdn.GDN_EINVAL, "multiple"),
    (dict(hq=0), gdn.GDN_EINVAL, "multiple"), (dict(hq=2048), gdn.GDN_EUNSUPPORTED, "hq"),
    (dict(rs=None), gdn.GDN_EINVAL, "row_start"), (dict(kv=None), gdn.GDN_EINVAL, "kv_len"),
    (dict(tb=None), gdn.GDN_EINVAL, "block_table"), (dict(q=P8), gdn.GDN_EINVAL, "q must be"),
    (dict(out=None), gdn.GDN_EINVAL, "out is NULL"), (dict(gate=P4), gdn.GDN_EINVAL, "gate must be 8"),
    (dict(gate=P8, gr=6), gdn.GDN_EINVAL, "strides"), (dict(gate=P8, gh=-4), gdn.GDN_EINVAL, "strides"),
    (dict(scale=float("nan")), gdn.GDN_EINVAL, "scale"), (dict(scale=float("inf")), gdn.GDN_EINVAL, "scale"),
    (dict(scale=3e38), gdn.GDN_EINVAL, "scale"),
    (dict(ws=None), gdn.GDN_EWORKSPACE, "workspace"), (dict(wsb=100), gdn.GDN_EWORKSPACE, "workspace"),
    (dict(ws=P8), gdn.GDN_EINVAL, "workspace must be"),
    (dict(n=1 << 24, total=1, max_kv=1 << 21), gdn.GDN_EUNSUPPORTED, "too many"),
    (dict(n=1 << 20, total=1 << 22, wsb=1 << 50), gdn.GDN_EUNSUPPORTED, "too many"),
])
def test_window_refusals(L, kw, code, needle):
    refused(L, window(L, **kw), code, needle)


def test_nothing_to_do(L):
    assert window(L, n=0, total=0, rs=None, q=None) == gdn.GDN_OK
    assert window(L, n=4, total=0, rs=None, q=None) == gdn.GDN_OK
    c, rope = cache(k=None, v=None), _Rope(None, 64, 0, 1.0)
    assert L.gdn_attn_prep(C.byref(c), 0, 24, None, 0, 0, None, 0, 0, None, 0, 0, None, None, 1e-6, C.byref(rope), None, None,
                           None, None) == gdn.GDN_OK
    assert L.gdn_attn_commit(C.byref(c), 0, 0, 16, 64, None, None, None, None, None, None, None) == gdn.GDN_OK


@pytest.mark.parametrize("kw,code,needle", [
    (dict(rows=-1), gdn.GDN_EINVAL, "rows"), (dict(hq=5), gdn.GDN_EINVAL, "multiple"), (dict(qr=4), gdn.GDN_EINVAL, "q strides"),
    (dict(kh=-8), gdn.GDN_EINVAL, "k strides"), (dict(vr=9), gdn.GDN_EINVAL, "v strides"), (dict(rot=63), gdn.GDN_EINVAL, "rot_dim"),
    (dict(rot=258), gdn.GDN_EINVAL, "rot_dim"), (dict(rot=-2), gdn.GDN_EINVAL, "rot_dim"), (dict(eps=0.0), gdn.GDN_EINVAL, "eps"),
    (dict(eps=float("nan")), gdn.GDN_EINVAL, "eps"), (dict(rs=float("inf")), gdn.GDN_EINVAL, "rot_scale"),
    (dict(q=None), gdn.GDN_EINVAL, "q is NULL"), (dict(k=P8), gdn.GDN_EINVAL, "k must be"), (dict(v=None), gdn.GDN_EINVAL, "v is NULL"),
    (dict(qn=P4), gdn.GDN_EINVAL, "q_norm"), (dict(freq=None), gdn.GDN_EINVAL, "inv_freq"), (dict(pos=None), gdn.GDN_EINVAL, "positions"),
    (dict(slots=None), gdn.GDN_EINVAL, "slots"), (dict(out=P8), gdn.GDN_EINVAL, "q_out"),
    (dict(rows=1 << 24), gdn.GDN_EUNSUPPORTED, "rows"),
])
def test_prep_refusals(L, kw, code, needle):
    def call(rows=3, hq=24, q=P16, k=P16, v=P16, qr=0, kh=0, vr=0, rot=64, freq=0x10000, rs=1.0, eps=1e-6, qn=None, pos=P16,
             slots=P16, out=P16):
        c, rope = cache(), _Rope(freq, rot, 0, rs)
        return L.gdn_attn_prep(C.byref(c), rows, hq, q, qr, 0, k, 0, kh, v, vr, 0, qn, None, eps, C.byref(rope), pos, slots, out,
                               None)
    refused(L, call(**kw), code, needle)


@pytest.mark.parametrize("kw,code,needle", [
    (dict(page=24), gdn.GDN_EUNSUPPORTED, "page_size"), (dict(n=-1), gdn.GDN_EINVAL, "n_streams"),
    (dict(n=4097), gdn.GDN_EUNSUPPORTED, "streams"), (dict(total=-1), gdn.GDN_EINVAL, "total_rows"),
    (dict(pages=0), gdn.GDN_EINVAL, "n_pages"), (dict(pages=1 << 28), gdn.GDN_EUNSUPPORTED, "pool"),
    (dict(blocks=0), gdn.GDN_EINVAL, "max_blocks"), (dict(n=4096, blocks=1 << 20), gdn.GDN_EUNSUPPORTED, "table"),
    (dict(rs=None), gdn.GDN_EINVAL, "row_start"), (dict(kv=None), gdn.GDN_EINVAL, "kv_len"), (dict(pc=None), gdn.GDN_EINVAL, "page_count"),
    (dict(fc=None), gdn.GDN_EINVAL, "free_count"), (dict(fp=None), gdn.GDN_EINVAL, "free_pages"), (dict(tb=None), gdn.GDN_EINVAL, "block_table"),
    (dict(sl=None), gdn.GDN_EINVAL, "slots"), (dict(pos=None), gdn.GDN_EINVAL, "positions"),
    (dict(total=(1 << 30) + 1), gdn.GDN_EUNSUPPORTED, "total_rows"), (dict(n=4096, blocks=(1 << 18) + 1), gdn.GDN_EUNSUPPORTED, "table"),
])
def test_tables_refusals(L, kw, code, needle):
    def call(n=16, total=256, page=16, pages=1000, blocks=64, rs=P16, kv=P16, pc=P16, fc=P16, fp=P16, tb=P16, sl=P16, pos=P16):
        return L.gdn_kv_tables(n, total, page, pages, blocks, rs, None, kv, pc, fc, fp, tb, sl, pos, pc, fc, None)
    refused(L, call(**kw), code, needle)


@pytest.mark.parametrize("kw,code,needle", [
    (dict(n=-1), gdn.GDN_EINVAL, "n_streams"), (dict(max_rows=17), gdn.GDN_EINVAL, "max_rows"), (dict(blocks=0), gdn.GDN_EINVAL, "max_blocks"),
    (dict(rs=None), gdn.GDN_EINVAL, "row_start"), (dict(acc=None), gdn.GDN_EINVAL, "accept_row"), (dict(kv=None), gdn.GDN_EINVAL, "kv_len"),
    (dict(tb=None), gdn.GDN_EINVAL, "block_table"), (dict(n=1 << 24), gdn.GDN_EUNSUPPORTED, "n_streams"),
])
def test_commit_refusals(L, kw, code, needle):
    def call(n=2, total=9, max_rows=16, blocks=64, rs=P16, acc=P16, kv=P16, tb=P16):
        c = cache()
        return L.gdn_attn_commit(C.byref(c), n, total, max_rows, blocks, rs, None, acc, kv, tb, P16, None)
    refused(L, call(**kw), code, needle)


def test_workspace_bytes(L):
    def need(**kw):
        a = dict(hq=24, hkv=4, d=256, n_streams=16, total_rows=256, max_rows=16, max_kv=4096) | kw
        return gdn.attn_workspace_bytes(**a)
    assert need(max_kv=1) == 0                              # one chunk: nothing to join
    for bad in (dict(hq=23), dict(d=80), dict(max_rows=17), dict(max_kv=0), dict(total_rows=-1)):
        assert need(**bad) == 0
    assert need() > 0 and need(total_rows=512, n_streams=32) == 2 * need()
    # a longer bound never needs less
    sizes = [need(max_kv=m) for m in (1, 100, 1000, 5000, 16000, 16384, 16385, 20000, 40000, 262144, 1 << 21)]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("hq,hkv,d", [(24, 4, 256), (4, 2, 64), (8, 8, 128), (16, 1, 64), (17, 1, 128), (64, 2, 64)])
def test_a_workspace_serves_every_smaller_call(L, hq, hkv, d):
    """Sized once for the largest call, it is enough for all with fewer rows, shorter windows or shorter streams."""
    def need(total, rows, kv):
        return gdn.attn_workspace_bytes(hq, hkv, d, 256, total, rows, kv)
    lengths = (1, 128, 129, 1000, 4096, 8192, 16384, 40000, 262144, 1 << 21)
    for total in (16, 256):
        for kv in lengths:
            sizes = [need(total, r, kv) for r in range(1, 17)]
            assert sizes == sorted(sizes)                   # more rows a window never need less
    for most in (4096, 262144, 1 << 21):
        size = need(256, 16, most)
        for kv in (k for k in lengths if k <= most):
            for rows in (1, 2, 3, 5, 9, 16):
                for total in (1, 64, 256):
                    if need(total, rows, kv) == 0:
                        continue
                    # enough: what is refused is the address, which is looked at after the size
                    rc = window(L, c=cache(hkv=hkv, d=d), n=256, total=total, max_rows=rows, max_kv=kv, blocks=1 << 16, hq=hq, ws=P8,
                                wsb=size)
                    refused(L, rc, gdn.GDN_EINVAL, "workspace must be")


def test_binding_refuses_before_the_library():
    cpu = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError, match="device tensor"):
        gdn.kv_tables(cpu, cpu, cpu, cpu, cpu, cpu.view(1, 3), cpu, cpu, page_size=16)
    with pytest.raises(TypeError, match="device tensor"):
        gdn.attn_window(cpu, cpu, cpu.view(1, 3), torch.zeros(1, 1, 64, dtype=torch.bfloat16), None, None, None, None, max_kv=1)
    dev = -1            # torch's number for the CPU: the checks run as on a device
    k = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16)
    f8 = k.to(torch.float8_e4m3fn)
    assert gdn._cache(dev, k, k.clone(), None, None)[1:] == (1, 64)
    for args, error, match in [
            ((k, k, torch.zeros(1), None), ValueError, "no scales"), ((k.float(), k, None, None), TypeError, "k_cache must be"),
            ((k, k[:1], None, None), ValueError, "v_cache must hold"), ((k, f8, None, None), TypeError, "v_cache must be"),
            ((f8, f8, None, None), ValueError, "needs k_scale"), ((f8, f8, torch.zeros(32), torch.zeros(31)), ValueError, "v_scale must hold"),
            ((f8, f8, torch.zeros(32).double(), torch.zeros(32)), TypeError, "k_scale must be"),
            ((k.transpose(2, 3), k.transpose(2, 3), None, None), ValueError, "contiguous"), ((k[0], k[0], None, None), ValueError, "k_cache must be")]:
        with pytest.raises(error, match=match):
            gdn._cache(dev, *args)
    q = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    assert gdn._heads(dev, "q", torch.zeros((3, 4, 64), dtype=torch.bfloat16)[:, ::2], (3, 2, 64))[1:] == (256, 128)
    with pytest.raises(ValueError, match="channels must be contiguous"):
        gdn._heads(dev, "q", torch.zeros((3, 64, 2), dtype=torch.bfloat16).transpose(1, 2), (3, 2, 64))
    with pytest.raises(ValueError, match="q must be"):
        gdn._heads(dev, "q", q, (3, 3, 64))
    with pytest.raises(TypeError, match="must be torch.bfloat16"):
        gdn._heads(dev, "q", q.float(), (3, 2, 64))
    with pytest.raises(ValueError, match="as the cache"):
        gdn._query(q, 128)
    with pytest.raises(TypeError, match="must be torch.int32"):
        gdn._i32s("kv_len", cpu.long(), dev, 3)
    with pytest.raises(ValueError, match="must hold 4"):
        gdn._i32s("kv_len", cpu, dev, 4)
    with pytest.raises(TypeError, match="cuda:0"):
        gdn._i32s("kv_len", cpu, 0, 3)


def test_strides_of_single_rows_and_heads_do_not_count():
    """One row, or one head, of a tensor whose rows have an odd length: its stride is not looked at."""
    x = torch.zeros((5, 133), dtype=torch.bfloat16)
    assert gdn._heads(-1, "q", x[2:3, :128].view(1, 2, 64), (1, 2, 64))[1:] == (0, 64)
    y = torch.zeros((1, 7, 67), dtype=torch.bfloat16)
    assert gdn._heads(-1, "k", y[:, 3:4, :64], (1, 1, 64))[1:] == (0, 0)
    z = torch.zeros((6, 131), dtype=torch.bfloat16).as_strided((3, 1, 64), (136, 67, 1))
    assert gdn._heads(-1, "v", z, (3, 1, 64))[1:] == (136, 0)
    assert gdn._heads(-1, "q", x[:, :128].view(5, 2, 64), (5, 2, 64))[1:] == (133, 64)     # five rows: it counts, and is refused


def test_binding_imports_on_a_torch_without_raw_calls(L):
    """A torch built without a GPU lacks its private stream and device calls: what needs no device still works."""
    import subprocess
    import sys
    code = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from verify_causal_conv1d_amd import gdn
gdn.check_layout([0, 3, 5], 16, 5, [-1, 0, 1, -1, 0])
assert gdn.attn_workspace_bytes(24, 4, 256, 16, 256, 16, 4096) > 0
torch.cuda.current_stream = lambda dev: type("S", (), {"cuda_stream": 40 + dev})
assert gdn._raw_stream(2) == 42 and gdn._current_device is torch.cuda.current_device
"""
    root = __file__.rsplit("/tests/", 1)[0]
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert done.returncode == 0, done.stderr


# ---- pins of the oracle -----------------------------------------------------

def test_oracle_tables_worked_by_hand():
    # page 4; stream 0 grows 2 -> 3 pages, stream 1 has finished (2 pages back), stream 2 is admitted with 5 rows
    table = np.array([[7, 3, -1], [5, 9, -1], [-1, -1, -1]], np.int32)
    r = ref.tables(4, [0, 2, 2, 7], None, np.array([7, -1, 0]), np.array([2, 2, 0]), 1, np.array([2, -1, -1, -1]), table,
                   np.zeros(7, np.int32), np.zeros(7, np.int32))
    # the stack: 2, then 5 and 9 on top; stream 0 takes 9, stream 2 takes 5 and 2
    assert r["block_table"].tolist() == [[7, 3, 9], [5, 9, -1], [5, 2, -1]]
    assert r["free_count"] == 0 and r["page_count"].tolist() == [3, 0, 2]
    assert r["slots"].tolist() == [3 * 4 + 3, 9 * 4, 20, 21, 22, 23, 8]
    assert r["positions"].tolist() == [7, 8, 0, 1, 2, 3, 4]


def test_oracle_window_special_cases():
    g = np.random.default_rng(3)
    page, d = 4, 8
    k, v = g.normal(size=(6, 1, page, d)), g.normal(size=(6, 1, page, d))
    table, rs = np.array([[4, 1, 2]]), [0, 3]
    q = g.normal(size=(3, 2, d))
    # zero queries: the mean of the visible values; a tree's second child sees the root but not its sibling
    out, mag, _ = ref.window(page, rs, [-1, 0, 0], [6], table, 0 * q, k, v, 1.0)
    seq = np.concatenate([v[4, 0], v[1, 0], v[2, 0]])
    np.testing.assert_allclose(out[0, 1], seq[:7].mean(0), atol=1e-12)
    np.testing.assert_allclose(out[2, 0], seq[[0, 1, 2, 3, 4, 5, 6, 8]].mean(0), atol=1e-12)
    np.testing.assert_allclose(mag[0, 0], np.abs(seq[:7]).mean(0), atol=1e-12)
    # a very large scale picks the best key; a gate of 0 halves the result
    big, _, _ = ref.window(page, rs, None, [6], table, q, k, v, 1e6, gate=np.zeros_like(q))
    keys = np.concatenate([k[4, 0], k[1, 0], k[2, 0]])[:9]
    np.testing.assert_allclose(big[2, 1], 0.5 * seq[np.argmax(keys @ q[2, 1])], atol=1e-12)


def test_oracle_rotation_and_norm():
    g = np.random.default_rng(4)
    x, freq = g.normal(size=(5, 2, 8)), np.array([1.0, 0.1, 0.01])
    pos = [0, 1, 7, 100, 1 << 18]
    for inter in (False, True):
        y, mag = ref.rotated(x, pos, freq, inter)
        np.testing.assert_allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-12)   # a rotation
        np.testing.assert_array_equal(y[0], x[0])
        np.testing.assert_array_equal(y[:, :, 6:], x[:, :, 6:])
        assert np.all(np.abs(y) <= mag * (1 + 1e-12))
        # scores depend on the distance alone
        a, _ = ref.rotated(x[:1], [5], freq, inter)
        b, _ = ref.rotated(x[1:2], [2], freq, inter)
        a2, _ = ref.rotated(x[:1], [1005], freq, inter)
        b2, _ = ref.rotated(x[1:2], [1002], freq, inter)
        np.testing.assert_allclose((a * b).sum(-1), (a2 * b2).sum(-1), atol=1e-9)
    n = ref.normed(x, np.ones(8), 0.0)
    np.testing.assert_allclose((n * n).mean(-1), 1.0, rtol=1e-12)


def test_oracle_commit_moves_the_path():
    pool = np.arange(4 * 1 * 4, dtype=np.float64).reshape(4, 1, 4)
    table = np.array([[2, 0, 3]])
    (got,), length = ref.commit(4, [0, 5], [-1, 0, 0, 2, 1], [3], [2], table, pool)     # path 0, 2, 3 at cache rows 2, 4, 5
    assert length.tolist() == [5]
    row = lambda p, i: p[table[0, i // 4], 0, i % 4]  # noqa: E731
    assert [row(got, i) for i in (2, 3, 4)] == [row(pool, i) for i in (2, 4, 5)]
    assert row(got, 5) == row(pool, 5)


def test_oracle_tables_without_pages():
    # page 4, nothing free: stream 0 asks for a second page where its table still names page 2, which stream 1 holds
    table = np.array([[7, 2, 9, -5], [5, 2, -1, -1]], np.int32)
    r = ref.tables(4, [0, 9, 10], None, np.array([3, 5]), np.array([1, 2]), 0, np.array([-1] * 9, np.int32), table,
                   np.zeros(10, np.int32), np.zeros(10, np.int32))
    assert r["block_table"].tolist() == [[7, -1, 9, -5], [5, 2, -1, -1]]
    assert r["page_count"].tolist() == [1, 2] and r["free_count"] == 0
    assert r["slots"].tolist() == [-1] * 9 + [2 * 4 + 1]
