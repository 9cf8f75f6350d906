"""Attention of whole prompts, the 4-bit cache and cached rows read back, without
a GPU: every host-side refusal, at the C boundary and in the binding, and the
oracle's pins."""
import ctypes as C

import numpy as np
import pytest
import torch

from oracle import attn as ref
from verify_causal_conv1d_amd import gdn

from test_abi_attn import L, P4, P8, P16, cache, refused  # noqa: F401

BAD_CACHES = [
    (dict(pages=0), gdn.GDN_EINVAL, "positive"), (dict(hkv=-1), gdn.GDN_EINVAL, "positive"),
    (dict(page=48), gdn.GDN_EUNSUPPORTED, "page_size"), (dict(d=96), gdn.GDN_EUNSUPPORTED, "d 96"),
    (dict(fmt=2), gdn.GDN_EINVAL, "format"), (dict(fmt=3), gdn.GDN_EINVAL, "format"), (dict(fmt=5), gdn.GDN_EINVAL, "format"),
    (dict(pages=1 << 23, page=64, hkv=4), gdn.GDN_EUNSUPPORTED, "2^31"),
    (dict(k=None), gdn.GDN_EINVAL, "k is NULL"), (dict(v=0x10004), gdn.GDN_EINVAL, "v must be 16-byte"),
    (dict(fmt=1), gdn.GDN_EINVAL, "k_scale"), (dict(fmt=4), gdn.GDN_EINVAL, "k_scale"),
    (dict(fmt=4, ks=0x10000), gdn.GDN_EINVAL, "v_scale"), (dict(fmt=4, ks=0x10001, vs=0x10000), gdn.GDN_EINVAL, "k_scale must be"),
]


def prompt(L, c=None, n=4, total=8306, max_kv=4722, blocks=80, hq=24, rs=P16, kv=P16, tb=P16, q=P16, gate=None, gr=0, gh=0,
           scale=1.0, out=P16, ws=P16, wsb=1 << 50):
    c = c or cache()
    return L.gdn_attn_prompt(C.byref(c), n, total, max_kv, blocks, hq, rs, kv, tb, q, gate, gr, gh, scale, out, ws, wsb, None)


def read(L, c=None, n=4, total=8306, blocks=80, rs=P16, first=P16, tb=P16, k=P16, v=P16):
    c = c or cache()
    return L.gdn_kv_read(C.byref(c), n, total, blocks, rs, first, tb, k, v, None)


@pytest.mark.parametrize("kw,code,needle", BAD_CACHES)
def test_bad_caches_are_refused(L, kw, code, needle):  # noqa: F811
    c = cache(**kw)
    refused(L, prompt(L, c=c, hq=24 if c.hkv > 0 else 1), code, needle)
    refused(L, read(L, c=c), code, needle)


@pytest.mark.parametrize("kw,code,needle", [
    (dict(n=-1), gdn.GDN_EINVAL, "negative"), (dict(total=-1), gdn.GDN_EINVAL, "negative"), (dict(max_kv=0), gdn.GDN_EINVAL, "max_kv"),
    (dict(max_kv=(1 << 21) + 1), gdn.GDN_EUNSUPPORTED, "max_kv"), (dict(blocks=0), gdn.GDN_EINVAL, "max_blocks"),
    (dict(blocks=1 << 26), gdn.GDN_EUNSUPPORTED, "max_blocks"), (dict(hq=22), gdn.GDN_EINVAL, "multiple"),
    (dict(hq=0), gdn.GDN_EINVAL, "multiple"), (dict(hq=2048), gdn.GDN_EUNSUPPORTED, "hq"),
    (dict(rs=None), gdn.GDN_EINVAL, "row_start"), (dict(kv=None), gdn.GDN_EINVAL, "kv_len"), (dict(tb=None), gdn.GDN_EINVAL, "block_table"),
    (dict(q=P8), gdn.GDN_EINVAL, "q must be"), (dict(q=None), gdn.GDN_EINVAL, "q is NULL"), (dict(out=None), gdn.GDN_EINVAL, "out is NULL"),
    (dict(gate=P4), gdn.GDN_EINVAL, "gate must be 8"), (dict(gate=P8, gr=6), gdn.GDN_EINVAL, "strides"),
    (dict(gate=P8, gh=-4), gdn.GDN_EINVAL, "strides"), (dict(scale=float("nan")), gdn.GDN_EINVAL, "scale"),
    (dict(scale=3e38), gdn.GDN_EINVAL, "scale"),
    (dict(total=65, max_kv=100000, blocks=2000, ws=None), gdn.GDN_EWORKSPACE, "workspace"),
    (dict(total=65, max_kv=100000, blocks=2000, wsb=100), gdn.GDN_EWORKSPACE, "workspace"),
    (dict(total=65, max_kv=100000, blocks=2000, ws=P8), gdn.GDN_EINVAL, "workspace must be"),
    (dict(total=(1 << 26) // 24 + 1), gdn.GDN_EUNSUPPORTED, "too many"), (dict(total=1 << 30), gdn.GDN_EUNSUPPORTED, "too many"),
])
def test_prompt_refusals(L, kw, code, needle):  # noqa: F811
    refused(L, prompt(L, **kw), code, needle)


@pytest.mark.parametrize("kw,code,needle", [
    (dict(n=-1), gdn.GDN_EINVAL, "negative"), (dict(total=-1), gdn.GDN_EINVAL, "negative"), (dict(blocks=0), gdn.GDN_EINVAL, "max_blocks"),
    (dict(blocks=1 << 26), gdn.GDN_EUNSUPPORTED, "max_blocks"), (dict(total=1 << 24), gdn.GDN_EUNSUPPORTED, "total_rows"),
    (dict(rs=None), gdn.GDN_EINVAL, "row_start"), (dict(first=None), gdn.GDN_EINVAL, "first"), (dict(tb=None), gdn.GDN_EINVAL, "block_table"),
    (dict(k=None), gdn.GDN_EINVAL, "k_out is NULL"), (dict(v=P8), gdn.GDN_EINVAL, "v_out must be"),
])
def test_read_refusals(L, kw, code, needle):  # noqa: F811
    refused(L, read(L, **kw), code, needle)


def test_nothing_to_do(L):  # noqa: F811
    for n in (0, 4):
        assert prompt(L, n=n, total=0, rs=None, q=None, ws=None) == gdn.GDN_OK
        assert read(L, n=n, total=0, rs=None, k=None) == gdn.GDN_OK
    assert prompt(L, n=0, total=5, rs=None, q=None, ws=None) == gdn.GDN_OK
    assert read(L, n=0, total=5, rs=None, k=None) == gdn.GDN_OK


@pytest.mark.parametrize("hq,hkv,d", [(24, 4, 256), (4, 2, 64), (8, 8, 128), (1024, 1, 64), (1, 1, 128), (1024, 1024, 64)])
def test_a_workspace_serves_every_smaller_call(L, hq, hkv, d):  # noqa: F811
    c = cache(hkv=hkv, d=d, page=16, pages=100)
    lengths = (1, 511, 512, 1023, 1024, 5000, 40000, 262144, 1 << 21)
    rows = (1, 2, 3, 10, 42, 43, 64, 65, 100, 255, 256, 257, 1000, 2730, 2731, 8306, 30000)
    assert gdn.attn_prompt_workspace_bytes(hq, hkv, d, 4, 100, 500) == 0               # not cut
    cut = 0
    for most_rows in (1, 65, 1000, 8306, 30000):
        for most in lengths:
            size = gdn.attn_prompt_workspace_bytes(hq, hkv, d, 16, most_rows, most)
            for total in (r for r in rows if r <= most_rows):
                for kv in (k for k in lengths if k <= most):
                    # enough: what is refused is an address, which is looked at after the size
                    rc = prompt(L, c=c, n=16, total=total, max_kv=kv, blocks=1 << 18, hq=hq, ws=P8, wsb=size, gate=P4)
                    refused(L, rc, gdn.GDN_EINVAL, "must be")
                    cut += "workspace" in L.gdn_last_error().decode()
    assert cut > 0 or hkv == 1024          # (whose tiles of one row each fill all 1,024 places of the chip)


def test_binding_takes_a_4_bit_cache():
    dev = -1
    k = torch.zeros((2, 1, 16, 32), dtype=torch.uint8)
    e = torch.zeros((2, 1, 16, 2), dtype=torch.uint8)
    packed, hkv, d = gdn._cache(dev, k, k.clone(), e, e.clone())
    assert (hkv, d) == (1, 64)
    assert packed[48:52] == (4).to_bytes(4, "little")
    for args, error, match in [
            ((k, k, None, None), ValueError, "uint8 cache needs k_scale"), ((k, k, e, None), ValueError, "needs k_scale"),
            ((k, k, e[:1], e), ValueError, "k_scale must hold"), ((k, k, e, e.float()), TypeError, "v_scale must be"),
            ((k, k.to(torch.int8), e, e), TypeError, "v_cache must be"), ((k.to(torch.int8), k, e, e), TypeError, "k_cache must be")]:
        with pytest.raises(error, match=match):
            gdn._cache(dev, *args)


def test_binding_refuses_before_the_library():
    cpu = torch.zeros(3, dtype=torch.int32)
    q = torch.zeros((1, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="device tensor"):
        gdn.attn_prompt(cpu, cpu, cpu.view(1, 3), q, None, None, None, None, max_kv=1)
    with pytest.raises(TypeError, match="device tensor"):
        gdn.kv_read(cpu, cpu, cpu.view(1, 3), None, None, None, None)


# ---- pins of the oracle -----------------------------------------------------

def test_oracle_mx_worked_by_hand():
    y = np.zeros((3, 32), np.float32)
    y[0, :8] = [6.0, -0.25, 0.75, 1.25, -1.75, 2.5, 3.5, -5.0]        # ties: to the even code
    y[1, :4] = [7.0, 3.4375, -0.2, 1e-30]                              # 7 goes a power of two up
    y[2, :2] = [448.0 * 2.0 ** -20, -1.0 * 2.0 ** -16]
    codes, exps = ref.mx_quantise(y)
    assert exps[:, 0].tolist() == [127, 128, 127 - 14 + 1]
    got = ref.mx_values(codes, exps)
    assert got[0, :8].tolist() == [6.0, 0.0, 1.0, 1.0, -2.0, 2.0, 4.0, -4.0]
    assert got[1, :4].tolist() == [8.0, 3.0, 0.0, 0.0]
    assert got[2, 0] == 4.0 * 2.0 ** -13 and got[2, 1] == -0.0
    assert codes[0, 0] == 0x87 and codes[0, 3] == 0xE6                 # even channels in the low halves, signs kept
    # ends of the range, and what is not finite
    top = float(np.finfo(np.float32).max)
    y = np.zeros((4, 32), np.float32)
    y[0, 0], y[1, 0], y[2, 5], y[3, 9] = top, 2.0 ** -120, np.inf, np.nan
    codes, exps = ref.mx_quantise(y)
    assert exps[:, 0].tolist() == [252, 25, 255, 255]
    got = ref.mx_values(codes, exps)
    assert got[0, 0] == 6.0 * 2.0 ** 125 and not got[1].any() and np.isnan(got[2:]).all()


def test_oracle_mx_keeps_its_own_values():
    g = np.random.default_rng(5)
    y = (g.normal(size=(64, 128)) * np.exp(g.normal(size=(64, 1)) * 9)).astype(np.float32)
    once = ref.mx_values(*ref.mx_quantise(y))
    codes, exps = ref.mx_quantise(once)
    np.testing.assert_array_equal(ref.mx_values(codes, exps), once)
    # in steps of the block, with a magnitude a and the block's largest, top >= a and
    # top >= 3.5: for a <= 4 off by 0.5 at most, so 0.5 / 3.5 of top; for 4 < a < 7 by
    # |a - 4|, |6 - a| or a - 6 of it, most at a = 5: 1 / 5
    assert np.max(np.abs(once - y) / np.abs(y).reshape(64, 4, 32).max(-1).repeat(32, -1)) <= 1.0 / 5.0


def test_oracle_prompt_is_the_window():
    g = np.random.default_rng(6)
    page, d = 4, 8
    k, v = g.normal(size=(9, 2, page, d)), g.normal(size=(9, 2, page, d))
    table, rs, kv = np.array([[4, 1, 2, 0], [7, 8, 3, 5], [6, 6, 6, 6]]), [0, 5, 12, 12], [6, 0, 3]
    q, gate = g.normal(size=(12, 4, d)), g.normal(size=(12, 4, d))
    for a, b in zip(ref.prompt(page, rs, kv, table, q, k, v, 0.3, gate), ref.window(page, rs, None, kv, table, q, k, v, 0.3, gate)):
        np.testing.assert_allclose(a, b, rtol=1e-12)


def test_oracle_read():
    pool = np.arange(3 * 1 * 4 * 2, dtype=np.float64).reshape(3, 1, 4, 2)
    out = ref.read(4, [0, 3], [3], np.array([[2, 0]]), pool, np.full((4, 1, 2), -1.0))
    assert out[:3, 0].tolist() == [pool[2, 0, 3].tolist(), pool[0, 0, 0].tolist(), pool[0, 0, 1].tolist()]
    assert (out[3] == -1.0).all()
