"""ctypes binding of libgdn.so: the same entry points as ``include/libgdn.h``.

Argument marshalling only: torch tensors go in as ``data_ptr()``, the launch
stream is torch's current stream on the tensors' device, and every step of the
computation runs in libgdn's HIP kernels.  A missing or unloadable library
raises; there is no fallback.
"""
from __future__ import annotations

import ctypes as C
import os
import struct
import threading
from typing import Optional

import torch

from .inputs import Shape

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")

GDN_OK, GDN_EINVAL, GDN_EUNSUPPORTED, GDN_EWORKSPACE, GDN_EHIP = 0, -1, -2, -3, -4
MAX_WINDOW_ROWS = 16
PREFILL_SCRATCH_BYTES = 128 * 1024 * 1024   # the fixed workspace of prefill_chunked_noalloc

EXPORTED = (
    "gdn_status_name", "gdn_last_error", "gdn_channels", "gdn_conv_step", "gdn_recur_window",
    "gdn_recur_tree", "gdn_commit", "gdn_recur_log", "gdn_commit_replay",
    "gdn_prefill_workspace_bytes", "gdn_prefill_chunked", "gdn_prefill_chunked_noalloc",
    "gdn_check_layout",
    "gdn_inproj_affine4", "gdn_inproj_pack_affine4", "gdn_inproj_padded_features",
    "gdn_kv_tables", "gdn_attn_prep", "gdn_attn_workspace_bytes", "gdn_attn_window", "gdn_attn_commit",
    "gdn_attn_prompt_workspace_bytes", "gdn_attn_prompt", "gdn_kv_read",
)


class GdnError(RuntimeError):
    def __init__(self, status: int, fn: str, msg: str):
        super().__init__(f"{fn}: {msg} ({status_name(status)})")
        self.status = status


class _Shape(C.Structure):
    _fields_ = [("hk", C.c_int32), ("hv", C.c_int32), ("dk", C.c_int32), ("dv", C.c_int32),
                ("conv_width", C.c_int32)]


class _Params(C.Structure):
    _fields_ = [("conv_w", C.c_void_p), ("a_log", C.c_void_p), ("dt_bias", C.c_void_p)]


_lock = threading.Lock()
_lib = None


def lib():
    """The loaded libgdn.so (built by ``verify_causal_conv1d_amd.build``)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is not built: run python -m verify_causal_conv1d_amd.build")
            L = C.CDLL(LIB_PATH)
            P, i32 = C.c_void_p, C.c_int32
            L.gdn_status_name.restype = C.c_char_p
            L.gdn_status_name.argtypes = [C.c_int]
            L.gdn_last_error.restype = C.c_char_p
            L.gdn_channels.restype = i32
            L.gdn_channels.argtypes = [P]
            L.gdn_conv_step.argtypes = [P, P, i32, P, P, P, P, P, P, P]
            L.gdn_recur_window.argtypes = [P, P, i32, i32, i32, P, P, P, P, P, P, P, P, P, P]
            L.gdn_recur_tree.argtypes = [P, P, i32, i32, i32, P, P, P, P, P, P, P, P, P, P, P]
            L.gdn_commit.argtypes = [P, i32, i32, P, P, P, P, P, P, P]
            L.gdn_recur_log.argtypes = [P, P, i32, i32, i32, P, P, P, P, P, P, P, P, P, P, P, P]
            L.gdn_commit_replay.argtypes = [P, i32, i32, i32, P, P, P, P, P, P, P, P, P, P]
            L.gdn_prefill_workspace_bytes.restype = C.c_size_t
            L.gdn_prefill_workspace_bytes.argtypes = [P, i32, i32]
            L.gdn_prefill_chunked.argtypes = [P, P, i32, i32, i32, P, P, P, P, P, P, P, P,
                                              C.c_size_t, P]
            L.gdn_prefill_chunked_noalloc.argtypes = [P, P, i32, i32, i32, P, P, P, P, P, P, P, P]
            L.gdn_check_layout.argtypes = [i32, i32, i32, P, P]
            L.gdn_inproj_affine4.argtypes = [P, i32, i32, i32, P, P, P, P, P, P, P, P]
            L.gdn_inproj_pack_affine4.argtypes = [P, i32, i32, P, P, P, P, P, P, P]
            L.gdn_inproj_padded_features.restype = i32
            L.gdn_inproj_padded_features.argtypes = [P]
            i64, f32 = C.c_int64, C.c_float
            L.gdn_kv_tables.argtypes = [i32] * 5 + [P] * 12
            L.gdn_attn_prep.argtypes = [P, i32, i32, P, i64, i64, P, i64, i64, P, i64, i64, P, P, f32, P, P, P, P, P]
            L.gdn_attn_workspace_bytes.restype = C.c_size_t
            L.gdn_attn_workspace_bytes.argtypes = [P, i32, i32, i32, i32, i32]
            L.gdn_attn_window.argtypes = [P] + [i32] * 6 + [P] * 6 + [i64, i64, f32, P, P, C.c_size_t, P]
            L.gdn_attn_commit.argtypes = [P] + [i32] * 4 + [P] * 7
            L.gdn_attn_prompt_workspace_bytes.restype = C.c_size_t
            L.gdn_attn_prompt_workspace_bytes.argtypes = [P, i32, i32, i32, i32]
            L.gdn_attn_prompt.argtypes = [P] + [i32] * 5 + [P] * 5 + [i64, i64, f32, P, P, C.c_size_t, P]
            L.gdn_kv_read.argtypes = [P] + [i32] * 3 + [P] * 6
            for name in ("gdn_conv_step", "gdn_recur_window", "gdn_recur_tree", "gdn_commit",
                         "gdn_recur_log", "gdn_commit_replay", "gdn_prefill_chunked",
                         "gdn_prefill_chunked_noalloc",
                         "gdn_check_layout", "gdn_inproj_affine4", "gdn_inproj_pack_affine4", "gdn_kv_tables",
                         "gdn_attn_prep", "gdn_attn_window", "gdn_attn_commit", "gdn_attn_prompt", "gdn_kv_read"):
                getattr(L, name).restype = C.c_int
            _lib = L
    return _lib


def status_name(status: int) -> str:
    return lib().gdn_status_name(int(status)).decode()


def _check(status: int, fn: str):
    if status != GDN_OK:
        raise GdnError(status, fn, lib().gdn_last_error().decode())


def _shape(shape: Shape) -> _Shape:
    return _Shape(shape.hk, shape.hv, shape.dk, shape.dv, 4)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else C.c_void_p(t.data_ptr())


def _dev(t: torch.Tensor, dtype, name):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _stream(t: torch.Tensor):
    return C.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


class LayerParams:
    """Device copies of one layer's parameters (conv weights, A_log, dt_bias)."""

    def __init__(self, conv_w: torch.Tensor, a_log: torch.Tensor, dt_bias: torch.Tensor):
        self.conv_w = _dev(conv_w, torch.float32, "conv_w")
        self.a_log = _dev(a_log, torch.float32, "a_log")
        self.dt_bias = _dev(dt_bias, torch.float32, "dt_bias")
        self._c = _Params(self.conv_w.data_ptr(), self.a_log.data_ptr(), self.dt_bias.data_ptr())

    @classmethod
    def from_host(cls, p, device="cuda"):
        return cls(p.conv_w.to(device), p.a_log.to(device), p.dt_bias.to(device))


def channels(shape: Shape) -> int:
    return int(lib().gdn_channels(C.byref(_shape(shape))))


def conv_step(shape: Shape, params: LayerParams, qkv, a, b, conv_tail, state, out):
    """One-row decode step of n streams; conv_tail and state are updated in place."""
    n = qkv.shape[0]
    for t, dt, nm in ((qkv, torch.bfloat16, "qkv"), (a, torch.bfloat16, "a"), (b, torch.bfloat16, "b"),
                      (conv_tail, torch.bfloat16, "conv_tail"), (state, torch.float32, "state"),
                      (out, torch.float32, "out")):
        _dev(t, dt, nm)
    sh = _shape(shape)
    _check(lib().gdn_conv_step(C.byref(sh), C.byref(params._c), n, _ptr(qkv), _ptr(a), _ptr(b),
                               _ptr(conv_tail), _ptr(state), _ptr(out), _stream(qkv)),
           "gdn_conv_step")


def _rows_call(fn, shape, params, row_start, qkv, a, b, conv_tail, state, out, tail_snap,
               state_snap, max_rows, parent=None):
    n = row_start.shape[0] - 1
    total = qkv.shape[0]
    for t, dt, nm in ((row_start, torch.int32, "row_start"), (qkv, torch.bfloat16, "qkv"),
                      (a, torch.bfloat16, "a"), (b, torch.bfloat16, "b"),
                      (conv_tail, torch.bfloat16, "conv_tail"), (state, torch.float32, "state"),
                      (out, torch.float32, "out"), (tail_snap, torch.bfloat16, "tail_snap"),
                      (state_snap, torch.float32, "state_snap")):
        _dev(t, dt, nm)
    sh = _shape(shape)
    args = [C.byref(sh), C.byref(params._c), n, total, int(max_rows), _ptr(row_start)]
    if parent is not None:
        _dev(parent, torch.int32, "parent")
        args.append(_ptr(parent))
    args += [_ptr(qkv), _ptr(a), _ptr(b), _ptr(conv_tail), _ptr(state), _ptr(out),
             _ptr(tail_snap), _ptr(state_snap), _stream(qkv)]
    return getattr(lib(), fn)(*args)


def recur_window(shape, params, row_start, qkv, a, b, conv_tail, state, out, tail_snap,
                 state_snap, max_rows=MAX_WINDOW_ROWS):
    """Verify windows (chains), recording every row's state and tail."""
    _check(_rows_call("gdn_recur_window", shape, params, row_start, qkv, a, b, conv_tail, state,
                      out, tail_snap, state_snap, max_rows), "gdn_recur_window")


def recur_tree(shape, params, row_start, parent, qkv, a, b, conv_tail, state, out, tail_snap,
               state_snap, max_rows=MAX_WINDOW_ROWS):
    """Tree windows: ``parent`` holds local parent indices (-1 = stream state)."""
    _check(_rows_call("gdn_recur_tree", shape, params, row_start, qkv, a, b, conv_tail, state,
                      out, tail_snap, state_snap, max_rows, parent=parent), "gdn_recur_tree")


def commit(shape, row_start, accept_row, tail_snap, state_snap, conv_tail, state):
    """Each stream's accepted row (packed index within its window of
    ``row_start``, -1 = keep) becomes its state and tail."""
    for t, dt, nm in ((row_start, torch.int32, "row_start"), (accept_row, torch.int32, "accept_row"),
                      (tail_snap, torch.bfloat16, "tail_snap"),
                      (state_snap, torch.float32, "state_snap"), (conv_tail, torch.bfloat16, "conv_tail"),
                      (state, torch.float32, "state")):
        _dev(t, dt, nm)
    sh = _shape(shape)
    _check(lib().gdn_commit(C.byref(sh), accept_row.shape[0], state_snap.shape[0], _ptr(row_start),
                            _ptr(accept_row), _ptr(tail_snap), _ptr(state_snap), _ptr(conv_tail), _ptr(state),
                            _stream(state)), "gdn_commit")


def recur_log(shape, params, row_start, qkv, a, b, conv_tail, state, out, log_alpha, log_delta,
              log_key, max_rows=MAX_WINDOW_ROWS, parent=None):
    """Verify windows (parent None) or trees that log every row's decay
    ``log_alpha`` [R][hv], write ``log_delta`` [R][hv][dv] and key ``log_key``
    [R][hk][dk] (fp32) instead of recording its state and tail."""
    n = row_start.shape[0] - 1
    total = qkv.shape[0]
    for t, dt, nm in ((row_start, torch.int32, "row_start"), (qkv, torch.bfloat16, "qkv"),
                      (a, torch.bfloat16, "a"), (b, torch.bfloat16, "b"),
                      (conv_tail, torch.bfloat16, "conv_tail"), (state, torch.float32, "state"),
                      (out, torch.float32, "out"), (log_alpha, torch.float32, "log_alpha"),
                      (log_delta, torch.float32, "log_delta"), (log_key, torch.float32, "log_key")):
        _dev(t, dt, nm)
    if parent is not None:
        _dev(parent, torch.int32, "parent")
    sh = _shape(shape)
    _check(lib().gdn_recur_log(C.byref(sh), C.byref(params._c), n, total, int(max_rows),
                               _ptr(row_start), _ptr(parent), _ptr(qkv), _ptr(a), _ptr(b),
                               _ptr(conv_tail), _ptr(state), _ptr(out), _ptr(log_alpha),
                               _ptr(log_delta), _ptr(log_key), _stream(qkv)), "gdn_recur_log")


def commit_replay(shape, row_start, accept_row, qkv, log_alpha, log_delta, log_key, conv_tail, state,
                  max_rows=MAX_WINDOW_ROWS, parent=None):
    """Each stream's kept path (accepted packed row, -1 = keep) replayed from
    the log onto its state; the path's last raw rows become its conv tail."""
    for t, dt, nm in ((row_start, torch.int32, "row_start"), (accept_row, torch.int32, "accept_row"),
                      (qkv, torch.bfloat16, "qkv"), (log_alpha, torch.float32, "log_alpha"),
                      (log_delta, torch.float32, "log_delta"), (log_key, torch.float32, "log_key"),
                      (conv_tail, torch.bfloat16, "conv_tail"), (state, torch.float32, "state")):
        _dev(t, dt, nm)
    if parent is not None:
        _dev(parent, torch.int32, "parent")
    sh = _shape(shape)
    _check(lib().gdn_commit_replay(C.byref(sh), accept_row.shape[0], qkv.shape[0], int(max_rows),
                                   _ptr(row_start), _ptr(parent), _ptr(accept_row), _ptr(qkv),
                                   _ptr(log_alpha), _ptr(log_delta), _ptr(log_key), _ptr(conv_tail),
                                   _ptr(state), _stream(state)), "gdn_commit_replay")


def prefill_workspace_bytes(shape: Shape, n_seqs: int, total_rows: int) -> int:
    sh = _shape(shape)
    return int(lib().gdn_prefill_workspace_bytes(C.byref(sh), int(n_seqs), int(total_rows)))


def prefill_chunked(shape, params, seq_start, qkv, a, b, conv_tail, state, out, workspace,
                    max_len: int):
    """Chunked prompt passes; conv_tail and state are updated in place."""
    for t, dt, nm in ((seq_start, torch.int32, "seq_start"), (qkv, torch.bfloat16, "qkv"),
                      (a, torch.bfloat16, "a"), (b, torch.bfloat16, "b"),
                      (conv_tail, torch.bfloat16, "conv_tail"), (state, torch.float32, "state"),
                      (out, torch.float32, "out"), (workspace, torch.uint8, "workspace")):
        _dev(t, dt, nm)
    sh = _shape(shape)
    _check(lib().gdn_prefill_chunked(C.byref(sh), C.byref(params._c), seq_start.shape[0] - 1,
                                     qkv.shape[0], int(max_len), _ptr(seq_start), _ptr(qkv),
                                     _ptr(a), _ptr(b), _ptr(conv_tail), _ptr(state), _ptr(out),
                                     _ptr(workspace), workspace.numel(), _stream(qkv)),
           "gdn_prefill_chunked")


def prefill_chunked_noalloc(shape, params, seq_start, qkv, a, b, conv_tail, state, out, max_len: int):
    """``prefill_chunked`` with the library's fixed workspace (allocates
    nothing; passes needing more than PREFILL_SCRATCH_BYTES are refused)."""
    for t, dt, nm in ((seq_start, torch.int32, "seq_start"), (qkv, torch.bfloat16, "qkv"),
                      (a, torch.bfloat16, "a"), (b, torch.bfloat16, "b"),
                      (conv_tail, torch.bfloat16, "conv_tail"), (state, torch.float32, "state"),
                      (out, torch.float32, "out")):
        _dev(t, dt, nm)
    sh = _shape(shape)
    _check(lib().gdn_prefill_chunked_noalloc(C.byref(sh), C.byref(params._c), seq_start.shape[0] - 1,
                                             qkv.shape[0], int(max_len), _ptr(seq_start), _ptr(qkv),
                                             _ptr(a), _ptr(b), _ptr(conv_tail), _ptr(state), _ptr(out),
                                             _stream(qkv)),
           "gdn_prefill_chunked_noalloc")


def inproj_pack(shape, wq, scales, biases, group: int):
    """Repack affine 4-bit weights (MLX layout: codes int32 [C + 2 hv][hidden/8],
    bf16 scales and biases [C + 2 hv][hidden/group]) into the tiled layout of
    the in-projection kernels; returns (wq_tiled, scales_tiled, biases_tiled)."""
    for t, dt, nm in ((wq, torch.int32, "wq"), (scales, torch.bfloat16, "scales"),
                      (biases, torch.bfloat16, "biases")):
        _dev(t, dt, nm)
    sh = _shape(shape)
    np_ = int(lib().gdn_inproj_padded_features(C.byref(sh)))
    if np_ < 0:
        raise ValueError("bad shape")
    hidden = wq.shape[1] * 8
    wt = torch.empty(np_ * hidden // 8, dtype=torch.int32, device=wq.device)
    st = torch.empty(np_ * hidden // group, dtype=torch.bfloat16, device=wq.device)
    bt = torch.empty_like(st)
    _check(lib().gdn_inproj_pack_affine4(C.byref(sh), hidden, int(group), _ptr(wq), _ptr(scales), _ptr(biases),
                                         _ptr(wt), _ptr(st), _ptr(bt), _stream(wq)), "gdn_inproj_pack_affine4")
    return wt, st, bt


def inproj_affine4(shape, x, wq, scales, biases, qkv, a, b, group: int):
    """The affine 4-bit in-projection: qkv, a, b (bf16, written) from hidden
    rows x (bf16 [R][hidden]) and the tiled weights of ``inproj_pack``."""
    for t, dt, nm in ((x, torch.bfloat16, "x"), (wq, torch.int32, "wq"), (scales, torch.bfloat16, "scales"),
                      (biases, torch.bfloat16, "biases"), (qkv, torch.bfloat16, "qkv"),
                      (a, torch.bfloat16, "a"), (b, torch.bfloat16, "b")):
        _dev(t, dt, nm)
    sh = _shape(shape)
    _check(lib().gdn_inproj_affine4(C.byref(sh), x.shape[0], x.shape[1], int(group), _ptr(x), _ptr(wq),
                                    _ptr(scales), _ptr(biases), _ptr(qkv), _ptr(a), _ptr(b), _stream(x)),
           "gdn_inproj_affine4")


# ---- attention layers -------------------------------------------------------
#
# These calls sit in latency-bound loops: the checks are one expression a tensor
# (what is wrong is worked out only when one fails), structs are packed bytes,
# and the stream comes from torch as its raw handle.

_BF16, _F32, _I32, _F8, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn, torch.uint8
_pack_cache = struct.Struct("PPPPiiiii4x").pack     # gdn_kv_cache
_pack_rope = struct.Struct("Piif4x").pack           # gdn_rope
# the current stream's handle and the current device, of a process that holds device
# tensors already: by torch's raw calls where it has them (a build without a GPU does
# not): 0.2 us a call instead of 1.3
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _wrong(name, t, dtype, dev, size):
    """Raises what is wrong with a tensor that is to be contiguous, of this type,
    on device number ``dev`` and of ``size`` elements (or of that shape)."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise TypeError(f"{name} must be on device cuda:{dev}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must hold {size}, got {tuple(t.shape)}")


def _i32s(name, t, dev, size):
    if t.dtype is not _I32 or t.get_device() != dev or t.numel() != size or not t.is_contiguous():
        _wrong(name, t, _I32, dev, size)
    return t.data_ptr()


def _f32s(name, t, dev, size):
    if t.dtype is not _F32 or t.get_device() != dev or t.numel() != size or not t.is_contiguous():
        _wrong(name, t, _F32, dev, size)
    return t.data_ptr()


def _u8s(name, t, dev, size):
    if t.dtype is not _U8 or t.get_device() != dev or t.numel() != size or not t.is_contiguous():
        _wrong(name, t, _U8, dev, size)
    return t.data_ptr()


def _on(t: torch.Tensor, name: str) -> int:
    dev = t.get_device()
    if dev < 0:
        raise TypeError(f"{name} must be a device tensor")
    return dev


def _launch(dev, fn, *args):
    """A call on torch's current stream of device ``dev``, with ``dev`` current."""
    f = getattr(_lib or lib(), fn)
    if _current_device() == dev:
        status = f(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = f(*args, _raw_stream(dev))
    if status:
        _check(status, fn)


def _cache(dev, k, v, k_scale, v_scale):
    """A packed gdn_kv_cache, its kv heads and channels."""
    if k.dim() != 4:
        raise ValueError(f"k_cache must be [pages][kv heads][page size][d], got {tuple(k.shape)}")
    shape = k.shape
    pages, hkv, page, d = shape
    dtype = k.dtype
    if dtype is not _BF16 and dtype is not _F8 and dtype is not _U8:
        raise TypeError(f"k_cache must be {_BF16}, {_F8} or {_U8} (two 4-bit codes), got {dtype}")
    if k.get_device() != dev or not k.is_contiguous():
        _wrong("k_cache", k, dtype, dev, tuple(shape))
    if v.dtype is not dtype or v.get_device() != dev or v.shape != shape or not v.is_contiguous():
        _wrong("v_cache", v, dtype, dev, tuple(shape))
    if dtype is _BF16:
        if k_scale is not None or v_scale is not None:
            raise ValueError("a bfloat16 cache has no scales")
        return _pack_cache(k.data_ptr(), v.data_ptr(), 0, 0, pages, page, hkv, d, 0), hkv, d
    if k_scale is None or v_scale is None:
        raise ValueError(f"a {str(dtype)[6:]} cache needs k_scale and v_scale")
    rows = pages * hkv * page
    if dtype is _U8:        # MXFP4
        d *= 2
        exps = rows * (d // 32)
        return _pack_cache(k.data_ptr(), v.data_ptr(), _u8s("k_scale", k_scale, dev, exps), _u8s("v_scale", v_scale, dev, exps),
                           pages, page, hkv, d, 4), hkv, d
    return _pack_cache(k.data_ptr(), v.data_ptr(), _f32s("k_scale", k_scale, dev, rows), _f32s("v_scale", v_scale, dev, rows),
                       pages, page, hkv, d, 1), hkv, d


def kv_tables(row_start, kv_len, page_count, free_count, free_pages, block_table, slots, positions, page_size: int,
              parent=None, page_count_out=None, free_count_out=None):
    """Block tables [n][max_blocks] (in place), slots and positions (written) of
    one pass's packed rows, from the streams' lengths and the stack of unused
    pages; the counts are updated in place unless outputs are given."""
    dev = _on(row_start, "row_start")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [streams][blocks]")
    n, blocks = block_table.shape
    total, pages = slots.numel(), free_pages.numel()
    counts = _i32s("page_count", page_count, dev, n)
    free = _i32s("free_count", free_count, dev, 1)
    _launch(dev, "gdn_kv_tables", n, total, page_size, pages, blocks, _i32s("row_start", row_start, dev, n + 1),
            None if parent is None else _i32s("parent", parent, dev, total), _i32s("kv_len", kv_len, dev, n), counts, free,
            _i32s("free_pages", free_pages, dev, pages), _i32s("block_table", block_table, dev, n * blocks),
            _i32s("slots", slots, dev, total), _i32s("positions", positions, dev, total),
            counts if page_count_out is None else _i32s("page_count_out", page_count_out, dev, n),
            free if free_count_out is None else _i32s("free_count_out", free_count_out, dev, 1))


def _heads(dev, name, t, shape):
    """A bf16 [rows][heads][d] view with contiguous channels: address and strides."""
    if t.dtype is not _BF16:
        raise TypeError(f"{name} must be {_BF16}, got {t.dtype}")
    if t.get_device() != dev:
        raise TypeError(f"{name} must be on device cuda:{dev}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    row, head, one = t.stride()
    if one != 1 and t.numel():
        raise ValueError(f"{name}'s channels must be contiguous")
    # a single row's or head's stride is never used, and may be anything
    return t.data_ptr(), row if shape[0] > 1 else 0, head if shape[1] > 1 else 0


def _query(q, d):
    if q.dim() != 3 or q.shape[2] != d:
        raise ValueError(f"q must be [rows][heads][{d}] as the cache, got {tuple(q.shape)}")
    return q.shape


def attn_prep(q, k, v, q_norm, k_norm, inv_freq, positions, slots, q_out, k_cache, v_cache, k_scale=None, v_scale=None,
              eps: float = 1e-6, interleaved: bool = False, rot_scale: float = 1.0):
    """RMS norms of the query and key heads (weights fp32 [d], None: no norm) and
    rotation of their first ``2 * len(inv_freq)`` channels; queries to q_out,
    keys and values to the cache.  q [R][hq][d], k and v [R][hkv][d] may be
    views into one projection's rows."""
    dev = _on(q, "q")
    cache, hkv, d = _cache(dev, k_cache, v_cache, k_scale, v_scale)
    shape = _query(q, d)
    rows, hq, _ = shape
    qp, qr, qh = _heads(dev, "q", q, shape)
    kp, kr, kh = _heads(dev, "k", k, (rows, hkv, d))
    vp, vr, vh = _heads(dev, "v", v, (rows, hkv, d))
    if q_out.dtype is not _BF16 or q_out.get_device() != dev or q_out.shape != shape or not q_out.is_contiguous():
        _wrong("q_out", q_out, _BF16, dev, tuple(shape))
    half = inv_freq.numel()
    _launch(dev, "gdn_attn_prep", cache, rows, hq, qp, qr, qh, kp, kr, kh, vp, vr, vh,
            None if q_norm is None else _f32s("q_norm", q_norm, dev, d),
            None if k_norm is None else _f32s("k_norm", k_norm, dev, d), eps,
            _pack_rope(_f32s("inv_freq", inv_freq, dev, half), 2 * half, 1 if interleaved else 0, rot_scale),
            _i32s("positions", positions, dev, rows), _i32s("slots", slots, dev, rows), q_out.data_ptr())


def attn_workspace_bytes(hq: int, hkv: int, d: int, n_streams: int, total_rows: int, max_rows: int, max_kv: int) -> int:
    """Bytes of workspace that serve every ``attn_window`` call with these heads and
    up to these sizes: any total_rows, max_rows and max_kv that are no larger."""
    return int(lib().gdn_attn_workspace_bytes(_pack_cache(0, 0, 0, 0, 1, 16, hkv, d, 0), int(n_streams), int(total_rows),
                                              int(max_rows), int(max_kv), int(hq)))


def attn_window(row_start, kv_len, block_table, q, k_cache, v_cache, out, workspace, max_kv: int,
                max_rows: int = MAX_WINDOW_ROWS, parent=None, gate=None, k_scale=None, v_scale=None, scale=None):
    """Attention of steps, windows (parent None) and trees over the cache, which
    holds this pass's rows already; ``scale`` of the scores d ** -0.5 unless
    given, ``gate`` (bf16 [R][hq][d], may be a view) applied as sigmoid(gate)."""
    dev = _on(q, "q")
    cache, _, d = _cache(dev, k_cache, v_cache, k_scale, v_scale)
    shape = _query(q, d)
    total, hq, _ = shape
    if block_table.dim() != 2:
        raise ValueError("block_table must be [streams][blocks]")
    n, blocks = block_table.shape
    if q.dtype is not _BF16 or not q.is_contiguous():
        _wrong("q", q, _BF16, dev, tuple(shape))
    if out.dtype is not _BF16 or out.get_device() != dev or out.shape != shape or not out.is_contiguous():
        _wrong("out", out, _BF16, dev, tuple(shape))
    gp, gr, gh = (None, 0, 0) if gate is None else _heads(dev, "gate", gate, shape)
    ws, size = None, 0
    if workspace is not None:
        size = workspace.numel()
        if workspace.dtype is not torch.uint8 or workspace.get_device() != dev or not workspace.is_contiguous():
            _wrong("workspace", workspace, torch.uint8, dev, size)
        ws = workspace.data_ptr()
    _launch(dev, "gdn_attn_window", cache, n, total, max_rows, max_kv, blocks, hq, _i32s("row_start", row_start, dev, n + 1),
            None if parent is None else _i32s("parent", parent, dev, total), _i32s("kv_len", kv_len, dev, n),
            _i32s("block_table", block_table, dev, n * blocks), q.data_ptr(), gp, gr, gh,
            d ** -0.5 if scale is None else scale, out.data_ptr(), ws, size)


def attn_prompt_workspace_bytes(hq: int, hkv: int, d: int, n_streams: int, total_rows: int, max_kv: int) -> int:
    """Bytes of workspace that serve every ``attn_prompt`` call with these heads and
    up to these sizes: any total_rows and max_kv that are no larger."""
    return int(lib().gdn_attn_prompt_workspace_bytes(_pack_cache(0, 0, 0, 0, 1, 16, hkv, d, 0), int(n_streams), int(total_rows),
                                                     int(max_kv), int(hq)))


def attn_prompt(row_start, kv_len, block_table, q, k_cache, v_cache, out, workspace, max_kv: int, gate=None, k_scale=None,
                v_scale=None, scale=None):
    """Causal attention of packed prompts of any lengths over the cache, which holds
    this pass's rows already: row t of stream s sees cache rows up to kv_len[s] + t.
    ``max_kv`` bounds every stream's cached rows and rows; long streams are cut by it
    and by the number of packed rows, so that bounds far above them cost time.
    ``scale`` of the scores d ** -0.5 unless given, ``gate`` (bf16 [R][hq][d], may
    be a view) applied as sigmoid(gate)."""
    dev = _on(q, "q")
    cache, _, d = _cache(dev, k_cache, v_cache, k_scale, v_scale)
    shape = _query(q, d)
    total, hq, _ = shape
    if block_table.dim() != 2:
        raise ValueError("block_table must be [streams][blocks]")
    n, blocks = block_table.shape
    if q.dtype is not _BF16 or not q.is_contiguous():
        _wrong("q", q, _BF16, dev, tuple(shape))
    if out.dtype is not _BF16 or out.get_device() != dev or out.shape != shape or not out.is_contiguous():
        _wrong("out", out, _BF16, dev, tuple(shape))
    gp, gr, gh = (None, 0, 0) if gate is None else _heads(dev, "gate", gate, shape)
    ws, size = None, 0
    if workspace is not None:
        size = workspace.numel()
        ws = _u8s("workspace", workspace, dev, size)
    _launch(dev, "gdn_attn_prompt", cache, n, total, max_kv, blocks, hq, _i32s("row_start", row_start, dev, n + 1),
            _i32s("kv_len", kv_len, dev, n), _i32s("block_table", block_table, dev, n * blocks), q.data_ptr(), gp, gr, gh,
            d ** -0.5 if scale is None else scale, out.data_ptr(), ws, size)


def kv_read(row_start, first, block_table, k_cache, v_cache, k_out, v_out, k_scale=None, v_scale=None):
    """Cached rows read back: packed row ``row_start[s] + t`` of k_out and v_out
    (bf16 [R][hkv][d], written) is cache row ``first[s] + t`` of stream s."""
    dev = _on(row_start, "row_start")
    cache, hkv, d = _cache(dev, k_cache, v_cache, k_scale, v_scale)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [streams][blocks]")
    n, blocks = block_table.shape
    if k_out.dim() != 3:
        raise ValueError(f"k_out must be [rows][kv heads][d], got {tuple(k_out.shape)}")
    total = k_out.shape[0]
    shape = (total, hkv, d)
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        if t.dtype is not _BF16 or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
            _wrong(name, t, _BF16, dev, shape)
    _launch(dev, "gdn_kv_read", cache, n, total, blocks, _i32s("row_start", row_start, dev, n + 1), _i32s("first", first, dev, n),
            _i32s("block_table", block_table, dev, n * blocks), k_out.data_ptr(), v_out.data_ptr())


def attn_commit(row_start, accept_row, kv_len, block_table, k_cache, v_cache, k_scale=None, v_scale=None, parent=None,
                kv_len_out=None, max_rows: int = MAX_WINDOW_ROWS):
    """Each stream's accepted path (the packed row ``accept_row``, -1 = keep none)
    moves to the end of its cached rows; the lengths are updated in place unless
    ``kv_len_out`` is given."""
    dev = _on(row_start, "row_start")
    cache, _, _ = _cache(dev, k_cache, v_cache, k_scale, v_scale)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [streams][blocks]")
    n, blocks = block_table.shape
    # without parents nothing tells the pass's rows, and none of them is read
    total = (1 << 31) - 1 if parent is None else parent.numel()
    lens = _i32s("kv_len", kv_len, dev, n)
    _launch(dev, "gdn_attn_commit", cache, n, total, max_rows, blocks, _i32s("row_start", row_start, dev, n + 1),
            None if parent is None else _i32s("parent", parent, dev, total), _i32s("accept_row", accept_row, dev, n), lens,
            _i32s("block_table", block_table, dev, n * blocks),
            lens if kv_len_out is None else _i32s("kv_len_out", kv_len_out, dev, n))


def check_layout(row_start, max_rows: int, total_rows: int, parent=None):
    """Host-side check of a window / tree layout (CPU int32 tensors or arrays)."""
    import numpy as np
    rs = np.ascontiguousarray(np.asarray(row_start), dtype=np.int32)
    par = None if parent is None else np.ascontiguousarray(np.asarray(parent), dtype=np.int32)
    _check(lib().gdn_check_layout(rs.shape[0] - 1, int(total_rows), int(max_rows),
                                  rs.ctypes.data_as(C.c_void_p),
                                  None if par is None else par.ctypes.data_as(C.c_void_p)),
           "gdn_check_layout")
