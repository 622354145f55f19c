"""ctypes binding of the C ABI in ``include/txl.h`` (argument marshalling only)."""

from __future__ import annotations

import contextlib
import ctypes
import os
import struct
import threading
from typing import NamedTuple

import torch

from . import build as _build

F32 = 0
BF16 = 1

_lock = threading.Lock()
_lib = None

_c_int, _c_size, _c_p, _c_float, _c_u64 = (ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p,
                                           ctypes.c_float, ctypes.c_uint64)


_c_ip = ctypes.POINTER(ctypes.c_int)
_c_ll = ctypes.c_longlong


class TxlError(RuntimeError):
    """A non-zero txl_status returned by the library."""

    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


class KVWindow(ctypes.Structure):
    """txl_kv_window: host-side state of a memory kept as a contiguous window of
    a larger buffer [planes, capacity, d] (capacity >= 2 M + L)."""

    _fields_ = [("start", ctypes.c_int), ("fill", ctypes.c_int), ("capacity", ctypes.c_int),
                ("M", ctypes.c_int)]

    def __repr__(self):
        return (f"KVWindow(start={self.start}, fill={self.fill}, capacity={self.capacity}, "
                f"M={self.M})")


class _PagedKV(ctypes.Structure):
    """txl_paged_kv."""

    _fields_ = [("pool", _c_p), ("table", _c_p), ("begin", _c_p), ("fill", _c_p),
                ("ticket", _c_p)] + [(f, ctypes.c_int) for f in (
                    "layers", "n_pages", "H", "page_rows", "dh", "B", "slots", "dtype")]


class _PagePool(ctypes.Structure):
    """txl_page_pool."""

    _fields_ = [("n_pages", ctypes.c_int), ("n_free", ctypes.c_int), ("free_list", _c_ip),
                ("users", _c_ip)]


class MemState(ctypes.Structure):
    """txl_mem_state: host-side ring-buffer state of one layer's memory."""

    _fields_ = [("head", ctypes.c_int), ("fill", ctypes.c_int), ("capacity", ctypes.c_int)]

    def __repr__(self):
        return f"MemState(head={self.head}, fill={self.fill}, capacity={self.capacity})"


def _debug() -> bool:
    return os.environ.get("TXL_DEBUG_LIB") == "1"


def lib_path() -> str:
    return _build.DEBUG_LIB_PATH if _debug() else _build.LIB_PATH


def lib():
    """Load ``libtxl_gb300.so`` (with TXL_DEBUG_LIB=1 in the environment: the
    debug build ``libtxl_gb300_debug.so``); build it first when the sources are
    newer.

    Raises if it cannot be built or loaded: nothing falls back to another
    implementation."""
    global _lib
    with _lock:
        if _lib is None:
            if os.environ.get("TXL_NO_BUILD") == "1":
                path = lib_path()
            else:
                path = _build.build(debug=_debug())
            if not os.path.exists(path):
                raise TxlError(-5, f"CUDA library missing: {path}")
            L = ctypes.CDLL(path)
            sig = {
                "txl_status_string": (ctypes.c_char_p, [_c_int]),
                "txl_version": (_c_int, []),
                "txl_rel_pos_emb": (_c_int, [_c_p, _c_int, _c_int, _c_int, _c_p]),
                "txl_relattn_workspace_size": (_c_size, [_c_int, _c_int, _c_int, _c_int, _c_int]),
                "txl_relattn_plan": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                              _c_int, _c_size, ctypes.POINTER(_c_int),
                                              ctypes.POINTER(_c_int)]),
                "txl_relattn_fwd": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_int, _c_p, _c_p, _c_p, _c_p,
                                             _c_int, _c_int, _c_int, _c_int, _c_int, _c_float,
                                             _c_int, _c_int, _c_p, _c_size, _c_p]),
                "txl_relattn_fwd_strided": (_c_int, [_c_p, _c_p, _c_p, ctypes.c_longlong, _c_p,
                                                     _c_int, _c_p, _c_p, _c_p, _c_p, _c_int, _c_int,
                                                     _c_int, _c_int, _c_int, _c_float, _c_int,
                                                     _c_int, _c_p, _c_size, _c_p]),
                "txl_kv_window_append": (_c_int, [_c_p, ctypes.POINTER(KVWindow), _c_p, _c_int,
                                                  _c_int, _c_int, _c_int, _c_p]),
                "txl_kv_window_advance": (_c_int, [ctypes.POINTER(KVWindow), _c_int]),
                "txl_qkv_project": (_c_int, [_c_p, _c_p, _c_int, _c_int, _c_int, _c_int, _c_int,
                                             _c_p, _c_p, ctypes.POINTER(KVWindow), _c_p,
                                             ctypes.POINTER(MemState), _c_p]),
                "txl_relattn_bwd_workspace_size": (_c_size, [_c_int, _c_int, _c_int, _c_int]),
                "txl_relattn_bwd": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_int, _c_p, _c_p, _c_p,
                                             _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_int, _c_int,
                                             _c_int, _c_int, _c_int, _c_float, _c_int, _c_p,
                                             _c_size, _c_p]),
                "txl_relattn_fwd_noalloc": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_int, _c_p, _c_p,
                                                     _c_p, _c_p, _c_int, _c_int, _c_int, _c_int,
                                                     _c_int, _c_float, _c_int, _c_int, _c_p]),
                "txl_mem_concat": (_c_int, [_c_p, _c_p, ctypes.POINTER(MemState), _c_p, _c_int,
                                            _c_int, _c_int, _c_int, _c_p]),
                "txl_mem_update": (_c_int, [_c_p, ctypes.POINTER(MemState), _c_p, _c_int, _c_int,
                                            _c_int, _c_int, _c_p]),
                # (the structs txl_paged_kv and txl_rows by address)
                "txl_paged_append": (_c_int, [_c_p, _c_int, _c_int, _c_p, _c_p, ctypes.c_longlong,
                                              _c_int, _c_p, _c_int, _c_p, _c_int, _c_int, _c_p,
                                              _c_p, _c_p]),
                "txl_paged_advance": (_c_int, [_c_p, _c_p, _c_int, _c_int, _c_p, _c_p, _c_p]),
                "txl_paged_copy": (_c_int, [_c_p, _c_p, _c_p, _c_int, _c_p]),
                "txl_relattn_tree_fwd": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_int, _c_p, _c_int,
                                                  _c_p, _c_p, _c_p, ctypes.c_longlong, _c_p, _c_p,
                                                  _c_p, _c_int, _c_float, _c_int, _c_p]),
                "txl_page_pool_init": (_c_int, [ctypes.POINTER(_PagePool), _c_int, _c_ip, _c_ip]),
                "txl_page_pool_alloc": (_c_int, [ctypes.POINTER(_PagePool), _c_ip, _c_int]),
                "txl_page_pool_retain": (_c_int, [ctypes.POINTER(_PagePool), _c_ip, _c_int]),
                "txl_page_pool_release": (_c_int, [ctypes.POINTER(_PagePool), _c_ip, _c_int, _c_ip]),
                "txl_embed_fwd": (_c_int, [_c_p, _c_int, _c_p, _c_ll, _c_p, _c_int, _c_int, _c_int,
                                           _c_float, _c_int, _c_p]),
                "txl_embed_bwd_workspace_size": (_c_size, [_c_int, _c_int, _c_int]),
                "txl_embed_bwd": (_c_int, [_c_p, _c_int, _c_p, _c_ll, _c_p, _c_int, _c_int, _c_int,
                                           _c_float, _c_int, _c_int, _c_int, _c_p, _c_size, _c_p]),
                "txl_logprob_fwd_workspace_size": (_c_size, [_c_int] * 5),
                "txl_logprob_fwd": (_c_int, [_c_p, _c_ll, _c_p, _c_ll, _c_p, _c_int, _c_p, _c_p, _c_p,
                                             _c_p, _c_p, _c_int, _c_int, _c_int, _c_int, _c_float,
                                             _c_int, _c_p, _c_size, _c_p]),
                "txl_logprob_bwd_workspace_size": (_c_size, [_c_int] * 5),
                "txl_logprob_bwd": (_c_int, [_c_p, _c_ll, _c_p, _c_ll, _c_p, _c_int, _c_p, _c_p, _c_p,
                                             _c_p, _c_p, _c_p, _c_int, _c_int, _c_int, _c_float,
                                             _c_int, _c_int, _c_p, _c_size, _c_p]),
                "txl_device_status": (_c_int, [_c_p]),
                "txl_set_wait_limit_ns": (_c_u64, [_c_u64]),
                "txl_debug_wait_timeout": (_c_int, [_c_u64, _c_p]),
                "txl_debug_checks": (_c_int, []),
                "txl_debug_index_probe": (_c_int, [_c_p]),
            }
            for name, (res, args) in sig.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().txl_status_string(int(status)).decode()


def version() -> int:
    return int(lib().txl_version())


def _check(rc: int, what: str):
    if rc != 0:
        raise TxlError(rc, f"{what}: {status_string(rc)} ({rc})")


def _stream(t: torch.Tensor | None = None, stream=None):
    if stream is None:
        dev = t.device if t is not None else torch.device("cuda", torch.cuda.current_device())
        stream = torch.cuda.current_stream(dev)
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dev(t: torch.Tensor, name: str, dtype=None) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library takes device pointers)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _code(dtype: torch.dtype) -> int:
    if dtype == torch.float32:
        return F32
    if dtype == torch.bfloat16:
        return BF16
    raise ValueError(f"unsupported dtype {dtype} (float32 or bfloat16)")


def rel_pos_emb(K: int, d_model: int, dtype=torch.float32, device=None, out=None, stream=None):
    """Sinusoid relative table R [K, d_model]; row rho holds distance K-1-rho."""
    if out is None:
        dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
        out = torch.empty(K, d_model, dtype=dtype, device=dev)
    _check(lib().txl_rel_pos_emb(_dev(out, "R"), int(K), int(d_model), _code(out.dtype),
                                 _stream(out, stream)), "txl_rel_pos_emb")
    return out


def workspace_size(B: int, H: int, L: int, dh: int, n_splits: int) -> int:
    return int(lib().txl_relattn_workspace_size(int(B), int(H), int(L), int(dh), int(n_splits)))


KERNELS = {1: "tc", 2: "decode", 3: "f32", 4: "decode_mma"}


def relattn_plan(B: int, H: int, M: int, L: int, dtype=torch.bfloat16, *, r_rows: int | None = None,
                 dh: int = 64, n_splits: int = 0, workspace_bytes: int = 0):
    """(kernel, splits) that relattn_fwd would use for these sizes: kernel is
    "tc", "decode" (one query, CUDA cores), "decode_mma" (2 to 8 queries,
    warp MMAs) or "f32".  Raises TxlError for sizes the call would reject."""
    kernel, splits = _c_int(0), _c_int(0)
    _check(lib().txl_relattn_plan(int(B), int(H), int(M), int(L),
                                  int(r_rows if r_rows is not None else M + L), int(dh),
                                  _code(dtype), int(n_splits), int(workspace_bytes),
                                  ctypes.byref(kernel), ctypes.byref(splits)), "txl_relattn_plan")
    return KERNELS[kernel.value], splits.value


def _kv_plane_stride(k, v):
    """0 for dense k, v; else the element stride between (b, h) planes when k and
    v are windows [B, H, K, dh] of larger buffers (rows contiguous within a plane,
    planes equally spaced)."""
    if k.is_contiguous() and v.is_contiguous():
        return 0
    B, H, K, dh = k.shape
    for t, name in ((k, "k"), (v, "v")):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (the library takes device pointers)")
        st = t.stride()
        if st[3] != 1 or st[2] != dh or st[0] != H * st[1]:
            raise ValueError(f"{name}: rows of a plane must be contiguous and planes equally "
                             f"spaced (strides {st})")
    if k.stride() != v.stride():
        raise ValueError("k and v must have the same strides")
    return int(k.stride(1))


def relattn_fwd(q, k, v, r, u, v_bias, M: int, scale: float, *, out=None, lse=None,
                n_splits: int = 0, workspace=None, stream=None):
    """Relative-position attention of one layer.

    q [B,H,L,dh]; k, v [B,H,M+L,dh] (memory rows first); r [H,r_rows,dh] in the
    reversed order (row rho = W_kR R_{r_rows-1-rho}); u, v_bias [H,dh].  All
    bf16 (tensor-core path) or all fp32 (CUDA-core path).  k and v may be
    windows of larger buffers (e.g. ``kv_window_view``): rows contiguous, the
    (b, h) planes equally spaced; they then go through txl_relattn_fwd_strided.
    ``lse``: True to return log-sum-exp [B,H,L] (fp32), or a tensor to fill.
    Returns ``out`` or ``(out, lse)``."""
    B, H, L, dh = q.shape
    dt = q.dtype
    code = _code(dt)
    if out is None:
        out = torch.empty_like(q)
    want_lse = lse is not None and lse is not False
    if lse is True:
        lse = torch.empty(B, H, L, dtype=torch.float32, device=q.device)
    lse_ptr = _dev(lse, "lse", torch.float32) if want_lse else None
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr, ws_bytes = _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()
    kv_stride = _kv_plane_stride(k, v)
    if kv_stride == 0:
        rc = lib().txl_relattn_fwd(
            _dev(q, "q", dt), _dev(k, "k", dt), _dev(v, "v", dt), _dev(r, "r", dt),
            int(r.shape[1]), _dev(u, "u", dt), _dev(v_bias, "v_bias", dt), _dev(out, "out", dt),
            lse_ptr, int(B), int(H), int(M), int(L), int(dh), float(scale), code, int(n_splits),
            ws_ptr, int(ws_bytes), _stream(q, stream))
        _check(rc, "txl_relattn_fwd")
    else:
        if k.dtype != dt or v.dtype != dt:
            raise ValueError(f"k and v must be {dt}")
        rc = lib().txl_relattn_fwd_strided(
            _dev(q, "q", dt), k.data_ptr(), v.data_ptr(), kv_stride, _dev(r, "r", dt),
            int(r.shape[1]), _dev(u, "u", dt), _dev(v_bias, "v_bias", dt), _dev(out, "out", dt),
            lse_ptr, int(B), int(H), int(M), int(L), int(dh), float(scale), code, int(n_splits),
            ws_ptr, int(ws_bytes), _stream(q, stream))
        _check(rc, "txl_relattn_fwd_strided")
    return (out, lse) if want_lse else out


def bwd_workspace_size(B: int, H: int, L: int, M: int) -> int:
    """Bytes of device workspace txl_relattn_bwd needs for a segment of L rows
    after a memory of M."""
    return int(lib().txl_relattn_bwd_workspace_size(int(B), int(H), int(L), int(M)))


def relattn_bwd(q, k, v, r, u, v_bias, dout, M: int, scale: float, *, grads=None,
                workspace=None, stream=None):
    """Backward of :func:`relattn_fwd` (bf16 inputs, same layouts) for the
    output gradient ``dout`` [B,H,L,dh].  Returns fp32
    ``(dq, dk, dv, dr, du, dv_bias)`` shaped like q, k, v, r, u, v_bias; dr, du,
    dv_bias are summed over the batch.  ``grads``: a tuple of such tensors to
    fill instead; ``workspace``: a device buffer of at least
    :func:`bwd_workspace_size` bytes (allocated when omitted)."""
    B, H, L, dh = q.shape
    bf = torch.bfloat16
    if grads is None:
        f = lambda t: torch.empty(t.shape, dtype=torch.float32, device=t.device)
        grads = (f(q), f(k), f(v), f(r), f(u), f(v_bias))
    dq, dk, dv, dr, du, dvb = grads
    if workspace is None:
        workspace = torch.empty(max(bwd_workspace_size(B, H, L, M), 256), dtype=torch.uint8,
                                device=q.device)
    f32 = torch.float32
    rc = lib().txl_relattn_bwd(
        _dev(q, "q", bf), _dev(k, "k", bf), _dev(v, "v", bf), _dev(r, "r", bf), int(r.shape[1]),
        _dev(u, "u", bf), _dev(v_bias, "v_bias", bf), _dev(dout, "dout", bf),
        _dev(dq, "dq", f32), _dev(dk, "dk", f32), _dev(dv, "dv", f32), _dev(dr, "dr", f32),
        _dev(du, "du", f32), _dev(dvb, "dv_bias", f32), int(B), int(H), int(M), int(L), int(dh),
        float(scale), BF16, _dev(workspace, "workspace"),
        int(workspace.numel() * workspace.element_size()), _stream(q, stream))
    _check(rc, "txl_relattn_bwd")
    return grads


def relattn_fwd_noalloc(q, k, v, r, u, v_bias, M: int, scale: float, *, out=None, lse=None,
                        n_splits: int = 0, stream=None):
    """relattn_fwd for callers that cannot allocate device memory at call time:
    split-key partial results go to the library's own scratch array (shared by
    all calls; calls that overlap on the GPU race on it).  The C entry point
    allocates nothing; a caller that cannot allocate passes ``out`` (and
    ``lse``) in, otherwise this wrapper creates them."""
    B, H, L, dh = q.shape
    dt = q.dtype
    code = _code(dt)
    if out is None:
        out = torch.empty_like(q)
    want_lse = lse is not None and lse is not False
    if lse is True:
        lse = torch.empty(B, H, L, dtype=torch.float32, device=q.device)
    lse_ptr = _dev(lse, "lse", torch.float32) if want_lse else None
    rc = lib().txl_relattn_fwd_noalloc(
        _dev(q, "q", dt), _dev(k, "k", dt), _dev(v, "v", dt), _dev(r, "r", dt), int(r.shape[1]),
        _dev(u, "u", dt), _dev(v_bias, "v_bias", dt), _dev(out, "out", dt), lse_ptr,
        int(B), int(H), int(M), int(L), int(dh), float(scale), code, int(n_splits),
        _stream(q, stream))
    _check(rc, "txl_relattn_fwd_noalloc")
    return (out, lse) if want_lse else out


def mem_concat(mem, state: MemState, h_new, out=None, stream=None):
    """Extended context [memory (oldest first) ; h_new] as [B, fill+L, d]."""
    B, L, d = h_new.shape
    if out is None:
        out = torch.empty(B, state.fill + L, d, dtype=h_new.dtype, device=h_new.device)
    mem_ptr = _dev(mem, "mem", h_new.dtype) if mem is not None and mem.numel() else None
    h_ptr = _dev(h_new, "h_new") if h_new.numel() else None
    ext_ptr = _dev(out, "ext", h_new.dtype) if out.numel() else None
    _check(lib().txl_mem_concat(ext_ptr, mem_ptr, ctypes.byref(state), h_ptr, int(B), int(L),
                                int(d), _code(h_new.dtype), _stream(h_new, stream)),
           "txl_mem_concat")
    return out


def mem_update(mem, state: MemState, h_new, stream=None):
    """Append h_new [B, L, d] to the ring-buffer memory mem [B, capacity, d];
    advances ``state`` in place."""
    B, L, d = h_new.shape
    mem_ptr = _dev(mem, "mem", h_new.dtype) if mem is not None and mem.numel() else None
    h_ptr = _dev(h_new, "h_new") if h_new.numel() else None
    _check(lib().txl_mem_update(mem_ptr, ctypes.byref(state), h_ptr, int(B),
                                int(L), int(d), _code(h_new.dtype), _stream(h_new, stream)),
           "txl_mem_update")
    return state


def kv_window_append(buf, state: KVWindow, seg, stream=None):
    """Append seg [planes, L, d] behind the memory rows of the window kept in buf
    [planes, capacity, d] (moving the memory to the buffer's front first when the
    rows would not fit); updates ``state.start`` in place."""
    P, L, d = seg.shape
    if buf.shape[0] != P or buf.shape[2] != d or buf.shape[1] != state.capacity:
        raise ValueError("buf must be [planes, capacity, d] matching seg and the state")
    _check(lib().txl_kv_window_append(_dev(buf, "buf", seg.dtype), ctypes.byref(state),
                                      _dev(seg, "seg") if seg.numel() else None, int(P), int(L),
                                      int(d), _code(seg.dtype), _stream(seg, stream)),
           "txl_kv_window_append")
    return state


def qkv_project(h, w, kv_buf, state: KVWindow, q=None, mem=None, mem_state: MemState | None = None,
                stream=None):
    """One layer's projections of the segment h [B, L, d_model] (bf16) by the
    stacked weights w [n_out*H*64, d_model] (W_q, W_kE, W_v rows when q is given,
    else W_kE, W_v): q into q [B, H, L, 64], k and v into the window rows behind
    the memory of kv_buf [2*B*H, capacity, 64] (keys' planes, then values'),
    and, when mem is given, h into the memory ring mem [B, capacity, d_model].
    Updates ``state.start`` and ``mem_state`` in place, as kv_window_append and
    mem_update do."""
    B, L, d = h.shape
    n_out = 3 if q is not None else 2
    if w.shape[1] != d or w.shape[0] % (n_out * 64):
        raise ValueError("w must be [n_out * H * 64, d_model]")
    H = w.shape[0] // (n_out * 64)
    if kv_buf.shape != (2 * B * H, state.capacity, 64):
        raise ValueError("kv_buf must be [2 * B * H, capacity, 64]")
    if q is not None and tuple(q.shape) != (B, H, L, 64):
        raise ValueError("q must be [B, H, L, 64]")
    if (mem is None) != (mem_state is None):
        raise ValueError("mem and mem_state go together")
    _check(lib().txl_qkv_project(_dev(h, "h", torch.bfloat16), _dev(w, "w", torch.bfloat16),
                                 int(B), int(L), int(d), int(H), 64,
                                 _dev(q, "q", torch.bfloat16) if q is not None else None,
                                 _dev(kv_buf, "kv_buf", torch.bfloat16), ctypes.byref(state),
                                 _dev(mem, "mem", torch.bfloat16) if mem is not None else None,
                                 ctypes.byref(mem_state) if mem_state is not None else None,
                                 _stream(h, stream)),
           "txl_qkv_project")
    return state


def kv_window_advance(state: KVWindow, L: int):
    """After attending to the appended segment of L rows: keep the newest M rows."""
    _check(lib().txl_kv_window_advance(ctypes.byref(state), int(L)), "txl_kv_window_advance")
    return state


def kv_window_view(buf, state: KVWindow, L: int, B: int, H: int):
    """The window [memory ; segment] of buf [B*H, capacity, d] as a [B, H, fill+L, d]
    view (no copy), for relattn_fwd."""
    d = buf.shape[2]
    return buf.view(B, H, state.capacity, d)[:, :, state.start:state.start + state.fill + L]


class PagedKV:
    """Keys and values of the memory in pages (txl_paged_kv), for sequences whose
    lengths differ and advance on the device.

    pool [2 * layers, n_pages, H, page_rows, 64] (bf16 or fp32): planes 2l and
    2l + 1 hold layer l's keys and values.  table [B, slots] int32: page ids; a
    sequence's table rows 0 .. slots * page_rows - 1 form a ring.  begin, fill [B]
    int32: table row of its oldest memory row, and how many it holds (both zero
    when omitted).  Holds the tensors, of which the calls below read and write
    the contents, not the tensors themselves; all on one device."""

    def __init__(self, pool, table, begin=None, fill=None):
        if pool.dim() != 5 or pool.shape[0] % 2 or pool.shape[0] == 0:
            raise ValueError("pool must be [2 * layers, n_pages, H, page_rows, 64]")
        if table.dim() != 2:
            raise ValueError("table must be [B, slots]")
        B = table.shape[0]
        zeros = lambda: torch.zeros(B, dtype=torch.int32, device=pool.device)
        begin = zeros() if begin is None else begin
        fill = zeros() if fill is None else fill
        ticket = torch.zeros(1, dtype=torch.int32, device=pool.device)
        self._tensors = pool, table, begin, fill, ticket
        self.layers, self.B, self.slots = pool.shape[0] // 2, B, table.shape[1]
        self.n_pages, self.H, self.page_rows = pool.shape[1:4]
        ints = [(table, "table"), (begin, "begin"), (fill, "fill")]
        for t, name in ints[1:]:
            if tuple(t.shape) != (B,):
                raise ValueError(f"{name} must be [B]")
        self._c = _PagedKV(_dev(pool, "pool"), *(_dev(t, n, torch.int32) for t, n in ints),
                           ticket.data_ptr(), self.layers, self.n_pages, self.H,
                           self.page_rows, pool.shape[4], B, self.slots, _code(pool.dtype))
        self._at = ctypes.addressof(self._c)
        self._dtype, self._index = pool.dtype, pool.get_device()
        for t, name in ints:
            _ptr(t, name, torch.int32, t.shape, self._index)
        self._shape = (B, self.H, pool.shape[4])

    # (not to be replaced: the calls use their addresses)
    pool, table, begin, fill, ticket = (property(lambda self, i=i: self._tensors[i]) for i in range(5))

    @property
    def rows(self) -> int:
        """Table rows of a sequence: the most memory rows it can hold."""
        return self.slots * self.page_rows


# The calls on a paged memory are made once per layer and token: their checks cost
# one comparison each where nothing is wrong.
_rows_struct = struct.Struct("@Pqqq").pack  # txl_rows
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _refuse(t, name: str, dtype, shape, index: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library takes device pointers)")
    if t.get_device() != index:
        raise ValueError(f"{name} is on another device than the memory")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be {list(shape)}, contiguous (rows operands: in the last "
                     f"dimension), got {list(t.shape)} with strides {t.stride()}")


def _ptr(t, name: str, dtype, shape, index: int) -> int:
    """Address of a contiguous tensor of this dtype, shape and device."""
    try:
        if (t.dtype is dtype and t.get_device() == index and t.shape == shape and
                t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, dtype, shape, index)


def _row_operand(t, name: str, shape, mem: PagedKV) -> bytes:
    """txl_rows of a tensor of this shape [..., B, H, N, 64], of the memory's dtype and
    device."""
    try:
        if t.dtype is mem._dtype and t.get_device() == mem._index and t.shape == shape:
            st = t.stride()
            if st[-1] == 1 or t.numel() == 0:
                return _rows_struct(t.data_ptr(), st[-4], st[-3], st[-2])
    except AttributeError:
        pass
    _refuse(t, name, mem._dtype, shape, mem._index)


def _paged_call(mem: PagedKV, name: str, stream, *args):
    """The library's function on the memory's device and (unless given) its current
    stream."""
    index = mem._index
    if stream is None:
        stream = (_raw_stream(index) if _raw_stream is not None
                  else torch.cuda.current_stream(index).cuda_stream)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    fn = getattr(_lib or lib(), name)
    if _current_device() == index:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, stream)
    if rc != 0:
        _check(rc, name)


def _on_stream(mem: PagedKV, stream):
    """Where a call makes its outputs: on its own stream, so that neither their filling
    nor what used their memory before comes after the kernel."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=mem._index)
    return torch.cuda.stream(stream)


def _state_out(mem: PagedKV, state_out):
    begin, fill = (mem.begin, mem.fill) if state_out is None else state_out
    shape = (mem.B,)
    return (_ptr(begin, "begin", torch.int32, shape, mem._index),
            _ptr(fill, "fill", torch.int32, shape, mem._index))


def paged_append(mem: PagedKV, k, v, *, layer: int = 0, n_new=None, rows=None,
                 keep: int | None = None, state_out=None, stream=None):
    """Put rows of k and v behind the memory's rows, in its pages.

    k, v [B, H, N, 64] for one layer, or [n, B, H, N, 64] for layers layer ..
    layer + n - 1 (any positive strides of 16 bytes' multiples, the last dimension dense).  Sequence b takes
    n_new[b] rows (int32 on the device; all when omitted): rows 0, 1, ... of k
    and v, or rows[b, 0], rows[b, 1], ... with rows [B, width] int32 (the accepted
    nodes of a drafted tree); n_new is taken into [0, N], or [0, width].  With ``keep``, the state is advanced to the
    newest ``keep`` rows: in ``mem``, or in the tensors ``state_out`` = (begin,
    fill) instead."""
    B, H, dh = mem._shape
    shape = k.shape
    layers, layer_stride = 1, 0
    if len(shape) == 5:
        layers, layer_stride = shape[0], k.stride(0)
        if layers > 1 and v.stride()[0] != layer_stride:
            raise ValueError("k and v must have the same layer stride")
    if len(shape) not in (4, 5) or shape[-4] != B or shape[-3] != H or shape[-1] != dh:
        raise ValueError(f"k and v must be [B, H, N, dh] or [n, B, H, N, dh] of the memory, got "
                         f"{list(shape)}")
    N = width = shape[-2]
    rows_k, rows_v = _row_operand(k, "k", shape, mem), _row_operand(v, "v", shape, mem)
    index = mem._index
    rows_at = n_at = b_out = f_out = None
    if rows is not None:
        if rows.dim() != 2:
            raise ValueError("rows must be [B, width]")
        width = rows.shape[1]
        rows_at = _ptr(rows, "rows", torch.int32, (B, width), index)
    if n_new is not None:
        n_at = _ptr(n_new, "n_new", torch.int32, (B,), index)
    if keep is not None:
        b_out, f_out = _state_out(mem, state_out)
    elif state_out is not None:
        raise ValueError("state_out needs keep")
    _paged_call(mem, "txl_paged_append", stream, mem._at, layer, layers, rows_k, rows_v, layer_stride, N,
                rows_at, width if rows is not None else 0, n_at, width, keep or 0, b_out, f_out)
    return mem


def paged_advance(mem: PagedKV, n, *, keep: int, max_rows: int | None = None, state_out=None,
                  stream=None):
    """Advance the state of rows appended without ``keep`` (layer by layer):
    sequence b has n[b] new rows (int32 on the device), or n each (an int), and keeps
    its newest ``keep`` rows.  Counts on the device are taken into [0, max_rows], as
    the append takes them into the rows it was given (by default the table's rows).
    Written to ``mem``, or to ``state_out``."""
    n_at, most = None, n
    if not isinstance(n, int):
        n_at, most = _ptr(n, "n", torch.int32, (mem.B,), mem._index), mem.rows
        if max_rows is not None:
            most = max_rows
    elif max_rows is not None and n > max_rows:
        raise ValueError(f"n is more than max_rows = {max_rows}")
    b_out, f_out = _state_out(mem, state_out)
    _paged_call(mem, "txl_paged_advance", stream, mem._at, n_at, most, keep, b_out, f_out)
    return mem


def paged_copy(mem: PagedKV, src, dst, *, stream=None):
    """Copy pages src[i] to pages dst[i] (int32 on the device) in every plane of the
    pool.  No page may be a destination twice, or a source and a destination."""
    if src.dim() != 1:
        raise ValueError("src and dst must be one-dimensional and of one length")
    shape = src.shape
    _paged_call(mem, "txl_paged_copy", stream, mem._at,
                _ptr(src, "src", torch.int32, shape, mem._index),
                _ptr(dst, "dst", torch.int32, shape, mem._index), shape[0])
    return mem


def relattn_tree_fwd(q, k_new, v_new, mem: PagedKV, layer: int, r, u, v_bias, parents, scale: float,
                     *, n_nodes=None, out=None, lse=None, n_splits: int = 0, stream=None):
    """Relative-position attention of a tree of drafted tokens over layer ``layer``
    of a paged memory: node i attends to the memory's rows, to its ancestors and to
    itself, at the distances its depth gives.

    q, k_new, v_new [B, H, N, 64], N <= 64 (any positive strides of 16 bytes' multiples, the last
    dimension dense);
    parents [B, N] (or [N], one tree for all) int32 on the device: an earlier node,
    or -1; r, u, v_bias as for :func:`relattn_fwd`, r [H, r_rows, 64] being
    attended as far as it goes; all of the memory's dtype (bf16 or fp32).
    n_nodes [B] int32: nodes of each sequence (all N when omitted); the rows of
    out and lse behind them are left as they were.  ``out``: a tensor to fill
    ([B, H, N, 64], strides as q's, no row over another); ``lse``: True, or a tensor [B, H, N] fp32.  Those made
    here hold zeros behind n_nodes.
    Returns ``out`` or ``(out, lse)``."""
    B, H, dh = mem._shape
    shape, index, dt = q.shape, mem._index, mem._dtype
    if len(shape) != 4 or shape[0] != B or shape[1] != H or shape[3] != dh:
        raise ValueError(f"q must be [B, H, N, dh] of the memory, got {list(shape)}")
    N = shape[2]
    lse_at = n_at = None
    want_lse = lse is not None and lse is not False
    if out is None or lse is True:
        # (zeros where there may be rows behind n_nodes, which are not written)
        make = torch.empty if n_nodes is None else torch.zeros
        with _on_stream(mem, stream):
            if out is None:
                out = make(shape, dtype=dt, device=q.device)
            if lse is True:
                lse = make(shape[:3], dtype=torch.float32, device=q.device)
    if want_lse:
        lse_at = _ptr(lse, "lse", torch.float32, shape[:3], index)
    if r.dim() != 3:
        raise ValueError("r must be [H, r_rows, 64]")
    r_rows = r.shape[1]
    if n_nodes is not None:
        n_at = _ptr(n_nodes, "n_nodes", torch.int32, (B,), index)
    stride = N if parents.dim() == 2 else 0
    _paged_call(mem, "txl_relattn_tree_fwd", stream, _row_operand(q, "q", shape, mem),
                _row_operand(k_new, "k_new", shape, mem), _row_operand(v_new, "v_new", shape, mem),
                mem._at, layer,
                _ptr(r, "r", dt, (H, r_rows, dh), index), r_rows, _ptr(u, "u", dt, (H, dh), index),
                _ptr(v_bias, "v_bias", dt, (H, dh), index),
                _ptr(parents, "parents", torch.int32, (B, N) if stride else (N,), index), stride, n_at,
                _row_operand(out, "out", shape, mem), lse_at, N, scale, n_splits)
    return (out, lse) if want_lse else out


class PagePool:
    """Host-side accounting of a pool's pages (txl_page_pool): which are free,
    and how many sequences use each."""

    def __init__(self, n_pages: int):
        n = int(n_pages)
        self._arrays = ((ctypes.c_int * max(n, 1))(), (ctypes.c_int * max(n, 1))())
        self._c = _PagePool()
        _check(lib().txl_page_pool_init(ctypes.byref(self._c), n, *self._arrays),
               "txl_page_pool_init")

    @property
    def n_free(self) -> int:
        return self._c.n_free

    def users(self, page: int) -> int:
        if not 0 <= page < self._c.n_pages:
            raise IndexError(page)
        return self._arrays[1][page]

    def alloc(self, n: int) -> list[int]:
        """n pages with one user each; raises TxlError when fewer are free."""
        out = (ctypes.c_int * max(int(n), 1))()
        _check(lib().txl_page_pool_alloc(ctypes.byref(self._c), out, int(n)), "txl_page_pool_alloc")
        return list(out[:int(n)])

    def retain(self, pages):
        """One user more for each page (a fork shares it)."""
        ids = (ctypes.c_int * max(len(pages), 1))(*pages)
        _check(lib().txl_page_pool_retain(ctypes.byref(self._c), ids, len(pages)),
               "txl_page_pool_retain")

    def release(self, pages) -> int:
        """One user less for each page; returns how many became free."""
        ids = (ctypes.c_int * max(len(pages), 1))(*pages)
        freed = ctypes.c_int(0)
        _check(lib().txl_page_pool_release(ctypes.byref(self._c), ids, len(pages),
                                           ctypes.byref(freed)), "txl_page_pool_release")
        return freed.value


# ---------------------------------------------------------------------------
# the model's two ends: token embedding and log probabilities
# ---------------------------------------------------------------------------

_INDEX_BYTES = {torch.int32: 4, torch.int64: 8}
_CODES = {torch.float32: F32, torch.bfloat16: BF16}


def _counts(*n: int) -> tuple:
    """Counts as C ints; one that is none stays as far out of range as an int goes, for the library to refuse
    (ctypes would cut its high bits off)."""
    if max(n) > 0x7fffffff or min(n) < -0x80000000:
        return tuple(max(-0x80000000, min(x, 0x7fffffff)) for x in n)
    return n


def _on_device(index: int, name: str, stream, *args):
    """The library's function on device ``index`` and (unless given) its current stream."""
    if stream is None:
        stream = (_raw_stream(index) if _raw_stream is not None
                  else torch.cuda.current_stream(index).cuda_stream)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    fn = getattr(_lib or lib(), name)
    if _current_device() == index:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, stream)
    if rc != 0:
        _check(rc, name)


def _made_on(index: int, stream):
    """Where a call makes its outputs and workspace: on its own stream."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=index)
    return torch.cuda.stream(stream)


def _cuda_tensor(t, name: str, index: int | None = None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library takes device pointers)")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} is on another device than the table")


def _table(t, name: str) -> tuple[int, int, int, int]:
    """Device, rows, width and row stride of a [V, d] table."""
    if not isinstance(t, torch.Tensor) or t.get_device() < 0:
        _cuda_tensor(t, name)
    shape, strides = t.shape, t.stride()
    if len(shape) != 2:
        raise ValueError(f"{name} must be [rows, d], got {list(shape)}")
    if t.dtype not in _CODES:
        raise ValueError(f"{name}: unsupported dtype {t.dtype} (float32 or bfloat16)")
    rows, d = shape
    if strides[1] != 1 and d > 1:
        raise ValueError(f"{name} must be dense in its last dimension (strides {strides})")
    return t.get_device(), rows, d, strides[0] if rows > 1 else d


def _rows_of(t, name: str, d: int, dtype, index: int) -> tuple[int, int]:
    """Rows and row stride of a [..., d] operand whose rows are equally spaced."""
    if not isinstance(t, torch.Tensor) or t.get_device() != index or index < 0:
        _cuda_tensor(t, name, index)
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) < 1 or shape[-1] != d or d < 1:
        raise ValueError(f"{name} must be [..., {d}], got {list(shape)}")
    n = t.numel() // d
    if n == 0 or t.is_contiguous():
        return n, d
    strides = t.stride()
    if strides[-1] != 1 and d > 1:
        raise ValueError(f"{name} must be dense in its last dimension (strides {strides})")
    stride, run = None, 1
    for size, st in zip(reversed(shape[:-1]), reversed(strides[:-1])):
        if size == 1:
            continue
        if stride is None:
            stride = st
        elif st != stride * run:
            raise ValueError(f"{name} must have equally spaced rows (strides {strides})")
        run *= size
    return n, d if stride is None else stride


def _ids(t, name: str, n: int, index: int) -> tuple[int, int]:
    """Address and index type of n contiguous token ids."""
    if not isinstance(t, torch.Tensor) or t.get_device() != index:
        _cuda_tensor(t, name, index)
    kind = _INDEX_BYTES.get(t.dtype)
    if kind is None:
        raise ValueError(f"{name} must be int32 or int64, got {t.dtype}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must hold {n} ids, contiguous, got {list(t.shape)} with strides "
                         f"{t.stride()}")
    return t.data_ptr(), kind


def _room(workspace, size: int, index: int, stream):
    """A workspace of at least ``size`` bytes: the caller's, or one made here."""
    if workspace is None:
        with _made_on(index, stream):
            workspace = torch.empty(max(size, 256), dtype=torch.uint8,
                                    device=torch.device("cuda", index))
    elif workspace.get_device() != index:
        raise ValueError("workspace is on another device than the table")
    return workspace, _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()


def embed_fwd(tokens, emb, *, scale: float = 1.0, out=None, stream=None):
    """Rows of the table emb [V, d] (bf16 or fp32, rows at any stride) times ``scale`` for the ids
    ``tokens`` (int32 or int64, any shape): [*tokens.shape, d].  -1: a row of zeros."""
    index, V, d, stride = _table(emb, "emb")
    if not isinstance(tokens, torch.Tensor):
        raise TypeError("tokens must be a torch.Tensor")
    n, dtype = tokens.numel(), emb.dtype
    at, kind = _ids(tokens, "tokens", n, index)
    shape = (*tokens.shape, d)
    if out is None:
        with _made_on(index, stream):
            out = torch.empty(shape, dtype=dtype, device=emb.device)
    at_out = _ptr(out, "out", dtype, shape, index)
    if (n | V | d) >> 31:
        n, V, d = _counts(n, V, d)
    _on_device(index, "txl_embed_fwd", stream, at, kind, emb.data_ptr(), stride, at_out, n, V, d, scale,
               _CODES[dtype])
    return out


def embed_bwd_workspace_size(n: int, V: int, d: int) -> int:
    """Bytes of device workspace embed_bwd needs for n tokens."""
    return int(lib().txl_embed_bwd_workspace_size(*_counts(int(n), int(V), int(d))))


def embed_bwd(dout, tokens, V: int, *, scale: float = 1.0, dtype=torch.float32, out=None,
              accumulate: bool = False, workspace=None, stream=None):
    """Gradient [V, d] of the table of :func:`embed_fwd` for dout [*tokens.shape, d] (equally
    spaced rows), in ``dtype`` (or that of ``out``); with ``accumulate`` added to ``out`` (fp32).
    ``workspace``: a device buffer of at least :func:`embed_bwd_workspace_size` bytes (allocated
    when omitted)."""
    for t, name in ((tokens, "tokens"), (dout, "dout")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    n, d, index = tokens.numel(), dout.shape[-1], dout.get_device()
    rows, stride = _rows_of(dout, "dout", d, dout.dtype, index)
    if rows != n:
        raise ValueError(f"dout must have a row for each of the {n} tokens, got {list(dout.shape)}")
    at, kind = _ids(tokens, "tokens", n, index)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        with _made_on(index, stream):
            out = torch.empty(V, d, dtype=dtype, device=dout.device)
    workspace, ws, ws_bytes = _room(workspace, embed_bwd_workspace_size(n, V, d), index, stream)
    _on_device(index, "txl_embed_bwd", stream, at, kind, dout.data_ptr(), stride,
               _ptr(out, "out", out.dtype, (V, d), index), *_counts(n, V, d), scale, _code(dout.dtype),
               _code(out.dtype), int(accumulate), ws, ws_bytes)
    return out


class LogProbs(NamedTuple):
    """What logprob_fwd gives for states [..., d]: logp, lse and entropy [...] (fp32), and the
    largest alternatives top_logp (fp32) and top_ids (int32) [..., top], or None."""

    logp: torch.Tensor | None
    lse: torch.Tensor | None
    entropy: torch.Tensor | None
    top_logp: torch.Tensor | None = None
    top_ids: torch.Tensor | None = None


def logprob_fwd_workspace_size(N: int, V: int, d: int, dtype=torch.bfloat16, *, top: int = 0) -> int:
    """Bytes of device workspace logprob_fwd needs for N states."""
    return int(lib().txl_logprob_fwd_workspace_size(*_counts(int(N), int(V), int(d), int(top)), _code(dtype)))


def logprob_fwd(h, w, targets=None, *, scale: float = 1.0, top: int = 0, out: LogProbs | None = None,
                workspace=None, stream=None) -> LogProbs:
    """Under softmax(scale * h w^T), for each of the states h [..., d] (equally spaced rows) over
    the table w [V, d] (both bf16 or both fp32): the log probability of its target (int32 or
    int64, -1: none, gives 0), the log-sum-exp, the entropy, and the ``top`` (up to 16) most
    probable tokens.  The logits are not kept.  ``out``: a LogProbs of tensors to fill (None
    entries are left out); ``workspace``: a device buffer of at least
    :func:`logprob_fwd_workspace_size` bytes (allocated when omitted)."""
    index, V, d, w_stride = _table(w, "w")
    N, h_stride = _rows_of(h, "h", d, w.dtype, index)
    shape = tuple(h.shape[:-1])
    at, kind = (None, 4) if targets is None else _ids(targets, "targets", N, index)
    if out is None:
        with _made_on(index, stream):
            f = lambda *s: torch.empty(*shape, *s, dtype=torch.float32, device=h.device)
            out = LogProbs(None if targets is None else f(), f(), f(), f(top) if top else None,
                           torch.empty(*shape, top, dtype=torch.int32, device=h.device) if top else None)
    f32 = torch.float32
    at_of = lambda t, name, dt, s: None if t is None else _ptr(t, name, dt, s, index)
    ptrs = [at_of(out.logp, "logp", f32, shape), at_of(out.lse, "lse", f32, shape),
            at_of(out.entropy, "entropy", f32, shape), at_of(out.top_logp, "top_logp", f32, (*shape, top)),
            at_of(out.top_ids, "top_ids", torch.int32, (*shape, top))]
    code = _code(w.dtype)
    size = 0 if workspace is not None else logprob_fwd_workspace_size(N, V, d, w.dtype, top=top)
    workspace, ws, ws_bytes = _room(workspace, size, index, stream)
    _on_device(index, "txl_logprob_fwd", stream, h.data_ptr(), h_stride, w.data_ptr(), w_stride, at,
               kind, *ptrs, *_counts(N, V, d, top), scale, code, ws, ws_bytes)
    return out


def logprob_bwd_workspace_size(N: int, V: int, d: int, dtype=torch.bfloat16, *,
                               grad_dtype=None) -> int:
    """Bytes of device workspace logprob_bwd needs for N states."""
    grad = dtype if grad_dtype is None else grad_dtype
    return int(lib().txl_logprob_bwd_workspace_size(*_counts(int(N), int(V), int(d)), _code(dtype), _code(grad)))


def logprob_bwd(h, w, targets, lse, dlogp, *, entropy=None, dentropy=None, scale: float = 1.0,
                grads=None, grad_dtype=None, workspace=None, stream=None):
    """Gradients (dh, dw) of h and w of :func:`logprob_fwd` for the gradients ``dlogp`` of its log
    probabilities (None with targets None) and ``dentropy`` of its entropies (may be None), from its
    ``lse`` and ``entropy``.  dh has h's type and shape, dw ``grad_dtype`` (w's type when omitted;
    fp32 for bf16 states too).  ``grads``: the tensors to fill instead, None for one that is not
    wanted; ``workspace``: a device buffer of at least :func:`logprob_bwd_workspace_size` bytes
    (allocated when omitted)."""
    index, V, d, w_stride = _table(w, "w")
    N, h_stride = _rows_of(h, "h", d, w.dtype, index)
    shape = tuple(h.shape[:-1])
    at, kind = (None, 4) if targets is None else _ids(targets, "targets", N, index)
    if grads is None:
        with _made_on(index, stream):
            grads = (torch.empty(h.shape, dtype=h.dtype, device=h.device),
                     torch.empty(V, d, dtype=w.dtype if grad_dtype is None else grad_dtype,
                                 device=w.device))
    dh, dw = grads
    grad = w.dtype if dw is None else dw.dtype
    f32 = torch.float32
    at_of = lambda t, name, dt, s: None if t is None else _ptr(t, name, dt, s, index)
    size = (0 if workspace is not None
            else logprob_bwd_workspace_size(N, V, d, w.dtype, grad_dtype=grad))
    workspace, ws, ws_bytes = _room(workspace, size, index, stream)
    _on_device(index, "txl_logprob_bwd", stream, h.data_ptr(), h_stride, w.data_ptr(), w_stride, at,
               kind, _ptr(lse, "lse", f32, shape, index), at_of(entropy, "entropy", f32, shape),
               at_of(dlogp, "dlogp", f32, shape), at_of(dentropy, "dentropy", f32, shape),
               at_of(dh, "dh", w.dtype, h.shape), at_of(dw, "dw", grad, (V, d)), *_counts(N, V, d), scale,
               _code(w.dtype), _code(grad), ws, ws_bytes)
    return dh, dw


def device_status(stream=None) -> int:
    """Synchronise and return (and clear) the kernels' device status word."""
    return int(lib().txl_device_status(_stream(None, stream)))


def set_wait_limit_ns(ns: int) -> int:
    return int(lib().txl_set_wait_limit_ns(int(ns)))


def debug_wait_timeout(ns: int, stream=None) -> int:
    return int(lib().txl_debug_wait_timeout(int(ns), _stream(None, stream)))


def debug_checks() -> bool:
    """True when the loaded library is the debug build (device-side index checks)."""
    return bool(lib().txl_debug_checks())


def debug_index_probe(stream=None) -> int:
    """Fail one device-side index check on purpose; returns the status then read
    (TXL_ERR_INDEX = -8 in the debug build, 0 in a release build)."""
    return int(lib().txl_debug_index_probe(_stream(None, stream)))
