"""Thin Python binding of the KDA C ABI (``include/kda.h``).

Argument marshalling only: every step of the operator runs in the CUDA kernels
of ``_build/libkda.so``.  Tensors are torch CUDA tensors (PyTorch supplies the
device memory and the stream); their data pointers are handed to the C entry
points.  If the library has not been built this module raises on first use --
there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libkda.so")

KDA_BF16, KDA_F32 = 0, 1
STATUS = {0: "KDA_OK", 1: "KDA_ERR_NULL", 2: "KDA_ERR_SHAPE", 3: "KDA_ERR_DTYPE",
          4: "KDA_ERR_ALIGN", 5: "KDA_ERR_SEQLENS", 6: "KDA_ERR_UNSUPPORTED",
          7: "KDA_ERR_CUDA", 8: "KDA_ERR_WORKSPACE", 9: "KDA_ERR_TIMEOUT"}
KDA_OK, KDA_ERR_TIMEOUT = 0, 9
WAIT_LIMIT_DEFAULT = 0xFFFFFFFF

EXPORTED = ["kda_prefill", "kda_prefill_recurrent", "kda_prefill_workspace_size",
            "kda_decode_step", "kda_gate_norm", "kda_status_str", "kda_last_error_string",
            "kda_version", "kda_launch_count", "kda_prefill_noalloc", "kda_prefill_snapshot_count",
            "kda_short_conv", "kda_short_conv_step", "kda_kcp_apply", "kda_prefill_records",
            "kda_prefill_scan", "kda_get_last_device_error", "kda_debug_set_wait_limit",
            "kda_prefill_from_host", "kda_prefill_from_host_staging_size",
            "kda_gdn_prefill", "kda_gdn_prefill_recurrent", "kda_gdn_prefill_workspace_size",
            "kda_gdn_decode_step", "kda_qk_norm_rope", "kda_window_prefill", "kda_window_decode"]

_vp = ctypes.c_void_p


class PrefillArgs(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int), ("T_total", ctypes.c_int),
        ("H", ctypes.c_int), ("dk", ctypes.c_int), ("dv", ctypes.c_int),
        ("qkv_dtype", ctypes.c_int),
        ("cu_seqlens", _vp), ("cu_seqlens_host", _vp),
        ("q", _vp), ("k", _vp), ("v", _vp), ("z", _vp), ("beta", _vp), ("A", _vp),
        ("g_min", ctypes.c_float), ("scale", ctypes.c_float), ("qk_l2norm", ctypes.c_int),
        ("S0", _vp), ("o", _vp), ("S_T", _vp),
        ("g_in", _vp), ("norm_w", _vp), ("norm_eps", ctypes.c_float), ("y", _vp),
        ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
        ("snap_interval", ctypes.c_int), ("S_snap", _vp), ("gate_mode", ctypes.c_int),
    ]


class DecodeArgs(ctypes.Structure):
    _fields_ = [
        ("N", ctypes.c_int), ("H", ctypes.c_int), ("dk", ctypes.c_int), ("dv", ctypes.c_int),
        ("num_slots", ctypes.c_int),
        ("q", _vp), ("k", _vp), ("v", _vp), ("z", _vp), ("beta", _vp), ("A", _vp),
        ("g_min", ctypes.c_float), ("scale", ctypes.c_float), ("qk_l2norm", ctypes.c_int),
        ("state", _vp), ("slots", _vp), ("o", _vp),
        ("g_in", _vp), ("norm_w", _vp), ("norm_eps", ctypes.c_float), ("y", _vp),
        ("gate_mode", ctypes.c_int),
    ]


GATES = {"bounded": 0, "softplus": 1}   # kda_gate: K3's bounded gate, Kimi Linear's Softplus gate


class ShortConvArgs(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int), ("T_total", ctypes.c_int), ("channels", ctypes.c_int),
        ("width", ctypes.c_int), ("dtype", ctypes.c_int),
        ("cu_seqlens", _vp), ("cu_seqlens_host", _vp),
        ("x", _vp), ("weight", _vp), ("bias", _vp), ("state_in", _vp), ("state_out", _vp),
        ("y", _vp), ("activation", ctypes.c_int),
    ]


class ShortConvStepArgs(ctypes.Structure):
    _fields_ = [
        ("N", ctypes.c_int), ("channels", ctypes.c_int), ("width", ctypes.c_int), ("num_slots", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("x", _vp), ("weight", _vp), ("bias", _vp), ("state", _vp), ("slots", _vp),
        ("y", _vp), ("activation", ctypes.c_int),
    ]


class GdnPrefillArgs(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int), ("T_total", ctypes.c_int),
        ("Hk", ctypes.c_int), ("Hv", ctypes.c_int), ("dk", ctypes.c_int), ("dv", ctypes.c_int),
        ("qkv_dtype", ctypes.c_int),
        ("cu_seqlens", _vp), ("cu_seqlens_host", _vp),
        ("q", _vp), ("k", _vp), ("v", _vp), ("z", _vp), ("beta", _vp), ("A", _vp),
        ("g_min", ctypes.c_float), ("scale", ctypes.c_float), ("qk_l2norm", ctypes.c_int),
        ("S0", _vp), ("o", _vp), ("S_T", _vp),
        ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t), ("gate_mode", ctypes.c_int),
    ]


class GdnDecodeArgs(ctypes.Structure):
    _fields_ = [
        ("N", ctypes.c_int), ("Hk", ctypes.c_int), ("Hv", ctypes.c_int), ("dk", ctypes.c_int), ("dv", ctypes.c_int),
        ("num_slots", ctypes.c_int),
        ("q", _vp), ("k", _vp), ("v", _vp), ("z", _vp), ("beta", _vp), ("A", _vp),
        ("g_min", ctypes.c_float), ("scale", ctypes.c_float), ("qk_l2norm", ctypes.c_int),
        ("state", _vp), ("slots", _vp), ("o", _vp), ("gate_mode", ctypes.c_int),
    ]


class QkNormRopeArgs(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("d", ctypes.c_int), ("rot", ctypes.c_int),
        ("num_pos", ctypes.c_int), ("dtype", ctypes.c_int),
        ("q", _vp), ("k", _vp), ("q_stride", ctypes.c_long), ("k_stride", ctypes.c_long),
        ("q_weight", _vp), ("k_weight", _vp), ("eps", ctypes.c_float),
        ("cos", _vp), ("sin", _vp), ("positions", _vp), ("interleaved", ctypes.c_int),
        ("q_out", _vp), ("k_out", _vp),
    ]


class WindowPrefillArgs(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int), ("T_total", ctypes.c_int), ("Tk_total", ctypes.c_int),
        ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("d", ctypes.c_int),
        ("window", ctypes.c_int), ("sinks", ctypes.c_int), ("dtype", ctypes.c_int),
        ("cu_seqlens", _vp), ("cu_seqlens_host", _vp), ("cu_seqlens_k", _vp), ("cu_seqlens_k_host", _vp),
        ("q", _vp), ("k", _vp), ("v", _vp),
        ("q_stride", ctypes.c_long), ("k_stride", ctypes.c_long), ("v_stride", ctypes.c_long),
        ("scale", ctypes.c_float), ("o", _vp), ("lse", _vp),
        ("k_cache", _vp), ("v_cache", _vp), ("slots", _vp), ("num_slots", ctypes.c_int), ("cache_rows", ctypes.c_int),
        ("error", _vp),
    ]


class WindowDecodeArgs(ctypes.Structure):
    _fields_ = [
        ("N", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("d", ctypes.c_int),
        ("window", ctypes.c_int), ("sinks", ctypes.c_int), ("dtype", ctypes.c_int),
        ("q", _vp), ("k", _vp), ("v", _vp),
        ("q_stride", ctypes.c_long), ("k_stride", ctypes.c_long), ("v_stride", ctypes.c_long),
        ("scale", ctypes.c_float), ("k_cache", _vp), ("v_cache", _vp),
        ("positions", _vp), ("slots", _vp), ("num_slots", ctypes.c_int), ("cache_rows", ctypes.c_int), ("o", _vp),
    ]


class KDAError(RuntimeError):
    pass


_lib = None


def load_library(path: str = LIB_PATH):
    """Load the compiled library (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"KDA CUDA library not built: {path} is missing "
                          "(run serving_kda_chunked_gated_gb300.build.build())")
    lib = ctypes.CDLL(path)
    lib.kda_prefill.argtypes = [ctypes.POINTER(PrefillArgs), _vp]
    lib.kda_prefill.restype = ctypes.c_int
    lib.kda_prefill_records.argtypes = [ctypes.POINTER(PrefillArgs), _vp]
    lib.kda_prefill_records.restype = ctypes.c_int
    lib.kda_prefill_scan.argtypes = [ctypes.POINTER(PrefillArgs), ctypes.c_int, _vp]
    lib.kda_prefill_scan.restype = ctypes.c_int
    lib.kda_prefill_noalloc.argtypes = [ctypes.POINTER(PrefillArgs), _vp]
    lib.kda_prefill_noalloc.restype = ctypes.c_int
    lib.kda_prefill_recurrent.argtypes = [ctypes.POINTER(PrefillArgs), _vp]
    lib.kda_prefill_recurrent.restype = ctypes.c_int
    lib.kda_prefill_workspace_size.argtypes = [ctypes.POINTER(PrefillArgs)]
    lib.kda_prefill_workspace_size.restype = ctypes.c_size_t
    lib.kda_prefill_snapshot_count.argtypes = [ctypes.POINTER(PrefillArgs)]
    lib.kda_prefill_snapshot_count.restype = ctypes.c_long
    lib.kda_decode_step.argtypes = [ctypes.POINTER(DecodeArgs), _vp]
    lib.kda_kcp_apply.restype = ctypes.c_int
    lib.kda_kcp_apply.argtypes = [_vp, _vp, _vp, ctypes.c_int, ctypes.c_int, ctypes.c_int, _vp]
    lib.kda_short_conv.restype = ctypes.c_int
    lib.kda_short_conv.argtypes = [ctypes.POINTER(ShortConvArgs), _vp]
    lib.kda_short_conv_step.restype = ctypes.c_int
    lib.kda_short_conv_step.argtypes = [ctypes.POINTER(ShortConvStepArgs), _vp]
    lib.kda_decode_step.restype = ctypes.c_int
    lib.kda_gate_norm.argtypes = [_vp, _vp, _vp, ctypes.c_float, _vp, ctypes.c_long,
                                  ctypes.c_int, ctypes.c_int, _vp]
    lib.kda_gate_norm.restype = ctypes.c_int
    lib.kda_status_str.argtypes = [ctypes.c_int]
    lib.kda_status_str.restype = ctypes.c_char_p
    lib.kda_last_error_string.restype = ctypes.c_char_p
    lib.kda_version.restype = ctypes.c_char_p
    lib.kda_launch_count.restype = ctypes.c_uint64
    lib.kda_get_last_device_error.argtypes = [_vp, _vp]
    lib.kda_get_last_device_error.restype = ctypes.c_int
    lib.kda_debug_set_wait_limit.argtypes = [ctypes.c_uint32]
    lib.kda_prefill_from_host.argtypes = [ctypes.POINTER(PrefillArgs), ctypes.c_int, _vp, ctypes.c_size_t, _vp]
    lib.kda_prefill_from_host.restype = ctypes.c_int
    lib.kda_prefill_from_host_staging_size.argtypes = [ctypes.POINTER(PrefillArgs), ctypes.c_int]
    lib.kda_prefill_from_host_staging_size.restype = ctypes.c_size_t
    lib.kda_debug_set_wait_limit.restype = ctypes.c_uint32
    for name, struct in (("kda_gdn_prefill", GdnPrefillArgs), ("kda_gdn_prefill_recurrent", GdnPrefillArgs),
                         ("kda_gdn_decode_step", GdnDecodeArgs), ("kda_qk_norm_rope", QkNormRopeArgs),
                         ("kda_window_prefill", WindowPrefillArgs), ("kda_window_decode", WindowDecodeArgs)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = [ctypes.POINTER(struct), _vp], ctypes.c_int
    lib.kda_gdn_prefill_workspace_size.argtypes = [ctypes.POINTER(GdnPrefillArgs)]
    lib.kda_gdn_prefill_workspace_size.restype = ctypes.c_size_t
    _lib = lib
    return lib


def launch_count() -> int:
    """Kernel launches enqueued by this library from the calling thread so far."""
    return int(load_library().kda_launch_count())


def device_error(workspace=None, stream=None) -> int:
    """``kda_get_last_device_error``: waits for ``stream``, then reads and clears
    the error word of ``workspace`` (a prefill workspace tensor, or the ``error`` of
    ``window_prefill``), or, when ``workspace`` is None, of the array
    ``kda_prefill_noalloc`` uses and of window prefills without one.  Returns
    KDA_OK (0) or KDA_ERR_TIMEOUT (9); raises on any other status."""
    st = load_library().kda_get_last_device_error(_p(workspace), _stream(stream))
    if st not in (KDA_OK, KDA_ERR_TIMEOUT):
        _check(st, "kda_get_last_device_error")
    return st


def set_wait_limit(polls: int) -> int:
    """``kda_debug_set_wait_limit`` (test hook): the poll bound of the prefill
    kernels' waits on copies and MMAs for later launches; WAIT_LIMIT_DEFAULT
    restores the default, 0 makes every such wait give up at once.  Returns the
    previous setting."""
    return int(load_library().kda_debug_set_wait_limit(ctypes.c_uint32(polls)))


def _check(status: int, what: str):
    if status != 0:
        lib = load_library()
        msg = lib.kda_status_str(status).decode()
        if status == 7:
            msg += ": " + lib.kda_last_error_string().decode()
        raise KDAError(f"{what} failed with {STATUS.get(status, status)} ({msg})")


def _p(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_F32
    raise KDAError(f"unsupported dtype {t.dtype}")


def make_prefill_args(q, k, v, z, beta, A, cu_seqlens, cu_seqlens_host, o, S0=None, S_T=None,
                      g_in=None, norm_w=None, y=None, g_min=-5.0, scale=1.0, qk_l2norm=True,
                      norm_eps=1e-6, workspace=None, gate="bounded") -> PrefillArgs:
    """Fill the C argument struct from tensors (no validation beyond dtype mapping)."""
    T, H, dk = q.shape
    dv = v.shape[2]
    cu_host = cu_seqlens_host
    a = PrefillArgs()
    a.num_seqs = int(cu_host.numel() - 1)
    a.T_total, a.H, a.dk, a.dv = int(T), int(H), int(dk), int(dv)
    a.qkv_dtype = _dtype_code(q)
    a.cu_seqlens = cu_seqlens.data_ptr()
    a.cu_seqlens_host = cu_host.data_ptr()
    for name, t in (("q", q), ("k", k), ("v", v), ("z", z), ("beta", beta), ("A", A),
                    ("S0", S0), ("o", o), ("S_T", S_T), ("g_in", g_in), ("norm_w", norm_w),
                    ("y", y)):
        setattr(a, name, t.data_ptr() if t is not None else None)
    a.g_min, a.scale, a.qk_l2norm, a.norm_eps = float(g_min), float(scale), int(bool(qk_l2norm)), float(norm_eps)
    a.gate_mode = GATES[gate]
    if workspace is not None:
        a.workspace = workspace.data_ptr()
        a.workspace_bytes = workspace.numel() * workspace.element_size()
    return a


def prefill_noalloc_raw(args: PrefillArgs, stream=None):
    """``kda_prefill_noalloc``: for callers that cannot allocate device memory.
    The workspace fields of ``args`` are ignored; the library's fixed device
    scratch array is used instead.  Calls on unordered streams race on it."""
    _check(load_library().kda_prefill_noalloc(ctypes.byref(args), _stream(stream)), "kda_prefill_noalloc")


def prefill_workspace_size(args: PrefillArgs) -> int:
    return int(load_library().kda_prefill_workspace_size(ctypes.byref(args)))


def prefill_raw(args: PrefillArgs, stream=None, recurrent: bool = False):
    lib = load_library()
    fn = lib.kda_prefill_recurrent if recurrent else lib.kda_prefill
    _check(fn(ctypes.byref(args), _stream(stream)), "kda_prefill_recurrent" if recurrent else "kda_prefill")


PREFILL_MIN_WORKSPACE = 256   # smallest workspace of the tensor-core path (single-pass schedule)
_WS_CACHE = {}                # workspace="cache": one buffer per device, stream and host thread


def _cache_key(dev):
    """What the calls that share a cached buffer have in common: they follow one another on
    one stream.  Calls of two host threads may interleave their kernels on it."""
    return dev.type, dev.index, torch.cuda.current_stream(dev).cuda_stream, threading.get_ident()


def _cached_workspace(dev, need, cache=None):
    """The workspace="cache" buffer of ``dev``'s current stream and this thread, grown on demand:
    it was allocated on that stream, so a buffer that is replaced goes back to it, behind its last use.
    During a capture a buffer of the graph's own pool instead: a cached one could be
    replaced, and its memory handed on, while the graph still replays."""
    if dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _cached_workspace(dev, need, cache)
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(need, dtype=torch.uint8, device=dev)
    cache = _WS_CACHE if cache is None else cache
    key = _cache_key(dev)
    ws = cache.get(key)
    if ws is None or ws.numel() < need:
        cache[key] = ws = torch.empty(need, dtype=torch.uint8, device=dev)
    return ws


def cached_workspace(dev):
    """The buffer that workspace="cache" uses on ``dev``'s current stream in this thread
    (None before the first such call)."""
    dev = torch.device(dev)
    if dev.index is None:
        dev = torch.device(dev.type, torch.cuda.current_device())
    return _WS_CACHE.get(_cache_key(dev))


def release_workspace_cache():
    """Drop the cached workspaces (their memory returns to torch's allocator)."""
    _WS_CACHE.clear()


_STAGING = {}                 # prefill_from_host: one staging buffer per device, stream and host thread


def prefill_from_host(q, k, v, z, beta, A, S0=None, g_in=None, norm_w=None, out=None, slab=16384,
                      g_min=-5.0, scale=1.0, qk_l2norm=True, norm_eps=1e-6, gate="bounded", stream=None):
    """KDA prefill of one sequence held in (pinned) host memory, results back to
    host memory, through ``kda_prefill_from_host``: the library cuts the sequence
    into slabs of ``slab`` tokens (a multiple of 64) and overlaps the copies with
    the compute.  q, k, v, g_in [T, H, d] bf16 (or f32), z [T, H, d] f32, beta
    [T, H], A [H], S0 [1, H, d, d] or None, all host tensors; out = (o, y, S_T)
    host tensors (y None without g_in), allocated pinned when None.  The device
    staging comes from a cache per device, stream and host thread.  Returns
    (o, S_T, y) on the host once the call's stream has completed.
    """
    T, H, d = q.shape
    dv = v.shape[2]
    dev = torch.device("cuda", torch.cuda.current_device())
    gate_on = g_in is not None
    if out is None:
        out = (torch.empty((T, H, dv), dtype=q.dtype).pin_memory(),
               torch.empty((T, H, dv), dtype=torch.bfloat16).pin_memory() if gate_on else None,
               torch.empty((1, H, d, dv), dtype=torch.float32).pin_memory())
    o_h, y_h, S_h = out
    a = PrefillArgs()
    a.num_seqs, a.T_total, a.H, a.dk, a.dv = 1, int(T), int(H), int(d), int(dv)
    a.qkv_dtype = _dtype_code(q)
    for name, t in (("q", q), ("k", k), ("v", v), ("z", z), ("beta", beta), ("A", A), ("S0", S0),
                    ("o", o_h), ("S_T", S_h), ("g_in", g_in), ("norm_w", norm_w), ("y", y_h)):
        setattr(a, name, t.data_ptr() if t is not None else None)
    a.g_min, a.scale, a.qk_l2norm, a.norm_eps = float(g_min), float(scale), int(bool(qk_l2norm)), float(norm_eps)
    a.gate_mode = GATES[gate]
    lib = load_library()
    need = int(lib.kda_prefill_from_host_staging_size(ctypes.byref(a), int(slab)))
    if need == 0:
        raise ValueError("kda_prefill_from_host: unsupported slab or shape")
    st = _temporary(stream, lambda: _cached_workspace(dev, need, _STAGING))
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    _check(lib.kda_prefill_from_host(ctypes.byref(a), int(slab), st.data_ptr(), st.numel(), _stream(s)),
           "kda_prefill_from_host")
    return o_h, S_h, y_h


def _temporary(stream, make):
    """``make()`` with ``stream`` (None: the current one) current: what a call allocates for itself
    belongs to the stream that uses it, so that its memory is given on behind that use only."""
    with torch.cuda.stream(stream):
        return make()


def _bounds(cu_seqlens, T, dev, stream):
    """Sequence bounds on the device (None: one sequence of T tokens) and their host copy."""
    if cu_seqlens is not None:
        return cu_seqlens, cu_seqlens.to("cpu")
    cu_host = torch.tensor([0, T], dtype=torch.int32)
    return _temporary(stream, lambda: cu_host.to(dev)), cu_host


def snapshot_count(cu_seqlens_host, interval: int) -> int:
    """Rows of the snapshot output for packed sequences (see kda.h)."""
    cu = [int(x) for x in cu_seqlens_host]
    return sum((cu[i + 1] - cu[i]) // interval for i in range(len(cu) - 1))


def prefill(q, k, v, z, beta, A, cu_seqlens=None, S0=None, g_in=None, norm_w=None,
            g_min=-5.0, scale=1.0, qk_l2norm=True, norm_eps=1e-6, want_state=True,
            out=None, stream=None, recurrent=False, workspace=None, snap_interval=0, gate="bounded",
            want_o=True):
    """KDA chunked prefill through ``kda_prefill``.

    q, k, z: [T, H, dk]; v: [T, H, dv]; beta: [T, H]; A: [H]; cu_seqlens: int32
    [N+1] on the device (None = one sequence).  Returns (o, S_T, y), or
    (o, S_T, y, S_snap) when snap_interval > 0 (prefix-cache snapshots).
    """
    T, H, dk = q.shape
    dv = v.shape[2]
    dev = q.device
    cu_seqlens, cu_host = _bounds(cu_seqlens, T, dev, stream)
    N = cu_host.numel() - 1
    o = (out["o"] if out else torch.empty((T, H, dv), dtype=q.dtype, device=dev)) if want_o else None
    S_T = (out["S_T"] if out else torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)) \
        if want_state else None
    y = None
    if g_in is not None:
        y = out["y"] if out else torch.empty((T, H, dv), dtype=torch.bfloat16, device=dev)
    args = make_prefill_args(q, k, v, z, beta, A, cu_seqlens, cu_host, o, S0=S0, S_T=S_T,
                             g_in=g_in, norm_w=norm_w, y=y, g_min=g_min, scale=scale,
                             qk_l2norm=qk_l2norm, norm_eps=norm_eps, gate=gate)
    S_snap = None
    if snap_interval:
        rows = snapshot_count(cu_host.tolist(), snap_interval)
        S_snap = torch.empty((max(rows, 1), H, dk, dv), dtype=torch.float32, device=dev)
        args.snap_interval = int(snap_interval)
        args.S_snap = S_snap.data_ptr()
        S_snap = S_snap[:rows]
    if not recurrent:
        need = prefill_workspace_size(args)
        if need > 0:
            # a caller's workspace is used as given: its size picks the schedule
            # (>= need: chunk-parallel; >= PREFILL_MIN_WORKSPACE: single pass);
            # "cache" reuses one buffer per device, stream and thread, grown on demand
            if isinstance(workspace, str) and workspace == "cache":
                workspace = _temporary(stream, lambda: _cached_workspace(dev, need))
            elif workspace is None:
                workspace = _temporary(stream, lambda: torch.empty(need, dtype=torch.uint8, device=dev))
            args.workspace = workspace.data_ptr()
            args.workspace_bytes = workspace.numel() * workspace.element_size()
    prefill_raw(args, stream=stream, recurrent=recurrent)
    if snap_interval:
        return o, S_T, y, S_snap
    return o, S_T, y


SCAN_ZERO_V = 1   # kda_prefill_scan flag: evaluate with v = 0


class Records:
    """Chunk records of one set of prefill inputs (``kda_prefill_records``),
    kept with their inputs and workspace so that several ``prefill_scan``
    calls can run the state recurrence over them from different S0."""

    def __init__(self, args, keep, workspace, shape):
        self.args, self.keep, self.workspace, self.shape = args, keep, workspace, shape


def prefill_records(q, k, v, z, beta, A, cu_seqlens=None, g_min=-5.0, qk_l2norm=True, gate="bounded",
                    stream=None) -> Records:
    """Plan + prep of the chunk-parallel prefill through ``kda_prefill_records``."""
    T, H, dk = q.shape
    dev = q.device
    cu_seqlens, cu_host = _bounds(cu_seqlens, T, dev, stream)
    args = make_prefill_args(q, k, v, z, beta, A, cu_seqlens, cu_host, None, g_min=g_min,
                             qk_l2norm=qk_l2norm, gate=gate)
    need = prefill_workspace_size(args)
    ws = _temporary(stream, lambda: torch.empty(max(need, 1), dtype=torch.uint8, device=dev))
    args.workspace, args.workspace_bytes = ws.data_ptr(), ws.numel()
    _check(load_library().kda_prefill_records(ctypes.byref(args), _stream(stream)), "kda_prefill_records")
    return Records(args, (q, k, v, z, beta, A, cu_seqlens, cu_host), ws, (T, H, dk, v.shape[2], cu_host.numel() - 1))


def prefill_scan(rec: Records, S0=None, g_in=None, norm_w=None, scale=1.0, norm_eps=1e-6, want_o=True,
                 want_state=True, zero_v=False, stream=None):
    """The state recurrence over ``rec`` through ``kda_prefill_scan``: returns
    (o, S_T, y) exactly as ``prefill`` would for the same inputs and S0
    (with v taken as zero when ``zero_v``)."""
    T, H, dk, dv, N = rec.shape
    dev = rec.workspace.device
    q = rec.keep[0]
    args = PrefillArgs.from_buffer_copy(rec.args)
    o = torch.empty((T, H, dv), dtype=q.dtype, device=dev) if want_o else None
    S_T = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev) if want_state else None
    y = torch.empty((T, H, dv), dtype=torch.bfloat16, device=dev) if g_in is not None else None
    for name, t in (("o", o), ("S0", S0), ("S_T", S_T), ("g_in", g_in), ("norm_w", norm_w), ("y", y)):
        setattr(args, name, t.data_ptr() if t is not None else None)
    args.scale, args.norm_eps = float(scale), float(norm_eps)
    _check(load_library().kda_prefill_scan(ctypes.byref(args), SCAN_ZERO_V if zero_v else 0, _stream(stream)),
           "kda_prefill_scan")
    return o, S_T, y


def make_decode_args(q, k, v, z, beta, A, state, o=None, y=None, g_in=None, norm_w=None,
                     slots=None, g_min=-5.0, scale=1.0, qk_l2norm=True, norm_eps=1e-6,
                     gate="bounded") -> DecodeArgs:
    N, H, dk = q.shape
    a = DecodeArgs()
    a.N, a.H, a.dk, a.dv = int(N), int(H), int(dk), int(v.shape[2])
    a.num_slots = int(state.shape[0])
    for name, t in (("q", q), ("k", k), ("v", v), ("z", z), ("beta", beta), ("A", A),
                    ("state", state), ("slots", slots), ("o", o), ("g_in", g_in),
                    ("norm_w", norm_w), ("y", y)):
        setattr(a, name, t.data_ptr() if t is not None else None)
    a.g_min, a.scale, a.qk_l2norm, a.norm_eps = float(g_min), float(scale), int(bool(qk_l2norm)), float(norm_eps)
    a.gate_mode = GATES[gate]
    return a


def decode_step_raw(args: DecodeArgs, stream=None):
    _check(load_library().kda_decode_step(ctypes.byref(args), _stream(stream)), "kda_decode_step")


def decode_step(q, k, v, z, beta, A, state, g_in=None, norm_w=None, slots=None, want_o=True,
                g_min=-5.0, scale=1.0, qk_l2norm=True, norm_eps=1e-6, stream=None, gate="bounded"):
    """One decode step through ``kda_decode_step``; ``state`` is updated in place.

    Returns (o or None, y or None).
    """
    N, H, _ = q.shape
    dv = v.shape[2]
    o = torch.empty((N, H, dv), dtype=torch.bfloat16, device=q.device) if want_o else None
    y = torch.empty((N, H, dv), dtype=torch.bfloat16, device=q.device) if g_in is not None else None
    args = make_decode_args(q, k, v, z, beta, A, state, o=o, y=y, g_in=g_in, norm_w=norm_w,
                            slots=slots, g_min=g_min, scale=scale, qk_l2norm=qk_l2norm,
                            norm_eps=norm_eps, gate=gate)
    decode_step_raw(args, stream)
    return o, y


def make_short_conv_args(x, weight, y, cu_seqlens, cu_seqlens_host, bias=None, state_in=None,
                         state_out=None, activation=True) -> ShortConvArgs:
    a = ShortConvArgs()
    a.num_seqs = int(cu_seqlens_host.numel() - 1)
    a.T_total, a.channels = int(x.shape[0]), int(x.shape[1])
    a.width = int(weight.shape[1])
    a.dtype = _dtype_code(x)
    a.cu_seqlens, a.cu_seqlens_host = cu_seqlens.data_ptr(), cu_seqlens_host.data_ptr()
    for name, t in (("x", x), ("weight", weight), ("bias", bias), ("state_in", state_in),
                    ("state_out", state_out), ("y", y)):
        setattr(a, name, t.data_ptr() if t is not None else None)
    a.activation = int(bool(activation))
    return a


def short_conv_raw(args: ShortConvArgs, stream=None):
    _check(load_library().kda_short_conv(ctypes.byref(args), _stream(stream)), "kda_short_conv")


def short_conv(x, weight, bias=None, cu_seqlens=None, state_in=None, want_state=True, activation=True,
               stream=None):
    """ShortConv + Swish prologue through ``kda_short_conv``.

    x: [T, C] (bf16 or f32); weight [C, W] f32; bias [C] or None; cu_seqlens int32
    [N+1] on the device (None = one sequence); state_in [N, W-1, C] f32 or None.
    Returns (y [T, C] in x's dtype, state_out [N, W-1, C] or None).
    """
    T, C = x.shape
    W = weight.shape[1]
    dev = x.device
    cu_seqlens, cu_host = _bounds(cu_seqlens, T, dev, stream)
    N = cu_host.numel() - 1
    y = torch.empty_like(x)
    state_out = torch.empty((N, W - 1, C), dtype=torch.float32, device=dev) if (want_state and W > 1) else None
    args = make_short_conv_args(x, weight, y, cu_seqlens, cu_host, bias=bias, state_in=state_in,
                                state_out=state_out, activation=activation)
    short_conv_raw(args, stream)
    return y, state_out


def short_conv_step(x, weight, state, bias=None, slots=None, activation=True, stream=None):
    """One decode step of the prologue through ``kda_short_conv_step``; ``state``
    [S, W-1, C] is updated in place.  Returns y [N, C]."""
    N, C = x.shape
    a = ShortConvStepArgs()
    a.N, a.channels, a.width = int(N), int(C), int(weight.shape[1])
    a.num_slots = int(state.shape[0]) if state is not None else 0
    a.dtype = _dtype_code(x)
    y = torch.empty_like(x)
    for name, t in (("x", x), ("weight", weight), ("bias", bias), ("state", state), ("slots", slots), ("y", y)):
        setattr(a, name, t.data_ptr() if t is not None else None)
    a.activation = int(bool(activation))
    _check(load_library().kda_short_conv_step(ctypes.byref(a), _stream(stream)), "kda_short_conv_step")
    return y


def kcp_apply(M, X, add=None, stream=None):
    """X[h] <- M[h] X[h] + add[h] for every head, in place (``kda_kcp_apply``).
    M [H, d, d], X [H, d, n], add [H, d, n] or None; float32 on the device."""
    H, d, n = X.shape
    _check(load_library().kda_kcp_apply(_p(M), _p(X), _p(add), int(H), int(d), int(n), _stream(stream)),
           "kda_kcp_apply")
    return X


def gate_norm(o, g_in, norm_w=None, eps=1e-6, out=None, stream=None):
    """y = Sigmoid(g_in) * RMSNorm(o) through ``kda_gate_norm`` (rows over the last dim)."""
    dv = o.shape[-1]
    rows = o.numel() // dv
    y = out if out is not None else torch.empty_like(o)
    lib = load_library()
    _check(lib.kda_gate_norm(_p(o), _p(g_in), _p(norm_w), ctypes.c_float(eps), _p(y),
                             ctypes.c_long(rows), int(dv), _dtype_code(o), _stream(stream)),
           "kda_gate_norm")
    return y


# ---------------------------------------------------------------------------
# the hybrid stack's other token mixers.  Each takes stream=None (the current
# stream of its tensors' device) beside the arguments shown.
# ---------------------------------------------------------------------------

def _dense(name, t, shape, dtype, dev):
    """``t``'s address, once it is what the entry point reads: ``shape`` (None: any
    extent), ``dtype``, contiguous, on ``dev``.  None stays None.  (The calls below
    are made once per token and layer: the checks take the shortest way.)"""
    if t is None:
        return None
    if t.dtype is dtype and t.is_contiguous() and t.device == dev:
        have = t.shape
        if have == shape or (len(have) == len(shape) and all(e is None or e == x for e, x in zip(shape, have))):
            return t.data_ptr()
    raise KDAError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on {dev}, "
                   f"got {t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")


def _heads(name, t, shape, dtype, dev):
    """Address and token stride of a [tokens, heads, d] tensor with dense heads:
    contiguous, or a slice of a packed projection."""
    if t.dtype is not dtype or t.device != dev or t.shape != shape:
        raise KDAError(f"{name}: expected {dtype} of shape {tuple(shape)} on {dev}, "
                       f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    n, h, d = shape
    if t.is_contiguous():
        return t.data_ptr(), h * d
    st = t.stride()
    if (d > 1 and st[2] != 1) or (h > 1 and st[1] != d):
        raise KDAError(f"{name}: the heads of a token must be dense, got strides {st}")
    return t.data_ptr(), (st[0] if n > 1 else h * d)


def _int32(name, x):
    """``x``, once it fits the entry point's int: ctypes would keep its low 32 bits."""
    if not -2 ** 31 <= x < 2 ** 31:
        raise KDAError(f"{name} must fit 32 bits, got {x}")
    return x


def _launch(name, args, dev):
    """The entry point ``name`` on the current stream of the tensors' device."""
    fn = getattr(_lib or load_library(), name)
    index = dev.index
    stream = torch._C._cuda_getCurrentRawStream(index)      # current_stream(dev) without the object
    if index == torch._C._cuda_getDevice():
        status = fn(ctypes.byref(args), stream)
    else:
        with torch.cuda.device(dev):
            status = fn(ctypes.byref(args), stream)
    if status != 0:
        _check(status, name)


def _on_stream(f):
    """Runs the call with ``stream`` (when given) current, so that what it allocates
    belongs to the stream that uses it."""
    @functools.wraps(f)
    def call(q, *args, stream=None, **kw):
        if stream is None:
            return f(q, *args, **kw)
        if q.device != stream.device:
            raise KDAError(f"the stream is on {stream.device}, the tensors on {q.device}")
        with torch.cuda.stream(stream):
            return f(q, *args, **kw)
    return call


def _cuda_device(t, name):
    if not t.is_cuda:
        raise KDAError(f"{name} must be a CUDA tensor, got {t.device}")
    return t.device


def _cu_pair(cu, cu_host, total, dev, name="cu_seqlens"):
    """Device and host copy of sequence bounds.  Both None: one sequence, written on the
    device (a copy from here could not be captured).  cu_host None: copied from the device
    (synchronises); a caller who has the lengths on the host passes both and saves that."""
    if cu is None and cu_host is None:
        cu_host = torch.tensor([0, total], dtype=torch.int32)
        cu = torch.zeros(2, dtype=torch.int32, device=dev)
        cu[1:].fill_(total)
    elif cu is None:
        cu = cu_host.to(dev)
    elif cu_host is None:
        cu_host = cu.to("cpu")
    _dense(name, cu, (None,), torch.int32, dev)
    if cu_host.device.type != "cpu" or cu_host.dtype != torch.int32 or not cu_host.is_contiguous() or \
            cu_host.shape != cu.shape or cu.shape[0] < 1:
        raise KDAError(f"{name}_host must be the contiguous int32 host copy of {name}")
    return cu, cu_host


def _gate_code(gate):
    if gate not in GATES:
        raise KDAError(f"gate must be one of {sorted(GATES)}, got {gate!r}")
    return GATES[gate]


@_on_stream
def gdn_prefill(q, k, v, z, beta, A, cu_seqlens=None, cu_seqlens_host=None, S0=None, g_min=-5.0, scale=1.0,
                qk_l2norm=True, want_o=True, want_state=True, out=None, recurrent=False, workspace=None,
                gate="softplus"):
    """Gated delta rule with one decay per value head, over packed sequences, through
    ``kda_gdn_prefill`` (``recurrent=True``: ``kda_gdn_prefill_recurrent``).

    q, k: [T, Hk, 128]; v: [T, Hv, 128], Hv a multiple of Hk (bf16, or float32: the
    per-token recurrence); z, beta: [T, Hv] f32; A: [Hv] f32; cu_seqlens int32 [N+1]
    on the device (None = one sequence) and its host copy; S0 [N, Hv, 128, 128] f32
    or None.  out: {"o": ..., "S_T": ...} to write into.  workspace as for ``prefill``
    (a uint8 tensor; None: one for this call; or "cache": a buffer kept for the calls of
    this thread on this stream, while a graph is captured one of its own).  Returns (o, S_T).
    """
    dev = _cuda_device(q, "q")
    T, Hk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    cu, cu_host = _cu_pair(cu_seqlens, cu_seqlens_host, T, dev)
    N = cu_host.shape[0] - 1
    o = (out["o"] if out else torch.empty((T, Hv, dv), dtype=q.dtype, device=dev)) if want_o else None
    S_T = (out["S_T"] if out else torch.empty((N, Hv, dk, dv), dtype=torch.float32, device=dev)) if want_state else None
    f32 = torch.float32
    a = GdnPrefillArgs(
        N, T, Hk, Hv, dk, dv, _dtype_code(q), cu.data_ptr(), cu_host.data_ptr(),
        _dense("q", q, (T, Hk, dk), q.dtype, dev), _dense("k", k, (T, Hk, dk), q.dtype, dev),
        _dense("v", v, (T, Hv, dv), q.dtype, dev), _dense("z", z, (T, Hv), f32, dev),
        _dense("beta", beta, (T, Hv), f32, dev), _dense("A", A, (Hv,), f32, dev),
        g_min, scale, 1 if qk_l2norm else 0, _dense("S0", S0, (N, Hv, dk, dv), f32, dev),
        _dense("o", o, (T, Hv, dv), q.dtype, dev), _dense("S_T", S_T, (N, Hv, dk, dv), f32, dev),
        None, 0, _gate_code(gate))
    lib = load_library()
    if recurrent:
        _launch("kda_gdn_prefill_recurrent", a, dev)
        return o, S_T
    need = lib.kda_gdn_prefill_workspace_size(ctypes.byref(a))
    if need:
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        elif isinstance(workspace, str):
            if workspace != "cache":
                raise KDAError(f"workspace must be a tensor, None or 'cache', got {workspace!r}")
            workspace = _cached_workspace(dev, need)
        elif workspace.device != dev or not workspace.is_contiguous():
            raise KDAError(f"the workspace must be a contiguous tensor on {dev}")
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _launch("kda_gdn_prefill", a, dev)
    return o, S_T


@_on_stream
def gdn_decode_step(q, k, v, z, beta, A, state, slots=None, g_min=-5.0, scale=1.0, qk_l2norm=True, out=None,
                    gate="softplus"):
    """One decode token per sequence of the scalar-gated delta rule through
    ``kda_gdn_decode_step``; ``state`` [slots, Hv, 128, 128] f32 is updated in place.

    q, k: [N, Hk, 128], v: [N, Hv, 128] bf16; z, beta: [N, Hv] f32; A: [Hv] f32;
    slots int32 [N] or None (row n).  Returns o [N, Hv, 128].
    """
    dev = _cuda_device(q, "q")
    N, Hk, dk = q.shape
    _, Hv, dv = v.shape
    bf, f32 = torch.bfloat16, torch.float32
    o = torch.empty_like(v) if out is None else out
    a = GdnDecodeArgs(
        N, Hk, Hv, dk, dv, state.shape[0],
        _dense("q", q, (N, Hk, dk), bf, dev), _dense("k", k, (N, Hk, dk), bf, dev),
        _dense("v", v, (N, Hv, dv), bf, dev), _dense("z", z, (N, Hv), f32, dev),
        _dense("beta", beta, (N, Hv), f32, dev), _dense("A", A, (Hv,), f32, dev),
        g_min, scale, 1 if qk_l2norm else 0, _dense("state", state, (state.shape[0], Hv, dk, dv), f32, dev),
        _dense("slots", slots, (N,), torch.int32, dev), _dense("out", o, (N, Hv, dv), bf, dev), _gate_code(gate))
    _launch("kda_gdn_decode_step", a, dev)
    return o


@_on_stream
def qk_norm_rope(q, k, cos, sin, positions, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, out=None):
    """RMSNorm of each query and key head and the rotation by position, in one pass,
    through ``kda_qk_norm_rope``.

    q: [T, Hq, d], k: [T, Hkv, d] (bf16 or f32; contiguous, or slices of a packed
    projection), cos, sin: [positions, rot/2] f32, positions: int32 [T];
    q_weight, k_weight: [d] f32 or None.  out: (q_out, k_out) to write into (q and k
    themselves when they are contiguous).  Returns (q_out, k_out), contiguous.
    """
    dev = _cuda_device(q, "q")
    T, Hq, d = q.shape
    Hkv, half = k.shape[1], cos.shape[1]
    dt, f32 = q.dtype, torch.float32
    qo, ko = (torch.empty((T, Hq, d), dtype=dt, device=dev), torch.empty((T, Hkv, d), dtype=dt, device=dev)) \
        if out is None else out
    qp, qs = _heads("q", q, (T, Hq, d), dt, dev)
    kp, ks = _heads("k", k, (T, Hkv, d), dt, dev)
    a = QkNormRopeArgs(
        T, Hq, Hkv, d, 2 * half, _int32("the number of positions", cos.shape[0]), _dtype_code(q), qp, kp, qs, ks,
        _dense("q_weight", q_weight, (d,), f32, dev), _dense("k_weight", k_weight, (d,), f32, dev), eps,
        _dense("cos", cos, (cos.shape[0], half), f32, dev), _dense("sin", sin, (cos.shape[0], half), f32, dev),
        _dense("positions", positions, (T,), torch.int32, dev), 1 if interleaved else 0,
        _dense("q_out", qo, (T, Hq, d), dt, dev), _dense("k_out", ko, (T, Hkv, d), dt, dev))
    _launch("kda_qk_norm_rope", a, dev)
    return qo, ko


def _caches(k_cache, v_cache, Hkv, d, dev):
    if (k_cache is None) != (v_cache is None):
        raise KDAError("k_cache and v_cache are given together")
    if k_cache is None:
        return None, None, 0, 0
    shape = (k_cache.shape[0], k_cache.shape[1], Hkv, d) if len(k_cache.shape) == 4 else (None, None, Hkv, d)
    return (_dense("k_cache", k_cache, shape, torch.bfloat16, dev), _dense("v_cache", v_cache, shape, torch.bfloat16, dev),
            k_cache.shape[0], k_cache.shape[1])


@_on_stream
def window_prefill(q, k, v, window, sinks=0, cu_seqlens=None, cu_seqlens_host=None, cu_seqlens_k=None,
                   cu_seqlens_k_host=None, scale=None, want_lse=False, k_cache=None, v_cache=None, slots=None, out=None,
                   error=None):
    """Causal attention through a sliding window with sinks over packed sequences,
    through ``kda_window_prefill``.

    q: [T, Hq, d] bf16, k, v: [Tk, Hkv, d] bf16 (contiguous, or slices of a packed
    projection), d = 64 or 128, Hq a multiple of Hkv; the query at position p sees
    the keys j <= p with j > p - window or j < sinks.  cu_seqlens bounds the
    queries, cu_seqlens_k the keys (None: the same bounds; a sequence's queries are
    the last of its keys).  scale: d ** -0.5 by default.  k_cache, v_cache
    [num_slots, rows >= sinks + window, Hkv, d] bf16 receive the rows that
    ``window_decode`` goes on from, in slot slots[n] (or n).  error: an int32 tensor of one
    zero that takes the call's error report, for ``device_error(error)``, apart from the other
    callers' (None: the word that ``device_error(None)`` reads).
    Returns o, or (o, lse [T, Hq] f32) with want_lse.
    """
    dev = _cuda_device(q, "q")
    T, Hq, d = q.shape
    Tk, Hkv = k.shape[0], k.shape[1]
    bf = torch.bfloat16
    cu, cu_host = _cu_pair(cu_seqlens, cu_seqlens_host, T, dev)
    if cu_seqlens_k is not None or cu_seqlens_k_host is not None:
        cuk, cuk_host = _cu_pair(cu_seqlens_k, cu_seqlens_k_host, Tk, dev, "cu_seqlens_k")
    elif cu_seqlens is None and cu_seqlens_host is None and Tk != T:
        cuk, cuk_host = _cu_pair(None, None, Tk, dev, "cu_seqlens_k")
    else:
        cuk, cuk_host = cu, cu_host
    if cuk_host.shape != cu_host.shape:
        raise KDAError("cu_seqlens and cu_seqlens_k bound the same sequences")
    N = cu_host.shape[0] - 1
    o = torch.empty((T, Hq, d), dtype=bf, device=dev) if out is None else out
    lse = torch.empty((T, Hq), dtype=torch.float32, device=dev) if want_lse else None
    qp, qs = _heads("q", q, (T, Hq, d), bf, dev)
    kp, ks = _heads("k", k, (Tk, Hkv, d), bf, dev)
    vp, vs = _heads("v", v, (Tk, Hkv, d), bf, dev)
    kc, vc, num_slots, rows = _caches(k_cache, v_cache, Hkv, d, dev)
    a = WindowPrefillArgs(
        N, T, Tk, Hq, Hkv, d, _int32("window", window), _int32("sinks", sinks), KDA_BF16, cu.data_ptr(),
        cu_host.data_ptr(), cuk.data_ptr(), cuk_host.data_ptr(), qp, kp, vp, qs, ks, vs, d ** -0.5 if scale is None else scale,
        _dense("out", o, (T, Hq, d), bf, dev), lse.data_ptr() if want_lse else None, kc, vc,
        _dense("slots", slots, (N,), torch.int32, dev), num_slots, rows, _dense("error", error, (1,), torch.int32, dev))
    _launch("kda_window_prefill", a, dev)
    return (o, lse) if want_lse else o


@_on_stream
def window_decode(q, k, v, k_cache, v_cache, positions, window, sinks=0, slots=None, scale=None, out=None):
    """One decode token per sequence of the windowed attention through
    ``kda_window_decode``: k, v [N, Hkv, d] are written into the ring caches at
    ``positions`` (int32 [N], the tokens before the new one), q [N, Hq, d] attends
    over them.  Returns o [N, Hq, d]; the caches are updated in place.
    """
    dev = _cuda_device(q, "q")
    N, Hq, d = q.shape
    Hkv, bf = k.shape[1], torch.bfloat16
    o = torch.empty((N, Hq, d), dtype=bf, device=dev) if out is None else out
    qp, qs = _heads("q", q, (N, Hq, d), bf, dev)
    kp, ks = _heads("k", k, (N, Hkv, d), bf, dev)
    vp, vs = _heads("v", v, (N, Hkv, d), bf, dev)
    kc, vc, num_slots, rows = _caches(k_cache, v_cache, Hkv, d, dev)
    a = WindowDecodeArgs(
        N, Hq, Hkv, d, _int32("window", window), _int32("sinks", sinks), KDA_BF16, qp, kp, vp, qs, ks, vs,
        d ** -0.5 if scale is None else scale, kc, vc,
        _dense("positions", positions, (N,), torch.int32, dev), _dense("slots", slots, (N,), torch.int32, dev),
        num_slots, rows, _dense("out", o, (N, Hq, d), bf, dev))
    _launch("kda_window_decode", a, dev)
    return o
