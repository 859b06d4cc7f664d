"""Python binding of the HLA-2 C ABI (include/hla2.h).

Argument marshalling only: every step of the computation runs in the CUDA library
``_build/libhla2.so``.  PyTorch provides device memory and streams.  If the library
has not been built, every call raises ``RuntimeError``; there is no other code path.

Tensors given on the CPU are copied to the current CUDA device, processed there and
copied back (the end-to-end path); CUDA tensors are processed in place on the
current stream.

The calls around a layer take a few microseconds on the GPU; their ordinary forms are marshalled by
a compiled module (csrc/host_calls.cpp) which calls the same library.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.machinery
import importlib.util
import os
import struct
import threading
import warnings
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libhla2.so")

HLA2_F32 = 0
HLA2_BF16 = 1
_DTYPES = {torch.float32: HLA2_F32, torch.bfloat16: HLA2_BF16}

_lib = None
_lib_lock = threading.Lock()


class HLA2Error(RuntimeError):
    """A C-ABI call returned an error code."""

    def __init__(self, func, code, message):
        super().__init__(f"{func} failed with code {code}: {message}")
        self.code = code


class Opts(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int),
        ("eps", ctypes.c_float),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("init_state", ctypes.c_void_p),
        ("final_state", ctypes.c_void_p),
        ("phase_events", ctypes.POINTER(ctypes.c_void_p)),
        ("n_phase_events", ctypes.c_int),
        ("flags", ctypes.c_int),
    ]


class View(ctypes.Structure):
    """Base address and element strides of batch, head and token (hla2_view)."""
    _fields_ = [("p", ctypes.c_void_p), ("sb", ctypes.c_longlong), ("sh", ctypes.c_longlong),
                ("sn", ctypes.c_longlong)]


_SIZE_MAX = ctypes.c_size_t(-1).value

FLAG_SAVE_FOR_BACKWARD = 1
FLAG_STATES_SAVED = 2


class SavedForBackward:
    """What a training-step forward keeps for the backward on the same inputs: a device
    workspace holding the segment summaries and the bf16 (S, Z) at every chunk start.
    Pass it to backward(saved=...) once; the buffer is owned by this object."""

    def __init__(self, ws, nbytes, key):
        self.ws, self.nbytes, self.key = ws, nbytes, key


def lib():
    """Load libhla2.so (once).  Raises RuntimeError when it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lib_lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"HLA-2 CUDA library not found at {LIB_PATH}; build it with "
                "`python -m chunked_scan_mixer_gb300.build` (there is no fallback)")
        L = ctypes.CDLL(LIB_PATH)
        P, I, Z, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
        L.hla2_version.restype = I
        L.hla2_last_error.restype = ctypes.c_char_p
        L.hla2_state_floats.argtypes = [I, I]
        L.hla2_state_floats.restype = Z
        L.hla2_forward_workspace_bytes.argtypes = [I, I, I, I, I, I, I, I, I]
        L.hla2_forward_workspace_bytes.restype = Z
        L.hla2_forward.argtypes = [P, P, P, P, I, I, I, I, I, P, I, I, P, ctypes.POINTER(Opts)]
        L.hla2_forward.restype = I
        L.hla2_forward_plan.argtypes = [I, I, I, I, I, I, I, I, I, ctypes.POINTER(I), ctypes.POINTER(I),
                                        ctypes.POINTER(I)]
        L.hla2_forward_plan.restype = I
        L.hla2_workspace_status.argtypes = [P, P]
        L.hla2_workspace_status.restype = I
        L.hla2_backward_workspace_bytes.argtypes = [I, I, I, I, I, I, I, I]
        L.hla2_backward_workspace_bytes.restype = Z
        L.hla2_backward.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, P, I, I, P, ctypes.POINTER(Opts)]
        L.hla2_backward.restype = I
        L.hla2_decode_step.argtypes = [P, P, P, P, P, I, I, I, I, P, I, P, ctypes.POINTER(Opts)]
        L.hla2_decode_step.restype = I
        L.hla2_forward_noalloc.argtypes = [P, P, P, P, I, I, I, I, I, P, I, I, I, F, P]
        L.hla2_forward_noalloc.restype = I
        L.hla2_noalloc_status.argtypes = [P]
        L.hla2_noalloc_status.restype = I
        L.hla2_noalloc_selftest_wait_timeout.argtypes = [P]
        L.hla2_noalloc_selftest_wait_timeout.restype = I
        L.hla2_debug_status.argtypes = [I]
        L.hla2_debug_status.restype = I
        L.hla2_debug_selftest.argtypes = [P]
        L.hla2_debug_selftest.restype = I
        L.hla2_ahla_forward_workspace_bytes.argtypes = [I, I, I, I, I, I, I, I]
        L.hla2_ahla_forward_workspace_bytes.restype = Z
        L.hla2_ahla_forward.argtypes = [P, P, P, P, I, I, I, I, I, P, I, I, P, ctypes.POINTER(Opts)]
        L.hla2_ahla_forward.restype = I
        L.hla2_ahla_state_floats.argtypes = [I, I]
        L.hla2_ahla_state_floats.restype = Z
        L.hla2_ahla_decode_step.argtypes = [P, P, P, P, P, I, I, I, I, P, I, P, ctypes.POINTER(Opts)]
        L.hla2_ahla_decode_step.restype = I
        L.hla2_compact_state_floats.argtypes = [I, I]
        L.hla2_compact_state_floats.restype = Z
        L.hla2_hla3_forward_workspace_bytes.argtypes = [I, I, I, I, I, I, I, I, I]
        L.hla2_hla3_forward_workspace_bytes.restype = Z
        L.hla2_hla3_forward.argtypes = [P, P, P, P, I, I, I, I, I, P, I, I, P, ctypes.POINTER(Opts)]
        L.hla2_hla3_forward.restype = I
        L.hla2_ahla_backward_workspace_bytes.argtypes = [I, I, I, I, I, I, I, I]
        L.hla2_ahla_backward_workspace_bytes.restype = Z
        L.hla2_ahla_backward.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, P, I, I, P, ctypes.POINTER(Opts)]
        L.hla2_ahla_backward.restype = I
        L.hla2_hla3_decode_step.argtypes = [P, P, P, P, P, I, I, I, I, I, P, ctypes.POINTER(Opts)]
        L.hla2_hla3_decode_step.restype = I
        L.hla2_selftest_wait_timeout.argtypes = [P, P]
        L.hla2_selftest_wait_timeout.restype = I
        L.hla2_mq_head_state_floats.argtypes = [I, I]
        L.hla2_mq_head_state_floats.restype = Z
        L.hla2_decode_step_mq.argtypes = [P, P, P, P, P, P, I, I, I, I, I, P, I, P, ctypes.POINTER(Opts)]
        L.hla2_decode_step_mq.restype = I
        L.hla2_linattn_workspace_bytes.argtypes = [P, I, I]
        L.hla2_linattn_workspace_bytes.restype = Z
        L.hla2_linattn_forward.argtypes = [P, View, P, P]
        L.hla2_linattn_forward.restype = I
        L.hla2_linattn_backward.argtypes = [P, View, View, View, View, P, P, P]
        L.hla2_linattn_backward.restype = I
        L.hla2_linattn_decode_step.argtypes = [P, P, P, P, P, I, I, I, I, I, P, F, I, P]
        L.hla2_linattn_decode_step.restype = I
        L.hla2_block_join.argtypes = [P, P, P, P]
        L.hla2_block_join.restype = I
        L.hla2_block_join_backward_workspace_bytes.argtypes = [P]
        L.hla2_block_join_backward_workspace_bytes.restype = Z
        L.hla2_block_join_backward.argtypes = [P, P, P, P, P, P, P, P, P, P, Z, P]
        L.hla2_block_join_backward.restype = I
        L.hla2_w4_matvec.argtypes = [P, ctypes.c_longlong, P, P, P, P, P, I, I, I, I, I, P]
        L.hla2_w4_matvec.restype = I
        for name in ("hla2_state_to_compact", "hla2_state_from_compact"):
            getattr(L, name).argtypes = [P, P, I, I, I, I, P]
            getattr(L, name).restype = I
        _lib = L
        _load_host(L)
        return L


HOST_PATH = os.path.join(_HERE, "_build", "_hla2_host.so")
_host = None  # module of csrc/host_calls.cpp


def _load_host(L):
    """The compiled host side of the short calls, bound to the library's entry points; without it (or where it does
    not load, say beside another torch than it was built with) they take the way through this file."""
    global _host
    if not os.path.exists(HOST_PATH):
        return
    try:
        loader = importlib.machinery.ExtensionFileLoader("_hla2_host", HOST_PATH)
        mod = importlib.util.module_from_spec(importlib.util.spec_from_loader("_hla2_host", loader))
        loader.exec_module(mod)
        mod.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            L.hla2_linattn_forward, L.hla2_linattn_backward, L.hla2_linattn_decode_step, L.hla2_block_join,
            L.hla2_block_join_backward, L.hla2_w4_matvec)))
    except Exception as e:
        warnings.warn(f"{HOST_PATH} does not load, short calls take longer on the host: {e}", RuntimeWarning)
        return
    _host = mod


EXPORTED_SYMBOLS = (
    "hla2_version", "hla2_last_error", "hla2_state_floats", "hla2_forward_workspace_bytes",
    "hla2_forward", "hla2_forward_plan", "hla2_workspace_status", "hla2_backward_workspace_bytes",
    "hla2_backward", "hla2_decode_step", "hla2_forward_noalloc", "hla2_compact_state_floats",
    "hla2_state_to_compact", "hla2_state_from_compact", "hla2_ahla_forward_workspace_bytes", "hla2_ahla_forward",
    "hla2_ahla_state_floats", "hla2_ahla_decode_step", "hla2_mq_head_state_floats", "hla2_decode_step_mq",
    "hla2_selftest_wait_timeout", "hla2_hla3_forward_workspace_bytes", "hla2_hla3_forward", "hla2_hla3_decode_step",
    "hla2_ahla_backward_workspace_bytes", "hla2_ahla_backward", "hla2_noalloc_status",
    "hla2_noalloc_selftest_wait_timeout", "hla2_debug_status", "hla2_debug_selftest",
    "hla2_linattn_workspace_bytes", "hla2_linattn_forward", "hla2_linattn_backward", "hla2_linattn_decode_step",
    "hla2_block_join", "hla2_block_join_backward_workspace_bytes", "hla2_block_join_backward", "hla2_w4_matvec",
)

FLAG_COMPACT_STATE = 4
FLAG_UNMASKED = 8


def _check(func, rc):
    if rc != 0:
        raise HLA2Error(func, rc, lib().hla2_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _on_its_device(f):
    """``f`` with the device of its first CUDA tensor made current: the library launches on the current device, and
    the default stream's handle means that device's."""
    @functools.wraps(f)
    def call(*args, **kw):
        for t in (*args, *kw.values()):
            if getattr(t, "is_cuda", False):
                index = t.get_device()
                if index != torch.cuda.current_device():
                    with torch.cuda.device(index):
                        return f(*args, **kw)
                break
        return f(*args, **kw)
    return call


_ws_cache: dict = {}
# The same for the calls around a layer, whose status word nobody clears (_with_scratch)
_scratch_cache: dict = {}

# Held while a call launches the kernels that pass their sums through a cached buffer: ctypes lets other threads run
# during the call, and one of them on the same stream would launch its own kernels on the buffer in between.
_scratch_lock = threading.RLock()


def _alone(fn, *args):
    """Result of a library call on cached scratch, with no other such call's launches in between."""
    with _scratch_lock:
        return fn(*args)


def _workspace(nbytes, device, stream_handle):
    """Scratch reused per (device, stream); grown on demand."""
    if nbytes == 0:
        return None
    key = (device.index, stream_handle.value)
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    return buf


def check_status(device=None):
    """Raise HLA2Error if a kernel that used this stream's cached workspaces reported a
    timed-out wait.  Synchronises the current stream.  (The replays of a captured graph use a workspace of
    the graph's own.)"""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    device = torch.device(device)
    sh = _stream_handle(device)
    index = torch.cuda.current_device() if device.index is None else device.index
    for cache in (_ws_cache, _scratch_cache):
        buf = cache.get((index, sh.value))
        if buf is not None:
            with torch.cuda.device(index):
                _check("hla2_workspace_status", lib().hla2_workspace_status(ctypes.c_void_p(buf.data_ptr()), sh))


def state_floats(d, dv, compact=False):
    """Floats in one head's decode state (packed layout, or the compact one)."""
    return int(lib().hla2_compact_state_floats(d, dv) if compact else lib().hla2_state_floats(d, dv))


@_on_its_device
def _convert_state(src, d, dv, to_compact):
    if src.device.type != "cuda" or src.dtype != torch.float32 or not src.is_contiguous():
        raise ValueError("state must be a contiguous float32 CUDA tensor")
    N, H = src.shape[:2]
    dst = torch.empty((N, H, state_floats(d, dv, compact=to_compact)), dtype=torch.float32, device=src.device)
    fn = lib().hla2_state_to_compact if to_compact else lib().hla2_state_from_compact
    _check(fn.__name__, fn(_ptr(src), _ptr(dst), N, H, d, dv, _stream_handle(src.device)))
    return dst


def state_to_compact(state, d, dv):
    """[N, H, state_floats(d, dv)] packed states -> [N, H, state_floats(d, dv, compact=True)]."""
    return _convert_state(state, d, dv, True)


def state_from_compact(compact, d, dv):
    """Compact states -> packed states (S mirrored from its stored upper block triangle)."""
    return _convert_state(compact, d, dv, False)


def forward_workspace_bytes(B, H, n, d, dv, chunk=64, dtype=torch.bfloat16, normalize=False,
                            want_final_state=False):
    r = lib().hla2_forward_workspace_bytes(B, H, n, d, dv, chunk, _DTYPES[dtype], int(normalize),
                                           int(want_final_state))
    if r == ctypes.c_size_t(-1).value:
        raise ValueError("arguments rejected by hla2_forward")
    return int(r)


def forward_plan(B, H, n, d, dv, chunk=64, dtype=torch.bfloat16, normalize=False, want_final_state=False):
    """(segments per head, chunks per segment, kernel launches per call)."""
    ns, sc, nl = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    _check("hla2_forward_plan", lib().hla2_forward_plan(B, H, n, d, dv, chunk, _DTYPES[dtype], int(normalize),
                                                        int(want_final_state), ctypes.byref(ns),
                                                        ctypes.byref(sc), ctypes.byref(nl)))
    return ns.value, sc.value, nl.value


def _gamma_tensor(gamma, H, device):
    if gamma is None:
        return None
    g = torch.as_tensor(gamma, dtype=torch.float32)
    if g.numel() == 1 and H != 1:
        g = g.reshape(1).expand(H)
    g = g.reshape(H).to(device=device, dtype=torch.float32).contiguous()
    return g


def _to_device(t, device):
    if t is None:
        return None
    if t.device.type == "cuda":
        return t.contiguous()
    return t.contiguous().to(device, non_blocking=True)


_side_streams: dict = {}
HOST_GROUPS = 8  # head groups of the pipelined host-tensor forward


def _pipelined_host_forward(q, k, v, gamma, normalize, chunk, eps, out, masked=True):
    """forward() on host tensors, overlapping the copies with the computation: the heads are
    independent, so they go through in groups -- the inputs of group i+1 are copied in on one
    stream while group i is computed on the current stream and group i-1's output is copied
    out on a third (two device buffers per group slot).  Returns None when the heads cannot
    be cut into at least two groups."""
    B, H, n, d = q.shape
    dv = v.shape[-1]
    # heads per group: a divisor of H giving at least HOST_GROUPS groups (the copies then
    # bound the call to within a group's compute and output copy of the link time), at
    # least two
    divisors = [c for c in range(H, 0, -1) if H % c == 0]
    gh = next((c for c in divisors if B * H // c >= HOST_GROUPS), next((c for c in divisors if B * H // c >= 2), 0))
    if gh == 0 or not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
        return None
    device = torch.device("cuda", torch.cuda.current_device())
    key = device.index
    if key not in _side_streams:
        _side_streams[key] = (torch.cuda.Stream(device=device), torch.cuda.Stream(device=device))
    s_in, s_out = _side_streams[key]
    cur = torch.cuda.current_stream(device)
    g = _gamma_tensor(gamma, H, device)
    res = out if out is not None else torch.empty((B, H, n, dv), dtype=q.dtype, pin_memory=True)
    qf, kf, vf, rf = (t.view(B * H, n, t.shape[-1]) for t in (q, k, v, res))
    stage = [[torch.empty((gh, n, x), dtype=q.dtype, device=device) for x in (d, d, dv, dv)] for _ in range(2)]
    ev_in, ev_comp, ev_out = ([torch.cuda.Event() for _ in range(2)] for _ in range(3))
    s_in.wait_stream(cur)
    s_out.wait_stream(cur)
    for i, r0 in enumerate(range(0, B * H, gh)):
        slot, r1, h0 = i % 2, r0 + gh, r0 % H
        qd, kd, vd, od = stage[slot]
        with torch.cuda.stream(s_in):
            if i >= 2:
                s_in.wait_event(ev_comp[slot])  # group i-2 has read its inputs
            qd.copy_(qf[r0:r1], non_blocking=True)
            kd.copy_(kf[r0:r1], non_blocking=True)
            vd.copy_(vf[r0:r1], non_blocking=True)
            ev_in[slot].record(s_in)
        cur.wait_event(ev_in[slot])
        if i >= 2:
            cur.wait_event(ev_out[slot])  # group i-2's output has left this slot
        forward(qd.view(1, gh, n, d), kd.view(1, gh, n, d), vd.view(1, gh, n, dv),
                gamma=None if g is None else g[h0:h0 + gh], normalize=normalize, chunk=chunk, eps=eps,
                out=od.view(1, gh, n, dv), masked=masked)
        ev_comp[slot].record(cur)
        with torch.cuda.stream(s_out):
            s_out.wait_event(ev_comp[slot])
            rf[r0:r1].copy_(od, non_blocking=True)
            ev_out[slot].record(s_out)
    cur.wait_stream(s_in)
    cur.wait_stream(s_out)
    cur.synchronize()
    return res


@_on_its_device
def forward(q, k, v, gamma=None, normalize=False, chunk=64, eps=1e-6, init_state=None,
            return_final_state=False, out=None, phase_events=None, save_for_backward=False, masked=True):
    """Masked HLA-2 forward.  q, k [B,H,n,d]; v [B,H,n,dv] (float32 or bfloat16).
    masked=False computes the unmasked output q^T S C instead (HLA2_FLAG_UNMASKED).

    gamma: None, a scalar, or [H] per-head decay in (0, 1].  init_state: packed
    [B,H,state_floats] float32 state to continue from.  Returns out [B,H,n,dv] (and the
    packed final state when ``return_final_state``).  phase_events: optional list of
    torch.cuda.Event recorded at the phase boundaries (see hla2_opts).
    save_for_backward: also return a SavedForBackward for backward(saved=...), which then
    skips recomputing the forward (bf16 device tensors, unnormalised, no state arguments)."""
    host = q.device.type == "cpu"
    device = torch.device("cuda", torch.cuda.current_device()) if host else q.device
    L = lib()
    if q.dtype not in _DTYPES or k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must all be float32 or all bfloat16")
    if (host and init_state is None and not return_final_state and phase_events is None and not save_for_backward
            and k.device.type == "cpu" and v.device.type == "cpu" and (out is None or out.device.type == "cpu")):
        res = _pipelined_host_forward(q, k, v, gamma, normalize, chunk, eps, out, masked)
        if res is not None:
            return res
    B, H, n, d = q.shape
    dv = v.shape[-1]
    if k.shape != q.shape or v.shape[:3] != q.shape[:3]:
        raise ValueError("shape mismatch between q, k, v")
    qd, kd, vd = (_to_device(t, device) for t in (q, k, v))
    g = _gamma_tensor(gamma, H, device)
    init = None
    if init_state is not None:
        init = _to_device(init_state, device).to(torch.float32).contiguous()
        if init.shape != (B, H, state_floats(d, dv)):
            raise ValueError("init_state must be [B, H, state_floats(d, dv)]")
    o = out if (out is not None and not host) else torch.empty((B, H, n, dv), dtype=q.dtype, device=device)
    fin = torch.empty((B, H, state_floats(d, dv)), dtype=torch.float32, device=device) \
        if return_final_state else None
    sh = _stream_handle(device)
    flags = 0 if masked else FLAG_UNMASKED
    if save_for_backward:
        if host:
            raise ValueError("save_for_backward needs device tensors")
        nbytes = L.hla2_backward_workspace_bytes(B, H, n, d, dv, chunk, _DTYPES[q.dtype], 0)
        if nbytes == ctypes.c_size_t(-1).value:
            raise HLA2Error("hla2_backward_workspace_bytes", -2, "these arguments have no backward")
        ws = torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)
        flags |= FLAG_SAVE_FOR_BACKWARD
    else:
        nbytes = forward_workspace_bytes(B, H, n, d, dv, chunk, q.dtype, normalize, return_final_state)
        ws = _workspace(nbytes, device, sh)
    opts = Opts(_DTYPES[q.dtype], float(eps), None if ws is None else ws.data_ptr(), nbytes,
                None if init is None else init.data_ptr(), None if fin is None else fin.data_ptr(),
                None, 0, flags)
    if phase_events:
        for e in phase_events:
            if not e.cuda_event:  # torch creates its events lazily
                e.record()
        ev = (ctypes.c_void_p * len(phase_events))(*[e.cuda_event for e in phase_events])
        opts.phase_events = ctypes.cast(ev, ctypes.POINTER(ctypes.c_void_p))
        opts.n_phase_events = len(phase_events)
    rc = _alone(L.hla2_forward, _ptr(qd), _ptr(kd), _ptr(vd), _ptr(o), B, H, n, d, dv, _ptr(g), int(normalize), chunk, sh,
                ctypes.byref(opts))
    _check("hla2_forward", rc)
    if save_for_backward:
        saved = SavedForBackward(ws, int(nbytes), (B, H, n, d, dv, chunk, q.dtype, device))
        return (o, fin, saved) if return_final_state else (o, saved)
    if host:
        o = o.to("cpu") if out is None else out.copy_(o)
        fin = None if fin is None else fin.to("cpu")
    return (o, fin) if return_final_state else o


def ahla_state_floats(d, dv):
    return int(lib().hla2_ahla_state_floats(d, dv))


@_on_its_device
def ahla_forward(q, k, v, gamma=None, normalize=False, chunk=64, eps=1e-6, out=None, phase_events=None,
                 return_final_state=False, init_state=None):
    """Asymmetric HLA forward (the masked left-cascaded product Q (K^T Q)(K^T V)).
    bf16 q, k, v [B,H,n,d] on the GPU (d == dv); chunk 32 or 64 (or 128 at d = 64,
    unnormalised).  Returns out [B,H,n,d] (and, with return_final_state, the state
    [B,H,ahla_state_floats] = P | E | m | n after the last token; a chunk-128 call with a final
    state runs at width 64).
    init_state: a state in that layout to continue from."""
    L = lib()
    if q.device.type != "cuda" or q.dtype != torch.bfloat16 or k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must be bfloat16 CUDA tensors")
    B, H, n, d = q.shape
    dv = v.shape[-1]
    device = q.device
    qd, kd, vd = (t.contiguous() for t in (q, k, v))
    g = _gamma_tensor(gamma, H, device)
    o = out if out is not None else torch.empty((B, H, n, dv), dtype=q.dtype, device=device)
    sh = _stream_handle(device)
    nbytes = L.hla2_ahla_forward_workspace_bytes(B, H, n, d, dv, chunk, _DTYPES[q.dtype], int(normalize))
    if nbytes == ctypes.c_size_t(-1).value:
        nbytes = 0
    ws = _workspace(int(nbytes), device, sh)
    fin = torch.empty((B, H, ahla_state_floats(d, dv)), dtype=torch.float32, device=device) \
        if return_final_state else None
    init = None
    if init_state is not None:
        init = init_state.to(device=device, dtype=torch.float32).contiguous()
        if init.shape != (B, H, ahla_state_floats(d, dv)):
            raise ValueError("init_state must be [B, H, ahla_state_floats(d, dv)]")
    opts = Opts(_DTYPES[q.dtype], float(eps), None if ws is None else ws.data_ptr(), int(nbytes),
                None if init is None else init.data_ptr(), None if fin is None else fin.data_ptr(), None, 0, 0)
    if phase_events:
        for e in phase_events:
            if not e.cuda_event:
                e.record()
        ev = (ctypes.c_void_p * len(phase_events))(*[e.cuda_event for e in phase_events])
        opts.phase_events = ctypes.cast(ev, ctypes.POINTER(ctypes.c_void_p))
        opts.n_phase_events = len(phase_events)
    _check("hla2_ahla_forward", _alone(L.hla2_ahla_forward, _ptr(qd), _ptr(kd), _ptr(vd), _ptr(o), B, H, n, d, dv, _ptr(g),
                                       int(normalize), chunk, sh, ctypes.byref(opts)))
    return (o, fin) if return_final_state else o


@_on_its_device
def ahla_decode_step(state, q, k, v, gamma=None, normalize=False, eps=1e-6, out=None):
    """One AHLA step; ``state`` [N,H,ahla_state_floats] float32 on the GPU is updated in
    place.  q, k [N,H,d]; v [N,H,dv].  Returns out [N,H,dv]."""
    L = lib()
    if state.device.type != "cuda" or state.dtype != torch.float32 or not state.is_contiguous():
        raise ValueError("state must be a contiguous float32 CUDA tensor")
    device = state.device
    N, H, d = q.shape
    dv = v.shape[-1]
    qd, kd, vd = (_to_device(t, device) for t in (q, k, v))
    g = _gamma_tensor(gamma, H, device)
    o = out if out is not None else torch.empty((N, H, dv), dtype=q.dtype, device=device)
    opts = Opts(_DTYPES[q.dtype], float(eps), None, 0, None, None, None, 0, 0)
    _check("hla2_ahla_decode_step", L.hla2_ahla_decode_step(_ptr(state), _ptr(qd), _ptr(kd), _ptr(vd), _ptr(o), N, H,
                                                            d, dv, _ptr(g), int(normalize), _stream_handle(device),
                                                            ctypes.byref(opts)))
    return o


@_on_its_device
def backward(q, k, v, dout, gamma=None, chunk=64, dq=None, dk=None, dv=None, saved=None, normalize=False,
             eps=1e-6):
    """Gradients (dq, dk, dv) for upstream dout of the unnormalised forward, or with
    ``normalize`` of the ratio-normalised one (o / (den + eps)).  saved: the
    SavedForBackward of forward(..., save_for_backward=True) on the same q, k, v, gamma
    and chunk (the forward is then not recomputed; unnormalised only)."""
    host = q.device.type == "cpu"
    device = torch.device("cuda", torch.cuda.current_device()) if host else q.device
    L = lib()
    B, H, n, d = q.shape
    dvdim = v.shape[-1]
    qd, kd, vd, dod = (_to_device(t, device) for t in (q, k, v, dout))
    g = _gamma_tensor(gamma, H, device)
    gq = torch.empty_like(qd) if dq is None or host else dq
    gk = torch.empty_like(kd) if dk is None or host else dk
    gv = torch.empty_like(vd) if dv is None or host else dv
    sh = _stream_handle(device)
    flags = 0
    if saved is not None:
        if saved.key != (B, H, n, d, dvdim, chunk, q.dtype, device):
            raise ValueError("saved was made for other sizes, chunk, dtype or device")
        ws, nbytes, flags = saved.ws, saved.nbytes, FLAG_STATES_SAVED
    else:
        nbytes = L.hla2_backward_workspace_bytes(B, H, n, d, dvdim, chunk, _DTYPES[q.dtype], int(normalize))
        if nbytes == ctypes.c_size_t(-1).value:
            nbytes = 0
        ws = _workspace(int(nbytes), device, sh)
    opts = Opts(_DTYPES[q.dtype], float(eps), None if ws is None else ws.data_ptr(), int(nbytes), None, None,
                None, 0, flags)
    rc = _alone(L.hla2_backward, _ptr(qd), _ptr(kd), _ptr(vd), _ptr(dod), _ptr(gq), _ptr(gk), _ptr(gv), B, H, n, d, dvdim,
                _ptr(g), int(normalize), chunk, sh, ctypes.byref(opts))
    _check("hla2_backward", rc)
    if host:
        return gq.cpu(), gk.cpu(), gv.cpu()
    return gq, gk, gv


@_on_its_device
def decode_step(state, q, k, v, gamma=None, normalize=False, eps=1e-6, out=None, compact=False, masked=True):
    """One decode step; ``state`` [N,H,state_floats(d, dv, compact)] float32 on the GPU is
    updated in place (compact: the block-triangular S layout).  q, k [N,H,d]; v [N,H,dv].
    masked=False: the unmasked output q^T S C (G and h untouched).  Returns out [N,H,dv]."""
    L = lib()
    if state.device.type != "cuda" or state.dtype != torch.float32 or not state.is_contiguous():
        raise ValueError("state must be a contiguous float32 CUDA tensor")
    device = state.device
    N, H, d = q.shape
    dv = v.shape[-1]
    qd, kd, vd = (_to_device(t, device) for t in (q, k, v))
    g = _gamma_tensor(gamma, H, device)
    o = out if out is not None else torch.empty((N, H, dv), dtype=q.dtype, device=device)
    flags = (FLAG_COMPACT_STATE if compact else 0) | (0 if masked else FLAG_UNMASKED)
    opts = Opts(_DTYPES[q.dtype], float(eps), None, 0, None, None, None, 0, flags)
    rc = L.hla2_decode_step(_ptr(state), _ptr(qd), _ptr(kd), _ptr(vd), _ptr(o), N, H, d, dv, _ptr(g),
                            int(normalize), _stream_handle(device), ctypes.byref(opts))
    _check("hla2_decode_step", rc)
    return o


def mq_head_state_floats(d, dv):
    """Floats of one head's part of the multi-query state: C | G | m | h."""
    return int(lib().hla2_mq_head_state_floats(d, dv))


def mq_split_state(state, d, dv, group):
    """Packed per-head states [N, H, state_floats(d, dv)] whose heads share S within groups of
    ``group`` (e.g. a forward's final state on keys repeated over each group's heads) ->
    (key_state [N, H/group, d*d], head_state [N, H, mq_head_state_floats(d, dv)]).  S is
    taken from each group's first head; a layout copy only (the packed order is
    S | C | G | m | h, so a head's part is the tail after S)."""
    N, H, sf = state.shape
    if sf != state_floats(d, dv) or H % group:
        raise ValueError("state must be [N, H, state_floats(d, dv)] with H a multiple of group")
    return state[:, ::group, :d * d].contiguous(), state[:, :, d * d:].contiguous()


def mq_merge_state(key_state, head_state, d, dv):
    """Inverse of mq_split_state: packed per-head states with each group's S repeated."""
    N, Hk, _ = key_state.shape
    H = head_state.shape[1]
    S = key_state.repeat_interleave(H // Hk, dim=1)
    return torch.cat([S, head_state], dim=-1).contiguous()


@_on_its_device
def decode_step_mq(key_state, head_state, q, k, v, gamma=None, normalize=False, eps=1e-6, out=None, masked=True):
    """One decode step with one key moment per key group (multi-query sharing).
    key_state [N,Hk,d*d] and head_state [N,H,mq_head_state_floats(d, dv)] float32 on the GPU
    are updated in place; q [N,H,d] with H = Hk * group; k [N,Hk,d]; v [N,Hk,dv];
    gamma None, a scalar or [Hk].  Returns out [N,H,dv]."""
    L = lib()
    for t in (key_state, head_state):
        if t.device.type != "cuda" or t.dtype != torch.float32 or not t.is_contiguous():
            raise ValueError("states must be contiguous float32 CUDA tensors")
    device = key_state.device
    N, H, d = q.shape
    Hk, dv = k.shape[1], v.shape[-1]
    if H % Hk:
        raise ValueError("the query heads must be a multiple of the key heads")
    group = H // Hk
    qd, kd, vd = (_to_device(t, device) for t in (q, k, v))
    g = _gamma_tensor(gamma, Hk, device)
    o = out if out is not None else torch.empty((N, H, dv), dtype=q.dtype, device=device)
    opts = Opts(_DTYPES[q.dtype], float(eps), None, 0, None, None, None, 0, 0 if masked else FLAG_UNMASKED)
    rc = L.hla2_decode_step_mq(_ptr(key_state), _ptr(head_state), _ptr(qd), _ptr(kd), _ptr(vd), _ptr(o), N, Hk,
                               group, d, dv, _ptr(g), int(normalize), _stream_handle(device), ctypes.byref(opts))
    _check("hla2_decode_step_mq", rc)
    return o


@_on_its_device
def hla3_forward(q, k, v, normalize=False, chunk=64, eps=1e-6, out=None, return_final_state=False):
    """Masked third-order output at gamma = 1 (every factor of A A^T A and the partial product
    of the first two causally masked).  q, k [B,H,n,d]; v [B,H,n,dv] on the GPU, float32 or
    bfloat16.  Returns out [B,H,n,dv] (and with return_final_state the streaming state
    [B,H,state_floats(d, dv)] after the last token, for hla3_decode_step)."""
    L = lib()
    if q.dtype not in _DTYPES or k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must all be float32 or all bfloat16")
    if q.device.type != "cuda":
        raise ValueError("q, k, v must be CUDA tensors")
    B, H, n, d = q.shape
    dv = v.shape[-1]
    device = q.device
    qd, kd, vd = (t.contiguous() for t in (q, k, v))
    o = out if out is not None else torch.empty((B, H, n, dv), dtype=q.dtype, device=device)
    sh = _stream_handle(device)
    nbytes = L.hla2_hla3_forward_workspace_bytes(B, H, n, d, dv, chunk, _DTYPES[q.dtype], int(normalize),
                                                 int(return_final_state))
    if nbytes == ctypes.c_size_t(-1).value:
        nbytes = 0
    ws = _workspace(int(nbytes), device, sh)
    fin = torch.empty((B, H, state_floats(d, dv)), dtype=torch.float32, device=device) if return_final_state else None
    opts = Opts(_DTYPES[q.dtype], float(eps), None if ws is None else ws.data_ptr(), int(nbytes), None,
                None if fin is None else fin.data_ptr(), None, 0, 0)
    _check("hla2_hla3_forward", _alone(L.hla2_hla3_forward, _ptr(qd), _ptr(kd), _ptr(vd), _ptr(o), B, H, n, d, dv, None,
                                       int(normalize), chunk, sh, ctypes.byref(opts)))
    return (o, fin) if return_final_state else o


@_on_its_device
def hla3_decode_step(state, q, k, v, normalize=False, eps=1e-6, out=None):
    """One third-order streaming step (gamma = 1).  state [N,H,state_floats(d, dv)] float32 on
    the GPU, laid out S^K | P^KV | Y | m^K | y, updated in place; q, k [N,H,d]; v [N,H,dv].
    Returns out [N,H,dv]."""
    L = lib()
    if state.device.type != "cuda" or state.dtype != torch.float32 or not state.is_contiguous():
        raise ValueError("state must be a contiguous float32 CUDA tensor")
    device = state.device
    N, H, d = q.shape
    dv = v.shape[-1]
    qd, kd, vd = (_to_device(t, device) for t in (q, k, v))
    o = out if out is not None else torch.empty((N, H, dv), dtype=q.dtype, device=device)
    opts = Opts(_DTYPES[q.dtype], float(eps), None, 0, None, None, None, 0, 0)
    _check("hla2_hla3_decode_step", L.hla2_hla3_decode_step(_ptr(state), _ptr(qd), _ptr(kd), _ptr(vd), _ptr(o), N,
                                                            H, d, dv, int(normalize), _stream_handle(device),
                                                            ctypes.byref(opts)))
    return o


@_on_its_device
def ahla_backward(q, k, v, dout, gamma=None, chunk=32):
    """Gradients (dq, dk, dv) of the unnormalised AHLA output for upstream dout.  float32 or
    bfloat16 CUDA tensors [B,H,n,d] (d == dv)."""
    L = lib()
    if q.dtype not in _DTYPES or any(t.dtype != q.dtype for t in (k, v, dout)):
        raise TypeError("q, k, v, dout must share a dtype (float32 or bfloat16)")
    B, H, n, d = q.shape
    dv = v.shape[-1]
    device = q.device
    qd, kd, vd, od = (t.contiguous() for t in (q, k, v, dout))
    g = _gamma_tensor(gamma, H, device)
    gq, gk, gv = torch.empty_like(qd), torch.empty_like(kd), torch.empty_like(vd)
    sh = _stream_handle(device)
    nbytes = L.hla2_ahla_backward_workspace_bytes(B, H, n, d, dv, chunk, _DTYPES[q.dtype], 0)
    if nbytes == ctypes.c_size_t(-1).value:
        nbytes = 0
    ws = _workspace(int(nbytes), device, sh)
    opts = Opts(_DTYPES[q.dtype], 1e-6, None if ws is None else ws.data_ptr(), int(nbytes), None, None, None, 0, 0)
    _check("hla2_ahla_backward", _alone(L.hla2_ahla_backward, _ptr(qd), _ptr(kd), _ptr(vd), _ptr(od), _ptr(gq), _ptr(gk),
                                        _ptr(gv), B, H, n, d, dv, _ptr(g), 0, chunk, sh, ctypes.byref(opts)))
    return gq, gk, gv


# ---------------------------------------------------------------------------------------
# Around a mixer layer: first-order linear attention, block norms, 4-bit projections
# ---------------------------------------------------------------------------------------

# These calls are short on the GPU (a step of one sequence takes a few microseconds), so the compiled
# module takes their ordinary forms (_quick), and the rest is kept lean: addresses go to the library as plain
# integers and the argument blocks as packed bytes in the C layout.

_raw_stream = torch._C._cuda_getCurrentRawStream  # current_stream(device).cuda_stream without the object

_LINATTN_ARGS = struct.Struct("@7if2P" + 3 * "P3q" + "PPN")   # hla2_linattn_args
_BLOCK_ARGS = struct.Struct("@3iqifPqPqPqPPP")                # hla2_block_args


def _need_cuda(first, *others):
    """Device index of CUDA tensors that share one device and one supported type."""
    dtype = first.dtype
    if not first.is_cuda or dtype not in _DTYPES:
        raise TypeError("tensors must be float32 or bfloat16 CUDA tensors")
    index = first.get_device()
    for t in others:
        if t is not None and (t.dtype != dtype or t.get_device() != index):
            raise TypeError("tensors must all have the same type and device")
    return index


_capturing = torch._C._cuda_isCurrentStreamCapturing
_ERR_WORKSPACE = -3
_STATUS_BYTES = 256  # at a workspace's start, for the calls with bounded waits


def _with_scratch(call, query, index, stream):
    """Return code of ``call(address, bytes)`` with scratch memory of at least ``query()`` bytes.  The stream's
    cached buffer is tried first: the library checks its size before it launches anything.  Under
    graph capture the buffer is the graph's own: the cached one is shared with eager calls on the
    stream, which a replay would race with.  The first bytes are the status word (see
    hla2_workspace_status): 0 in a first buffer, taken along to a larger one, so that a wait that gave up stays
    recorded.  Every rejection without memory is the call's."""
    key = (index, stream or None)  # as check_status has it
    capturing = _capturing()
    known = None if capturing else _scratch_cache.get(key)
    if known is not None:
        rc = _alone(call, known.data_ptr(), known.numel())
        if rc != _ERR_WORKSPACE:
            return rc
    nbytes = query()
    if nbytes == _SIZE_MAX or nbytes == 0:
        return call(0, 0)
    with _scratch_lock:
        known = None if capturing else _scratch_cache.get(key)  # another thread's call may have grown it
        if known is None or known.numel() < nbytes:
            buf = torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", index))
            if known is None:
                buf[:_STATUS_BYTES].zero_()
            else:
                buf[:_STATUS_BYTES].copy_(known[:_STATUS_BYTES])
            if not capturing:
                _scratch_cache[key] = buf
        else:
            buf = known
        return call(buf.data_ptr(), buf.numel())


def _cached_scratch(t):
    """The buffer that _with_scratch would try first for a call on t's device, or None."""
    index = t.get_device()
    return None if index < 0 or _capturing() else _scratch_cache.get((index, _raw_stream(index) or None))


def _quick(name, *args):
    """The call by the compiled host side; None where it is not an ordinary one (host_calls.cpp)."""
    if _host is None:
        if _lib is None and os.path.exists(LIB_PATH):
            lib()
        if _host is None:
            return None
    return getattr(_host, name)(*args)


def _quick_scratch(name, t, *args):
    """_quick for a call on the cached scratch of t's device and stream."""
    with _scratch_lock:
        return _quick(name, *args, _cached_scratch(t))


def _contiguous_like(t):
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _float_vector(gamma, H, device):
    """_gamma_tensor; a tensor that already is what the kernels read goes through as it is."""
    if gamma is None:
        return None
    if (isinstance(gamma, torch.Tensor) and gamma.dtype == torch.float32 and gamma.is_cuda and gamma.dim() == 1
            and gamma.shape[0] == H and gamma.stride(0) == 1 and gamma.device == device):
        return gamma
    return _gamma_tensor(gamma, H, device)


def _view4(t):
    """(tensor, address, strides of batch, head, token) of [B, H, n, D]: the tensor itself where its
    strides serve, else a copy."""
    (B, H, n, D), (sb, sh, sn, sd) = t.shape, t.stride()
    p = t.data_ptr()
    per16 = 16 // t.element_size()
    if (p % 16 or sd != 1 and D > 1 or B > 1 and (sb % per16 or sb < D) or H > 1 and (sh % per16 or sh < D)
            or n > 1 and (sn % per16 or sn < D)):
        t = t.clone(memory_format=torch.contiguous_format)
        p, (sb, sh, sn, _) = t.data_ptr(), t.stride()
    return t, p, sb, sh, sn


def _out4(name, out, like, shape):
    """Output [B, H, n, D]: the caller's, or a new one with the token / head order of ``like``."""
    if out is None:
        B, H, n, D = shape
        if like.stride(2) > like.stride(1):  # token-major
            return torch.empty((B, n, H, D), dtype=like.dtype, device=like.device).transpose(1, 2)
        return torch.empty(shape, dtype=like.dtype, device=like.device)
    if tuple(out.shape) != tuple(shape) or out.dtype != like.dtype or out.device != like.device:
        raise ValueError(f"{name} must be {tuple(shape)} of the inputs' type and device")
    if out.numel() and out.stride(3) != 1 and out.shape[3] > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return out


def _plain_view(t):
    return View(t.data_ptr(), *t.stride()[:3])


class _Lin(NamedTuple):
    """One checked call: sizes, the fields of its argument block but for the workspace, and the
    tensors that they point into."""
    B: int
    H: int
    Hk: int
    n: int
    d: int
    dv: int
    device: torch.device
    index: int
    head: tuple
    keep: tuple

    def run(self, fn, backward, want_final, *rest):
        stream = _raw_stream(self.index)
        rc = _with_scratch(lambda p, nbytes: fn(_LINATTN_ARGS.pack(*self.head, p, nbytes), *rest, stream),
                           lambda: lib().hla2_linattn_workspace_bytes(_LINATTN_ARGS.pack(*self.head, 0, 0), backward,
                                                                      want_final), self.index, stream)
        if rc:
            _check(fn.__name__, rc)


def _linattn_args(q, k, v, gamma, scale, lengths, init_state):
    index = _need_cuda(q, k, v)
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [B, heads, n, dim]")
    device = q.device
    B, H, n, d = q.shape
    Hk, dv = k.shape[1], v.shape[3]
    if k.shape != (B, Hk, n, d) or v.shape != (B, Hk, n, dv):
        raise ValueError("shape mismatch between q, k, v")
    if (Hk == 0) != (H == 0) or (Hk and H % Hk):
        raise ValueError("the query heads must be a multiple of the key heads")
    g = _float_vector(gamma, Hk, device)
    if lengths is not None and not (isinstance(lengths, torch.Tensor) and lengths.dtype == torch.int32
                                    and lengths.device == device and lengths.is_contiguous()):
        lengths = torch.as_tensor(lengths, device=device)
        if lengths.dtype not in (torch.int32, torch.int64):
            raise ValueError("lengths must be integers")
        lengths = (lengths.clamp(0, n) if lengths.dtype == torch.int64 else lengths).to(torch.int32).contiguous()
    if lengths is not None and lengths.shape != (B,):
        raise ValueError("lengths must be B integers")
    init = _state_arg("init_state", init_state, (B, Hk, d, dv), device)
    qt, *qv = _view4(q)
    kt, *kv = _view4(k)
    vt, *vv = _view4(v)
    head = (_DTYPES[q.dtype], B, H, Hk, n, d, dv, scale, 0 if g is None else g.data_ptr(),
            0 if lengths is None else lengths.data_ptr(), *qv, *kv, *vv, 0 if init is None else init.data_ptr())
    return _Lin(B, H, Hk, n, d, dv, device, index, head, (qt, kt, vt, g, lengths, init))


def _state_arg(name, state, shape, device):
    if state is None:
        return None
    if tuple(state.shape) != shape or state.dtype != torch.float32 or state.device != device:
        raise ValueError(f"{name} must be a float32 {shape} tensor on the inputs' device")
    return _packed16(state)


def linattn_forward(q, k, v, gamma=None, scale=1.0, lengths=None, init_state=None, return_final_state=False, out=None):
    """First-order linear attention with a decay for each key head, chunk-parallel:
    P_t = gamma P_{t-1} + k_t v_t^T, out_t = scale * P_t^T q_t.

    q [B,H,n,d]; k [B,Hk,n,d]; v [B,Hk,n,dv]; H a multiple of Hk (query head h reads key head
    h // (H // Hk)); float32 or bfloat16 on the GPU, any strides (a layout with 16-byte
    rows is read in place, e.g. a transposed [B,n,H,d]; another is copied).  gamma: None, a scalar, or
    [Hk] in (0, 1].  lengths: None or B token counts; the rows past a sequence's length are padding,
    whatever they hold: 0 in the output, and not in the state.  init_state: float32 [B,Hk,d,dv]
    to continue from.  Returns out [B,H,n,dv], in q's token / head order, and with
    ``return_final_state`` the float32 state after each sequence's last token, which
    linattn_decode_step goes on from."""
    if out is None:
        res = _quick_scratch("linattn_forward", q, q, k, v, gamma, scale, lengths, init_state, bool(return_final_state))
        if res is not None:
            return res
    return _linattn_forward(q, k, v, gamma, scale, lengths, init_state, return_final_state, out)


@_on_its_device
def _linattn_forward(q, k, v, gamma, scale, lengths, init_state, return_final_state, out):
    a = _linattn_args(q, k, v, gamma, scale, lengths, init_state)
    o = _out4("out", out, q, (a.B, a.H, a.n, a.dv))
    fin = torch.empty((a.B, a.Hk, a.d, a.dv), dtype=torch.float32, device=a.device) if return_final_state else None
    a.run(lib().hla2_linattn_forward, 0, 0 if fin is None else 1, _plain_view(o), None if fin is None else fin.data_ptr())
    return (o, fin) if return_final_state else o


def linattn_backward(q, k, v, dout, gamma=None, scale=1.0, lengths=None, init_state=None, dfinal_state=None,
                     dq=None, dk=None, dv=None):
    """Gradients of linattn_forward for the upstream gradient dout [B,H,n,dv] of its output and
    dfinal_state (None: zero) of its final state.  Returns (dq, dk, dv), dk and dv summed over
    the query heads that share a key head, and with an init_state also its float32 gradient.
    gamma has no gradient."""
    if dq is None and dk is None and dv is None:
        res = _quick_scratch("linattn_backward", q, q, k, v, gamma, scale, lengths, init_state, dout, dfinal_state)
        if res is not None:
            return res
    return _linattn_backward(q, k, v, dout, gamma, scale, lengths, init_state, dfinal_state, dq, dk, dv)


@_on_its_device
def _linattn_backward(q, k, v, dout, gamma, scale, lengths, init_state, dfinal_state, dq, dk, dv):
    a = _linattn_args(q, k, v, gamma, scale, lengths, init_state)
    _need_cuda(q, dout)
    if dout.shape != (a.B, a.H, a.n, a.dv):
        raise ValueError("dout must be [B, H, n, dv]")
    states = (a.B, a.Hk, a.d, a.dv)
    dfin = _state_arg("dfinal_state", dfinal_state, states, a.device)
    dot, *dov = _view4(dout)
    gq = _out4("dq", dq, q, (a.B, a.H, a.n, a.d))
    gk = _out4("dk", dk, k, (a.B, a.Hk, a.n, a.d))
    gv = _out4("dv", dv, v, (a.B, a.Hk, a.n, a.dv))
    dinit = torch.empty(states, dtype=torch.float32, device=a.device) if init_state is not None else None
    a.run(lib().hla2_linattn_backward, 1, 0 if dinit is None and dfin is None else 1, View(*dov), _plain_view(gq),
          _plain_view(gk), _plain_view(gv), None if dfin is None else dfin.data_ptr(),
          None if dinit is None else dinit.data_ptr())
    return (gq, gk, gv) if dinit is None else (gq, gk, gv, dinit)


def linattn_decode_step(state, q, k, v, gamma=None, scale=1.0, out=None):
    """One token for each of N sequences: ``state`` [N,Hk,d,dv] float32 on the GPU is updated in
    place.  q [N,H,d]; k [N,Hk,d]; v [N,Hk,dv].  Returns out [N,H,dv] = scale * P^T q."""
    if out is None:
        res = _quick("linattn_decode_step", state, q, k, v, gamma, scale)
        if res is not None:
            return res
    return _linattn_decode_step(state, q, k, v, gamma, scale, out)


@_on_its_device
def _linattn_decode_step(state, q, k, v, gamma, scale, out):
    if not state.is_cuda or state.dtype != torch.float32 or not state.is_contiguous():
        raise ValueError("state must be a contiguous float32 CUDA tensor")
    index = _need_cuda(q, k, v)
    N, H, d = q.shape
    Hk, dv = k.shape[1], v.shape[2]
    if (k.shape != (N, Hk, d) or v.shape != (N, Hk, dv) or state.shape != (N, Hk, d, dv)
            or state.get_device() != index):
        raise ValueError("shape or device mismatch between state, q, k, v")
    q, k, v = _packed16(q), _packed16(k), _packed16(v)
    g = _float_vector(gamma, Hk, q.device)
    if out is None:
        out = torch.empty((N, H, dv), dtype=q.dtype, device=q.device)
    elif out.shape != (N, H, dv) or out.dtype != q.dtype or not out.is_contiguous() or out.get_device() != index:
        raise ValueError("out must be a contiguous [N, H, dv] tensor of the inputs' type")
    rc = lib().hla2_linattn_decode_step(state.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), N, H,
                                        Hk, d, dv, None if g is None else g.data_ptr(), scale, _DTYPES[q.dtype],
                                        _raw_stream(index))
    if rc:
        _check("hla2_linattn_decode_step", rc)
    return out


def _packed16(t):
    """The tensor, or a copy where it is not contiguous at a 16-byte address."""
    if not t.is_contiguous():
        return t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


GATE_ACTS = {"sigmoid": 0, "silu": 1}


class BlockJoinGrads(NamedTuple):
    """Gradients of block_join's inputs (None where the input was None); those of the weights and
    the scale are float32."""
    dx: torch.Tensor
    dy: torch.Tensor
    dgate: Optional[torch.Tensor]
    dpost_weight: torch.Tensor
    dscale: Optional[torch.Tensor]
    dnext_weight: Optional[torch.Tensor]


def _rows(t, D):
    """(rows tensor, rows, row stride) of [..., D]: in place where all leading dimensions are one stride."""
    if t.dim() != 2:
        if t.dim() == 0:
            raise ValueError(f"the last dimension must be {D}")
        t = t.reshape(-1, D) if D else t.reshape(0, 0)  # a view where the strides allow it
    rows, cols = t.shape
    if cols != D:
        raise ValueError(f"the last dimension must be {D}")
    if D > 1 and t.stride(1) != 1:
        t = t.contiguous()
    return t, rows, t.stride(0) if rows > 1 else D


def _vector(name, w, D):
    if w is None:
        return None
    if w.shape != (D,):
        raise ValueError(f"{name} must be [{D}]")
    return w if w.is_contiguous() else w.contiguous()


def _addr(t):
    return 0 if t is None else t.data_ptr()


def _block_args(x, y, post_weight, gate, gate_act, scale, next_weight, eps):
    """(packed argument block, D, device index, tensors to keep)"""
    index = _need_cuda(x, y, post_weight, gate, scale, next_weight)
    act = GATE_ACTS.get(gate_act)
    if act is None:
        raise ValueError(f"gate_act must be one of {sorted(GATE_ACTS)}")
    shape = x.shape
    D = shape[-1] if x.dim() else 0
    pw, sc, nw = _vector("post_weight", post_weight, D), _vector("scale", scale, D), _vector("next_weight", next_weight, D)
    xr, rows, xs = _rows(x, D)
    yr = zr = None
    ys = zs = cols = 0
    if y is not None:
        if y.shape != shape:
            raise ValueError("y must have x's shape")
        yr, _, ys = _rows(y, D)
    if gate is not None:
        cols = gate.shape[-1] if gate.dim() else 0
        if gate.shape[:-1] != shape[:-1] or cols not in (1, D):
            raise ValueError("gate must have x's shape, or one value a row")
        zr, _, zs = _rows(gate, cols)
    args = _BLOCK_ARGS.pack(_DTYPES[x.dtype], act, cols, rows, D, eps, xr.data_ptr(), xs, _addr(yr), ys, _addr(zr), zs,
                            _addr(pw), _addr(sc), _addr(nw))
    return args, D, index, (xr, yr, zr, pw, sc, nw)


def block_norm(x, weight, eps=1e-6, out=None):
    """The norm before a block: x / sqrt(mean(x^2) + eps) * weight over the last dimension (1 to
    8192 values; float32 or bfloat16 on the GPU).  out may be x itself."""
    if out is None and weight is not None:
        res = _quick("block_join", x, None, None, None, 0, None, weight, eps)
        if res is not None:
            return res[1]
    return _block_norm(x, weight, eps, out)


@_on_its_device
def _block_norm(x, weight, eps, out):
    args, _, index, keep = _block_args(x, None, None, None, "sigmoid", None, weight, eps)
    if out is None:
        out = _contiguous_like(x)
    elif out.shape != x.shape or out.dtype != x.dtype or out.device != x.device or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor of x's shape, type and device")
    rc = lib().hla2_block_join(args, None, out.data_ptr(), _raw_stream(index))
    if rc:
        _check("hla2_block_join", rc)
    return out


def block_norm_backward(x, weight, dout, eps=1e-6):
    """(dx, dweight) of block_norm; dweight is a float32 sum over the rows."""
    res = _quick_scratch("block_join_backward", x, x, None, None, None, 0, None, weight, eps, None, dout)
    if res is not None:
        return res[0], res[5]
    g = _block_backward(x, None, None, None, "sigmoid", None, weight, None, dout, eps)
    return g.dx, g.dnext_weight


def block_join(x, y, post_weight, gate=None, gate_act="sigmoid", scale=None, next_weight=None, eps=1e-6):
    """The end of a block and the start of the next: r = x + scale * act(gate) * norm(y) * post_weight
    and h = norm(r) * next_weight (None without next_weight), norm(t) = t / sqrt(mean(t^2) + eps) over
    the last dimension.  x the residual stream, y the block's output [..., D]; gate None, [..., D]
    or one value a row [..., 1], act "sigmoid" or "silu"; post_weight, scale (None: 1) and
    next_weight [D]; all of one type, float32 or bfloat16 on the GPU.  Returns (r, h)."""
    if y is None:
        raise ValueError("block_join needs y (block_norm is the norm alone)")
    act = GATE_ACTS.get(gate_act)
    if act is not None:
        res = _quick("block_join", x, y, post_weight, gate, act, scale, next_weight, eps)
        if res is not None:
            return res
    return _block_join(x, y, post_weight, gate, gate_act, scale, next_weight, eps)


@_on_its_device
def _block_join(x, y, post_weight, gate, gate_act, scale, next_weight, eps):
    args, _, index, keep = _block_args(x, y, post_weight, gate, gate_act, scale, next_weight, eps)
    r = _contiguous_like(x)
    h = _contiguous_like(x) if next_weight is not None else None
    rc = lib().hla2_block_join(args, r.data_ptr(), None if h is None else h.data_ptr(), _raw_stream(index))
    if rc:
        _check("hla2_block_join", rc)
    return r, h


@_on_its_device
def _block_backward(x, y, post_weight, gate, gate_act, scale, next_weight, dr, dh, eps):
    args, D, index, keep = _block_args(x, y, post_weight, gate, gate_act, scale, next_weight, eps)
    device = x.device
    for name, t in (("dr", dr), ("dh", dh)):
        if t is not None and (t.shape != x.shape or t.dtype != x.dtype or t.get_device() != index):
            raise ValueError(f"{name} must have x's shape, type and device")
    if (next_weight is None) != (dh is None):
        raise ValueError("dh is needed with next_weight, and only then")
    if dr is None and dh is None:
        raise ValueError("dr or dh is needed")
    dr, dh = (None if t is None else t.contiguous() for t in (dr, dh))
    dx, dy, dgate = (None if t is None else _contiguous_like(t) for t in (x, y, gate))
    if y is None:
        dpw = dsc = None
        dnw = torch.empty(D, dtype=torch.float32, device=device)
    else:
        sums = torch.empty((3, D), dtype=torch.float32, device=device)
        dpw, dsc, dnw = (None if w is None else g for g, w in zip(sums, (post_weight, scale, next_weight)))
    stream = _raw_stream(index)
    L = lib()
    outs = (_addr(dr), _addr(dh), _addr(dx), _addr(dy), _addr(dgate), _addr(dpw), _addr(dsc), _addr(dnw))
    skip = _STATUS_BYTES

    def query():
        nbytes = L.hla2_block_join_backward_workspace_bytes(args)
        return nbytes if nbytes in (0, _SIZE_MAX) else nbytes + skip

    rc = _with_scratch(lambda p, nbytes: L.hla2_block_join_backward(args, *outs, p and p + skip, max(nbytes - skip, 0), stream),
                       query, index, stream)
    if rc:
        _check("hla2_block_join_backward", rc)
    return BlockJoinGrads(dx, dy, dgate, dpw, dsc, dnw)


def block_join_backward(x, y, post_weight, gate=None, gate_act="sigmoid", scale=None, next_weight=None, dr=None,
                        dh=None, eps=1e-6):
    """BlockJoinGrads of block_join for the upstream gradients dr of r (None: zero) and dh of h
    (needed with next_weight).  Nothing is kept from the forward."""
    if y is None:
        raise ValueError("block_join_backward needs y (block_norm_backward is the norm alone)")
    act = GATE_ACTS.get(gate_act)
    if act is not None:
        res = _quick_scratch("block_join_backward", x, x, y, post_weight, gate, act, scale, next_weight, eps, dr, dh)
        if res is not None:
            return BlockJoinGrads(*res)
    return _block_backward(x, y, post_weight, gate, gate_act, scale, next_weight, dr, dh, eps)


def w4_matvec(x, qweight, scales, zeros=None, bias=None, out=None):
    """Products of a few rows with 4-bit weights: y = x W^T (+ bias) with
    W[n, k] = (q[n, k] - z[n, k // group]) * scales[n, k // group].

    x [..., K] with 1 to 16 rows; qweight uint8 [N, K / 2], value 2 j of a row in the low half of
    byte j and 2 j + 1 in the high half; scales [N, K / group], group 32, 64 or 128; zeros uint8
    [N, K / group] in 0..15 (None: 8); bias [N].  x, scales and bias float32 or bfloat16
    of one type on the GPU.  Returns y [..., N].  The products are exact and the sums float32."""
    if out is None:
        res = _quick("w4_matvec", x, qweight, scales, zeros, bias)
        if res is not None:
            return res
    return _w4_matvec(x, qweight, scales, zeros, bias, out)


@_on_its_device
def _w4_matvec(x, qweight, scales, zeros, bias, out):
    index = _need_cuda(x, scales, bias)
    shape = x.shape
    K = shape[-1] if x.dim() else 0
    if qweight.dim() != 2 or qweight.dtype != torch.uint8 or qweight.shape[1] * 2 != K or qweight.get_device() != index:
        raise ValueError("qweight must be uint8 [N, K / 2] on x's device")
    N = qweight.shape[0]
    if scales.dim() != 2 or scales.shape[0] != N or scales.shape[1] == 0 or K % scales.shape[1]:
        raise ValueError("scales must be [N, K / group]")
    group = K // scales.shape[1]
    if zeros is not None and (zeros.dtype != torch.uint8 or zeros.shape != scales.shape or zeros.get_device() != index):
        raise ValueError("zeros must be uint8 of scales' shape")
    if bias is not None and bias.shape != (N,):
        raise ValueError("bias must be [N]")
    x2, M, stride = _rows(x, K)
    if x2.data_ptr() % 16 or M > 1 and stride * x2.element_size() % 16:
        x2, stride = x2.clone(memory_format=torch.contiguous_format), K
    qweight, scales = _packed16(qweight), scales.contiguous()
    zeros, bias = (None if t is None else t.contiguous() for t in (zeros, bias))
    if out is None:
        out = torch.empty((*shape[:-1], N), dtype=x.dtype, device=x.device)
    elif out.shape != (*shape[:-1], N) or out.dtype != x.dtype or out.get_device() != index or not out.is_contiguous():
        raise ValueError("out must be a contiguous [..., N] tensor of x's type and device")
    rc = lib().hla2_w4_matvec(x2.data_ptr(), stride, qweight.data_ptr(), scales.data_ptr(), _addr(zeros), _addr(bias),
                              out.data_ptr(), M, N, K, group, _DTYPES[x.dtype], _raw_stream(index))
    if rc:
        _check("hla2_w4_matvec", rc)
    return out
