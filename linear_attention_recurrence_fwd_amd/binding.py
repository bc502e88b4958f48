"""ctypes binding of libgdn.so (the C ABI in include/gdn.h).

Argument marshalling only: this module checks dtypes/shapes, allocates the
outputs and the workspace with torch (device memory), and passes raw pointers
plus the current HIP stream to the library.  The entries of the rotation with
several axes and of the paged cache first take the same steps in native code
(_calls), which leaves everything out of the ordinary to the functions here.  Every step of the computation runs
in the library's kernels.  There is no fallback: if libgdn.so is missing or a
call fails, an exception is raised.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import warnings

import torch

try:
    from . import _calls  # the short way to the entries for single tokens (csrc/gdn_calls.cpp)
except ImportError as _error:  # the long way, in this module, is whole without it
    _calls = None
    warnings.warn("_calls.so was not loaded (%s): calls of the rotation with several axes and of the paged cache take "
                  "about 10 us longer on the host; __graft_entry__.build() builds it" % _error, RuntimeWarning)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")
CHUNK = 64

GDN_F32, GDN_BF16 = 0, 1
ALGO_AUTO, ALGO_SCAN, ALGO_CHUNK, ALGO_CHUNK_TPAR = 0, 1, 2, 3
STATUS = {0: "GDN_OK", 1: "GDN_ERR_INVALID_ARG", 2: "GDN_ERR_UNSUPPORTED",
          3: "GDN_ERR_WORKSPACE", 4: "GDN_ERR_HIP"}

# every entry point declared in include/gdn.h
EXPORTS = ("gdn_ckpt_elems", "gdn_ckpt_bytes", "gdn_workspace_bytes", "gdn_fwd_workspace_bytes", "gdn_bwd_workspace_bytes",
           "gdn_fwd", "gdn_fwd_noalloc", "gdn_bwd", "gdn_decode_conv", "gdn_vg_ckpt_elems", "gdn_vg_ckpt_bytes",
           "gdn_fwd_vg_workspace_bytes",
           "gdn_bwd_vg_workspace_bytes", "gdn_fwd_vg", "gdn_bwd_vg",
           "gdn_decay_fwd_workspace_bytes", "gdn_decay_bwd_workspace_bytes", "gdn_decay_fwd", "gdn_decay_bwd",
           "gdn_norm_rope_fwd", "gdn_norm_rope_bwd_workspace_bytes", "gdn_norm_rope_bwd",
           "gdn_norm_rope_axes_fwd", "gdn_norm_rope_axes_bwd",
           "gdn_paged_append", "gdn_prefix_attention_workspace_bytes", "gdn_prefix_attention",
           "gdn_set_kernel_events",
           "gdn_status_string", "gdn_version")


class Dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("Hk", ctypes.c_int64),
                ("Hv", ctypes.c_int64), ("Dk", ctypes.c_int64), ("Dv", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("algo", ctypes.c_int32), ("save", ctypes.c_int32)]


class NormDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("Hq", ctypes.c_int64),
                ("Hk", ctypes.c_int64), ("D", ctypes.c_int64), ("R", ctypes.c_int64),
                ("P", ctypes.c_int64), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("eps", ctypes.c_float), ("w_offset", ctypes.c_float)]


class PagedDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("N", "S", "Hq", "Hk", "D", "pages", "page", "width", "page_stride",
                                              "head_stride", "token_stride")] + [("dtype", ctypes.c_int32)]


class Turn(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("P", "R", "q_stride", "k_stride", "v_stride", "first")] + \
               [("A", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("eps", ctypes.c_float),
                ("w_offset", ctypes.c_float)]


class GdnError(RuntimeError):
    def __init__(self, fn, code, hint=""):
        self.code = code
        super().__init__("%s failed: %s (%s)%s" % (fn, STATUS.get(code, code),
                                                   lib().gdn_status_string(code).decode(), hint))


_lib = None


def lib():
    """Load libgdn.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libgdn.so not built (run __graft_entry__.build()): %s" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        P, S = ctypes.c_void_p, ctypes.c_size_t
        PD = ctypes.POINTER(Dims)
        for n in ("gdn_ckpt_elems", "gdn_fwd_workspace_bytes", "gdn_bwd_workspace_bytes", "gdn_vg_ckpt_elems",
                  "gdn_vg_ckpt_bytes", "gdn_fwd_vg_workspace_bytes", "gdn_bwd_vg_workspace_bytes",
                  "gdn_decay_fwd_workspace_bytes", "gdn_decay_bwd_workspace_bytes"):
            getattr(L, n).argtypes = [PD, ctypes.POINTER(S)]
            getattr(L, n).restype = ctypes.c_int
        L.gdn_ckpt_bytes.argtypes = [PD, ctypes.POINTER(S)]
        L.gdn_ckpt_bytes.restype = ctypes.c_int
        L.gdn_workspace_bytes.argtypes = [PD, ctypes.c_int, ctypes.POINTER(S)]
        L.gdn_workspace_bytes.restype = ctypes.c_int
        L.gdn_fwd.argtypes = [PD] + [P] * 13 + [S, P]
        L.gdn_fwd.restype = ctypes.c_int
        L.gdn_fwd_noalloc.argtypes = [PD] + [P] * 13
        L.gdn_fwd_noalloc.restype = ctypes.c_int
        L.gdn_bwd.argtypes = [PD] + [P] * 21 + [S, P]
        L.gdn_bwd.restype = ctypes.c_int
        L.gdn_decode_conv.argtypes = [PD] + [P] * 4 + [ctypes.c_int32] + [P] * 9
        L.gdn_decode_conv.restype = ctypes.c_int
        L.gdn_fwd_vg.argtypes = [PD] + [P] * 11 + [S, P]
        L.gdn_fwd_vg.restype = ctypes.c_int
        L.gdn_bwd_vg.argtypes = [PD] + [P] * 17 + [S, P]
        L.gdn_bwd_vg.restype = ctypes.c_int
        L.gdn_decay_fwd.argtypes = [PD] + [P] * 4 + [ctypes.c_float] + [P] * 5 + [S, P]
        L.gdn_decay_fwd.restype = ctypes.c_int
        L.gdn_decay_bwd.argtypes = [PD] + [P] * 4 + [ctypes.c_float] + [P] * 10 + [S, P]
        L.gdn_decay_bwd.restype = ctypes.c_int
        PN = ctypes.POINTER(NormDims)
        L.gdn_norm_rope_fwd.argtypes = [PN] + [P] * 9
        L.gdn_norm_rope_fwd.restype = ctypes.c_int
        L.gdn_norm_rope_bwd_workspace_bytes.argtypes = [PN, ctypes.POINTER(S)]
        L.gdn_norm_rope_bwd_workspace_bytes.restype = ctypes.c_int
        L.gdn_norm_rope_bwd.argtypes = [PN] + [P] * 13 + [S, P]
        L.gdn_norm_rope_bwd.restype = ctypes.c_int
        L.gdn_norm_rope_axes_fwd.argtypes = [PN, ctypes.c_int32] + [P] * 10
        L.gdn_norm_rope_axes_fwd.restype = ctypes.c_int
        L.gdn_norm_rope_axes_bwd.argtypes = [PN, ctypes.c_int32] + [P] * 14 + [S, P]
        L.gdn_norm_rope_axes_bwd.restype = ctypes.c_int
        PP, I64 = ctypes.POINTER(PagedDims), ctypes.c_int64
        L.gdn_paged_append.argtypes = [PP, ctypes.POINTER(Turn)] + [P] * 15
        L.gdn_paged_append.restype = ctypes.c_int
        L.gdn_prefix_attention_workspace_bytes.argtypes = [PP, I64, I64, I64, ctypes.POINTER(S)]
        L.gdn_prefix_attention_workspace_bytes.restype = ctypes.c_int
        L.gdn_prefix_attention.argtypes = [PP] + [P] * 6 + [I64, P, I64, I64, ctypes.c_float] + [P] * 3 + [S, P]
        L.gdn_prefix_attention.restype = ctypes.c_int
        L.gdn_set_kernel_events.argtypes = [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int]
        L.gdn_set_kernel_events.restype = ctypes.c_int
        L.gdn_status_string.argtypes = [ctypes.c_int]
        L.gdn_status_string.restype = ctypes.c_char_p
        L.gdn_version.argtypes = []
        L.gdn_version.restype = ctypes.c_char_p
        _lib = L
    return _lib


def make_dims(B, T, Hk, Hv, Dk, Dv, dtype, algo=ALGO_AUTO, save=False) -> Dims:
    dt = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}.get(dtype, dtype)
    return Dims(B, T, Hk, Hv, Dk, Dv, dt, algo, 1 if save else 0)


def _query(fn, d: Dims) -> int:
    out = ctypes.c_size_t(0)
    rc = getattr(lib(), fn)(ctypes.byref(d), ctypes.byref(out))
    if rc:
        raise GdnError(fn, rc)
    return out.value


def ckpt_elems(d: Dims) -> int:
    return _query("gdn_ckpt_elems", d)


def vg_ckpt_elems(d: Dims) -> int:
    return _query("gdn_vg_ckpt_elems", d)


def fwd_workspace_bytes(d: Dims) -> int:
    return _query("gdn_fwd_workspace_bytes", d)


def bwd_workspace_bytes(d: Dims) -> int:
    return _query("gdn_bwd_workspace_bytes", d)


def _p(x):
    return None if x is None else ctypes.c_void_p(x.data_ptr())


def _check(x, name, shape, dtype, device):
    if x.dtype == dtype and x.shape == shape and x.device == device and x.is_contiguous():
        return
    if x.dtype != dtype:
        raise TypeError("%s: expected %s, got %s" % (name, dtype, x.dtype))
    if tuple(x.shape) != tuple(shape):
        raise ValueError("%s: expected shape %s, got %s" % (name, tuple(shape), tuple(x.shape)))
    if x.device != device:
        raise ValueError("%s: expected device %s, got %s" % (name, device, x.device))
    if not x.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _dims_of(q, v, algo, save=False):
    B, T, Hk, Dk = q.shape
    Hv, Dv = v.shape[2], v.shape[3]
    return make_dims(B, T, Hk, Hv, Dk, Dv, q.dtype, algo, save)


def _alloc_ckpt(d, dev, vg=False):
    """The checkpoint buffer: [ceil(T/64)-1, B, Hv, Dk, Dv] fp32, or, when the
    dims save (chunk family), a flat buffer of gdn_ckpt_elems (vg:
    gdn_vg_ckpt_elems) fp32 elements with contents private to the library."""
    nslab = max((d.T + CHUNK - 1) // CHUNK - 1, 0)
    nck = vg_ckpt_elems(d) if vg else ckpt_elems(d)
    if nck == nslab * d.B * d.Hv * d.Dk * d.Dv:
        return torch.empty((nslab, d.B, d.Hv, d.Dk, d.Dv), dtype=torch.float32, device=dev)
    return torch.empty((nck,), dtype=torch.float32, device=dev)


def _check_inputs(d, q, k, v, a, b, A_log, dt_bias, state0, mask):
    dev, dt = q.device, q.dtype
    if dev.type != "cuda":
        raise ValueError("gdn runs on the GPU; got device %s" % dev)
    B, T, Hk, Hv, Dk, Dv = d.B, d.T, d.Hk, d.Hv, d.Dk, d.Dv
    _check(q, "q", (B, T, Hk, Dk), dt, dev)
    _check(k, "k", (B, T, Hk, Dk), dt, dev)
    _check(v, "v", (B, T, Hv, Dv), dt, dev)
    _check(a, "a", (B, T, Hv), dt, dev)
    _check(b, "b", (B, T, Hv), dt, dev)
    _check(A_log, "A_log", (Hv,), torch.float32, dev)
    _check(dt_bias, "dt_bias", (Hv,), torch.float32, dev)
    if state0 is not None:
        _check(state0, "state0", (B, Hv, Dk, Dv), torch.float32, dev)
    if mask is not None:
        _check(mask, "mask", (B, T), torch.uint8, dev)


def fwd(q, k, v, a, b, A_log, dt_bias, state0=None, mask=None, *, need_ckpt=True,
        state_out=None, algo=ALGO_AUTO, save=False):
    """Forward scan.  Returns (o, state_out, ckpt); ckpt is None when not
    requested.  Pass state_out=state0 for an in-place state update.  With
    save=True the chunk form writes what the backward needs (bf16 chunk-start
    states, chunk matrices) into the checkpoint buffer instead of fp32 states
    (pass the same save to bwd)."""
    d = _dims_of(q, v, algo, save)
    if save and not need_ckpt:
        raise ValueError("save=True needs the checkpoint buffer (need_ckpt=True)")
    _check_inputs(d, q, k, v, a, b, A_log, dt_bias, state0, mask)
    dev = q.device
    o = torch.empty((d.B, d.T, d.Hv, d.Dv), dtype=q.dtype, device=dev)
    if state_out is None:
        state_out = torch.empty((d.B, d.Hv, d.Dk, d.Dv), dtype=torch.float32, device=dev)
    else:
        _check(state_out, "state_out", (d.B, d.Hv, d.Dk, d.Dv), torch.float32, dev)
    nck = ckpt_elems(d)
    ckpt = _alloc_ckpt(d, dev) if need_ckpt else None
    wsb = fwd_workspace_bytes(d)
    ws = torch.empty((max(wsb, 1),), dtype=torch.uint8, device=dev)
    rc = lib().gdn_fwd(ctypes.byref(d), _p(q), _p(k), _p(v), _p(a), _p(b), _p(A_log), _p(dt_bias),
                       _p(state0), _p(mask), _p(o), _p(state_out),
                       _p(ckpt) if (ckpt is not None and nck) else None,
                       _p(ws), wsb, _stream(dev))
    if rc:
        raise GdnError("gdn_fwd", rc)
    return o, state_out, ckpt


NOALLOC_SCRATCH_BYTES = 64 << 20  # GDN_NOALLOC_SCRATCH_BYTES


def fwd_noalloc(q, k, v, a, b, A_log, dt_bias, state0=None, mask=None, *, o, state_out, ckpt=None,
                algo=ALGO_AUTO, save=False):
    """gdn_fwd_noalloc: the forward with the library's static workspace.  The
    caller passes every output (o, state_out and, when wanted, ckpt); nothing
    is allocated here or in the library."""
    d = _dims_of(q, v, algo, save)
    _check_inputs(d, q, k, v, a, b, A_log, dt_bias, state0, mask)
    dev = q.device
    _check(o, "o", (d.B, d.T, d.Hv, d.Dv), q.dtype, dev)
    _check(state_out, "state_out", (d.B, d.Hv, d.Dk, d.Dv), torch.float32, dev)
    nck = ckpt_elems(d)
    if ckpt is not None and ckpt.numel() != nck:
        raise ValueError("ckpt must have %d elements" % nck)
    rc = lib().gdn_fwd_noalloc(ctypes.byref(d), _p(q), _p(k), _p(v), _p(a), _p(b), _p(A_log),
                               _p(dt_bias), _p(state0), _p(mask), _p(o), _p(state_out),
                               _p(ckpt) if (ckpt is not None and nck) else None, _stream(dev))
    if rc:
        raise GdnError("gdn_fwd_noalloc", rc)
    return o, state_out, ckpt


def bwd(q, k, v, a, b, A_log, dt_bias, state0, mask, ckpt, dO, dS_final=None, *,
        algo=ALGO_AUTO, save=False):
    """VJP.  Returns dict(dq, dk, dv, da, db, dA_log, ddt_bias, dstate).
    `save` must match the fwd call that wrote ckpt."""
    d = _dims_of(q, v, algo, save)
    _check_inputs(d, q, k, v, a, b, A_log, dt_bias, state0, mask)
    dev = q.device
    _check(dO, "dO", (d.B, d.T, d.Hv, d.Dv), q.dtype, dev)
    if dS_final is not None:
        _check(dS_final, "dS_final", (d.B, d.Hv, d.Dk, d.Dv), torch.float32, dev)
    nck = ckpt_elems(d)
    if nck:
        if ckpt is None or ckpt.numel() != nck:
            raise ValueError("ckpt from gdn_fwd with %d elements is required" % nck)
        if ckpt.dtype != torch.float32 or not ckpt.is_contiguous() or ckpt.device != dev:
            raise ValueError("ckpt must be a contiguous fp32 tensor on %s" % dev)
    out = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
               da=torch.empty_like(a), db=torch.empty_like(b),
               dA_log=torch.empty((d.Hv,), dtype=torch.float32, device=dev),
               ddt_bias=torch.empty((d.Hv,), dtype=torch.float32, device=dev),
               dstate=torch.empty((d.B, d.Hv, d.Dk, d.Dv), dtype=torch.float32, device=dev))
    wsb = bwd_workspace_bytes(d)
    ws = torch.empty((max(wsb, 1),), dtype=torch.uint8, device=dev)
    rc = lib().gdn_bwd(ctypes.byref(d), _p(q), _p(k), _p(v), _p(a), _p(b), _p(A_log), _p(dt_bias),
                       _p(state0), _p(mask), _p(ckpt) if nck else None, _p(dO), _p(dS_final),
                       *[_p(out[n]) for n in ("dq", "dk", "dv", "da", "db", "dA_log", "ddt_bias",
                                              "dstate")],
                       _p(ws), wsb, _stream(dev))
    if rc:
        raise GdnError("gdn_bwd", rc)
    return out


class GatedDeltaRule(torch.autograd.Function):
    """Autograd wrapper: forward returns (o, state_out); backward calls gdn_bwd."""

    @staticmethod
    def forward(ctx, q, k, v, a, b, A_log, dt_bias, state0, mask=None):
        o, st, ck = fwd(q, k, v, a, b, A_log, dt_bias, state0, mask, save=True)
        ctx.save_for_backward(q, k, v, a, b, A_log, dt_bias, state0, mask, ck)
        return o, st

    @staticmethod
    def backward(ctx, dO, dS):
        q, k, v, a, b, A_log, dt_bias, state0, mask, ck = ctx.saved_tensors
        g = bwd(q, k, v, a, b, A_log, dt_bias, state0, mask, ck, dO.contiguous(),
                None if dS is None else dS.contiguous(), save=True)
        return (g["dq"], g["dk"], g["dv"], g["da"], g["db"], g["dA_log"], g["ddt_bias"],
                g["dstate"] if state0 is not None else None, None)


class Plan:
    """Repeated fwd + bwd on fixed device tensors with every output and
    workspace allocated once and the ctypes argument lists built once, so a
    call costs one C-ABI call (used by the benchmark's timed loop).

    `t` maps q, k, v, a, b, A_log, dt_bias, state0, mask, dO, dS_final to
    device tensors (state0, mask, dS_final may be None).  save: the forward
    saves the bf16 states and chunk matrices for the backward (as in
    training)."""

    def __init__(self, t, algo=ALGO_AUTO, stream=None, save=True):
        q, v = t["q"], t["v"]
        self.d = d = _dims_of(q, v, algo, save)
        _check_inputs(d, q, k=t["k"], v=v, a=t["a"], b=t["b"], A_log=t["A_log"],
                      dt_bias=t["dt_bias"], state0=t["state0"], mask=t["mask"])
        dev = q.device
        self.t = t
        self.o = torch.empty((d.B, d.T, d.Hv, d.Dv), dtype=q.dtype, device=dev)
        self.state_out = torch.empty((d.B, d.Hv, d.Dk, d.Dv), dtype=torch.float32, device=dev)
        self.ckpt = _alloc_ckpt(d, dev)
        nck = self.ckpt.numel()
        self.g = dict(dq=torch.empty_like(q), dk=torch.empty_like(t["k"]), dv=torch.empty_like(v),
                      da=torch.empty_like(t["a"]), db=torch.empty_like(t["b"]),
                      dA_log=torch.empty((d.Hv,), dtype=torch.float32, device=dev),
                      ddt_bias=torch.empty((d.Hv,), dtype=torch.float32, device=dev),
                      dstate=torch.empty((d.B, d.Hv, d.Dk, d.Dv), dtype=torch.float32, device=dev))
        fws, bws = fwd_workspace_bytes(d), bwd_workspace_bytes(d)
        self.ws_f = torch.empty((max(fws, 1),), dtype=torch.uint8, device=dev)
        self.ws_b = torch.empty((max(bws, 1),), dtype=torch.uint8, device=dev)
        st = stream if stream is not None else torch.cuda.current_stream(dev)
        self.stream = st
        sp = ctypes.c_void_p(st.cuda_stream)
        ck = _p(self.ckpt) if nck else None
        ins = [_p(t[n]) for n in ("q", "k", "v", "a", "b", "A_log", "dt_bias", "state0", "mask")]
        self._fargs = (ctypes.byref(d), *ins, _p(self.o), _p(self.state_out), ck,
                       _p(self.ws_f), fws, sp)
        self._bargs = (ctypes.byref(d), *ins, ck, _p(t["dO"]), _p(t["dS_final"]),
                       *[_p(self.g[n]) for n in ("dq", "dk", "dv", "da", "db", "dA_log",
                                                 "ddt_bias", "dstate")],
                       _p(self.ws_b), bws, sp)
        self.fwd_ws_bytes, self.bwd_ws_bytes = fws, bws

    def fwd(self):
        rc = lib().gdn_fwd(*self._fargs)
        if rc:
            raise GdnError("gdn_fwd", rc)

    def bwd(self):
        rc = lib().gdn_bwd(*self._bargs)
        if rc:
            raise GdnError("gdn_bwd", rc)


# ---- per-key-channel gate (gdn_fwd_vg / gdn_bwd_vg)

def _check_inputs_vg(d, q, k, v, lg, b, state0, mask):
    dev, dt = q.device, q.dtype
    if dev.type != "cuda":
        raise ValueError("gdn runs on the GPU; got device %s" % dev)
    B, T, Hk, Hv, Dk, Dv = d.B, d.T, d.Hk, d.Hv, d.Dk, d.Dv
    _check(q, "q", (B, T, Hk, Dk), dt, dev)
    _check(k, "k", (B, T, Hk, Dk), dt, dev)
    _check(v, "v", (B, T, Hv, Dv), dt, dev)
    _check(lg, "lg", (B, T, Hv, Dk), torch.float32, dev)
    _check(b, "b", (B, T, Hv), dt, dev)
    if state0 is not None:
        _check(state0, "state0", (B, Hv, Dk, Dv), torch.float32, dev)
    if mask is not None:
        _check(mask, "mask", (B, T), torch.uint8, dev)


def vg_uses_chunk(d) -> bool:
    """Whether gdn_fwd_vg / gdn_bwd_vg run the chunk form for these dims (the
    library's rule: bf16, Dk 64 / 128 / 192, Dv a multiple of 32 up to 128,
    under AUTO more than one step, and the chunk buffers within 4 GiB)."""
    if d.T == 0 or d.algo == ALGO_SCAN:
        return False
    ok = (d.dtype == GDN_BF16 and d.Dk in (64, 128, 192) and d.Dv % 32 == 0 and d.Dv <= 128)
    bhc = d.B * d.Hv * ((d.T + 63) // 64)
    ok = ok and max(bhc * 64 * d.Dk * 2, bhc * 64 * 64 * 2, bhc * 8 * 64 * 4) < 1 << 32
    return d.algo == ALGO_CHUNK or (d.T > 1 and ok)


def fwd_vg(q, k, v, lg, b, state0=None, mask=None, *, need_ckpt=True, state_out=None,
           algo=ALGO_AUTO, save=False):
    """Forward with a per-key-channel gate: lg [B,T,Hv,Dk] fp32 holds log g,
    and g scales the state's rows.  Returns (o, state_out, ckpt).  With
    save=True the chunk form writes the backward's rows, matrices and X into
    ckpt (pass the same save to bwd_vg)."""
    d = _dims_of(q, v, algo, save)
    if save and not need_ckpt:
        raise ValueError("save=True needs the checkpoint buffer (need_ckpt=True)")
    _check_inputs_vg(d, q, k, v, lg, b, state0, mask)
    dev = q.device
    o = torch.empty((d.B, d.T, d.Hv, d.Dv), dtype=q.dtype, device=dev)
    if state_out is None:
        state_out = torch.empty((d.B, d.Hv, d.Dk, d.Dv), dtype=torch.float32, device=dev)
    else:
        _check(state_out, "state_out", (d.B, d.Hv, d.Dk, d.Dv), torch.float32, dev)
    nck = vg_ckpt_elems(d)
    ckpt = _alloc_ckpt(d, dev, vg=True) if need_ckpt else None
    wsb = _query("gdn_fwd_vg_workspace_bytes", d)
    ws = torch.empty((max(wsb, 1),), dtype=torch.uint8, device=dev)
    rc = lib().gdn_fwd_vg(ctypes.byref(d), _p(q), _p(k), _p(v), _p(lg), _p(b), _p(state0),
                          _p(mask), _p(o), _p(state_out),
                          _p(ckpt) if (ckpt is not None and nck) else None,
                          _p(ws), wsb, _stream(dev))
    if rc:
        raise GdnError("gdn_fwd_vg", rc)
    return o, state_out, ckpt


def bwd_vg(q, k, v, lg, b, state0, mask, ckpt, dO, dS_final=None, *, algo=ALGO_AUTO, save=False):
    """VJP of fwd_vg.  Returns dict(dq, dk, dv, dlg, db, dstate).  `save`
    must match the fwd_vg call that wrote ckpt."""
    d = _dims_of(q, v, algo, save)
    _check_inputs_vg(d, q, k, v, lg, b, state0, mask)
    dev = q.device
    _check(dO, "dO", (d.B, d.T, d.Hv, d.Dv), q.dtype, dev)
    if dS_final is not None:
        _check(dS_final, "dS_final", (d.B, d.Hv, d.Dk, d.Dv), torch.float32, dev)
    nck = vg_ckpt_elems(d)
    if nck:
        if ckpt is None or ckpt.numel() != nck:
            raise ValueError("ckpt from gdn_fwd_vg with %d elements is required" % nck)
        if ckpt.dtype != torch.float32 or not ckpt.is_contiguous() or ckpt.device != dev:
            raise ValueError("ckpt must be a contiguous fp32 tensor on %s" % dev)
    out = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
               dlg=torch.empty_like(lg), db=torch.empty_like(b),
               dstate=torch.empty((d.B, d.Hv, d.Dk, d.Dv), dtype=torch.float32, device=dev))
    wsb = _query("gdn_bwd_vg_workspace_bytes", d)
    ws = torch.empty((max(wsb, 1),), dtype=torch.uint8, device=dev)
    rc = lib().gdn_bwd_vg(ctypes.byref(d), _p(q), _p(k), _p(v), _p(lg), _p(b), _p(state0),
                          _p(mask), _p(ckpt) if nck else None, _p(dO), _p(dS_final),
                          *[_p(out[n]) for n in ("dq", "dk", "dv", "dlg", "db", "dstate")],
                          _p(ws), wsb, _stream(dev))
    if rc:
        raise GdnError("gdn_bwd_vg", rc)
    return out


class PlanVg:
    """Plan (above) for the per-key-channel-gate form: `t` maps q, k, v, lg,
    b, state0, mask, dO, dS_final to device tensors."""

    def __init__(self, t, algo=ALGO_AUTO, stream=None, save=False):
        q, v = t["q"], t["v"]
        self.d = d = _dims_of(q, v, algo, save)
        self.family = "chunk" if vg_uses_chunk(d) else "scan"
        _check_inputs_vg(d, q, t["k"], v, t["lg"], t["b"], t["state0"], t["mask"])
        dev = q.device
        self.t = t
        self.o = torch.empty((d.B, d.T, d.Hv, d.Dv), dtype=q.dtype, device=dev)
        self.state_out = torch.empty((d.B, d.Hv, d.Dk, d.Dv), dtype=torch.float32, device=dev)
        self.ckpt = _alloc_ckpt(d, dev, vg=True)
        nck = self.ckpt.numel()
        self.g = dict(dq=torch.empty_like(q), dk=torch.empty_like(t["k"]), dv=torch.empty_like(v),
                      dlg=torch.empty_like(t["lg"]), db=torch.empty_like(t["b"]),
                      dstate=torch.empty((d.B, d.Hv, d.Dk, d.Dv), dtype=torch.float32, device=dev))
        fws = _query("gdn_fwd_vg_workspace_bytes", d)
        bws = _query("gdn_bwd_vg_workspace_bytes", d)
        self.ws_f = torch.empty((max(fws, 1),), dtype=torch.uint8, device=dev)
        self.ws_b = torch.empty((max(bws, 1),), dtype=torch.uint8, device=dev)
        st = stream if stream is not None else torch.cuda.current_stream(dev)
        self.stream = st
        sp = ctypes.c_void_p(st.cuda_stream)
        ck = _p(self.ckpt) if nck else None
        ins = [_p(t[n]) for n in ("q", "k", "v", "lg", "b", "state0", "mask")]
        self._fargs = (ctypes.byref(d), *ins, _p(self.o), _p(self.state_out), ck,
                       _p(self.ws_f), fws, sp)
        self._bargs = (ctypes.byref(d), *ins, ck, _p(t["dO"]), _p(t["dS_final"]),
                       *[_p(self.g[n]) for n in ("dq", "dk", "dv", "dlg", "db", "dstate")],
                       _p(self.ws_b), bws, sp)
        self.fwd_ws_bytes, self.bwd_ws_bytes = fws, bws

    def fwd(self):
        rc = lib().gdn_fwd_vg(*self._fargs)
        if rc:
            raise GdnError("gdn_fwd_vg", rc)

    def bwd(self):
        rc = lib().gdn_bwd_vg(*self._bargs)
        if rc:
            raise GdnError("gdn_bwd_vg", rc)


def decode_conv(x, conv_w, conv_state, a, b, A_log, dt_bias, Hk, Dk, Hv, Dv, state0=None,
                mask=None, *, conv_state_out=None, state_out=None):
    """One decode step preceded by the conv update (gdn_decode_conv).

    x: [B, C] (C = 2 Hk Dk + Hv Dv: q, k, v channels); conv_w: [C, K];
    conv_state: [B, C, K]; a, b: [B, Hv]; A_log, dt_bias: [Hv] fp32; state0:
    [B, Hv, Dk, Dv] fp32 or None; mask: [B] uint8 or None.  Pass
    conv_state_out=conv_state and / or state_out=state0 to update in place.
    Returns (o [B, Hv, Dv], state_out, conv_state_out)."""
    B, C = x.shape
    K = conv_w.shape[1]
    dt, dev = x.dtype, x.device
    if C != 2 * Hk * Dk + Hv * Dv:
        raise ValueError("x has %d channels, expected 2 Hk Dk + Hv Dv = %d" % (C, 2 * Hk * Dk + Hv * Dv))
    d = make_dims(B, 1, Hk, Hv, Dk, Dv, dt)
    _check(x, "x", (B, C), dt, dev)
    _check(conv_w, "conv_w", (C, K), dt, dev)
    _check(conv_state, "conv_state", (B, C, K), dt, dev)
    _check(a, "a", (B, Hv), dt, dev)
    _check(b, "b", (B, Hv), dt, dev)
    _check(A_log, "A_log", (Hv,), torch.float32, dev)
    _check(dt_bias, "dt_bias", (Hv,), torch.float32, dev)
    if state0 is not None:
        _check(state0, "state0", (B, Hv, Dk, Dv), torch.float32, dev)
    if mask is not None:
        _check(mask, "mask", (B,), torch.uint8, dev)
    if conv_state_out is None:
        conv_state_out = torch.empty_like(conv_state)
    else:
        _check(conv_state_out, "conv_state_out", (B, C, K), dt, dev)
    if state_out is None:
        state_out = torch.empty((B, Hv, Dk, Dv), dtype=torch.float32, device=dev)
    else:
        _check(state_out, "state_out", (B, Hv, Dk, Dv), torch.float32, dev)
    o = torch.empty((B, Hv, Dv), dtype=dt, device=dev)
    rc = lib().gdn_decode_conv(ctypes.byref(d), _p(x), _p(conv_w), _p(conv_state), _p(conv_state_out), K,
                               _p(a), _p(b), _p(A_log), _p(dt_bias), _p(state0), _p(mask), _p(o),
                               _p(state_out), _stream(dev))
    if rc:
        raise GdnError("gdn_decode_conv", rc)
    return o, state_out, conv_state_out


# The entry points below are also called for single tokens, where a call's time on
# the host counts: pointers go as plain integers, the current device is only switched
# where it is another one, and the decay entries' dims are made and their sizes asked
# for once for each set of them (the norm's, which also hold the strides, at every
# call).

def _a(x):
    return None if x is None else x.data_ptr()


@functools.lru_cache(maxsize=256)
def _decay_dims(query, *dims):
    """(dims, workspace bytes)"""
    d = make_dims(*dims)
    return d, _query(query, d)


_here = contextlib.nullcontext()


def _on_device(dev):
    """The context of a call on dev's tensors."""
    return _here if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


def _cotangent(x):
    """A gradient as the entries take it: dense, and at 16 bytes (autograd hands on
    views into larger gradients, which may begin anywhere)."""
    x = x.contiguous()
    return x if x.data_ptr() % 16 == 0 else x.clone()


# the handle of a device's current stream, without the object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


# ---- linear attention with a decay for each head (gdn_decay_fwd / gdn_decay_bwd)

def _check_decay(query, q, k, v, lg, state0, mask, algo):
    """(dims, workspace bytes, shape of the states) of checked arguments."""
    dev, dt = q.device, q.dtype
    if dev.type != "cuda":
        raise ValueError("gdn runs on the GPU; got device %s" % dev)
    if dt != torch.bfloat16 and dt != torch.float32:
        raise TypeError("q: expected float32 or bfloat16, got %s" % dt)
    B, T, Hk, Dk = q.shape
    Hv, Dv = v.shape[2], v.shape[3]
    states = (B, Hv, Dk, Dv)
    _check(q, "q", (B, T, Hk, Dk), dt, dev)
    _check(k, "k", (B, T, Hk, Dk), dt, dev)
    _check(v, "v", (B, T, Hv, Dv), dt, dev)
    _check(lg, "lg", (Hv,), torch.float32, dev)
    if state0 is not None:
        _check(state0, "state0", states, torch.float32, dev)
    if mask is not None:
        _check(mask, "mask", (B, T), torch.uint8, dev)
    d, wsb = _decay_dims(query, B, T, Hk, Hv, Dk, Dv, dt, algo)
    return d, wsb, states


def decay_fwd(q, k, v, lg, state0=None, mask=None, *, scale=None, state_out=None, algo=ALGO_AUTO):
    """Linear attention with a decay for each head (gdn_decay_fwd): S <- e^lg S
    + k v^T, o = scale S^T q (scale: Dk^-1/2 by default), T = 1 for a single
    token.  Returns (o, state_out).  Pass state_out=state0 to update the state
    in place."""
    d, wsb, states = _check_decay("gdn_decay_fwd_workspace_bytes", q, k, v, lg, state0, mask, algo)
    dev = q.device
    if state_out is None:
        state_out = (torch.empty(states, dtype=torch.float32, device=dev) if state0 is None
                     else torch.empty_like(state0))
    else:
        _check(state_out, "state_out", states, torch.float32, dev)
    o = torch.empty_like(v)
    ws = torch.empty((wsb,), dtype=torch.uint8, device=dev) if wsb else None
    with _on_device(dev):
        rc = lib().gdn_decay_fwd(d, _a(q), _a(k), _a(v), _a(lg), states[2] ** -0.5 if scale is None else scale,
                                 _a(state0), _a(mask), _a(o), _a(state_out), _a(ws), wsb,
                                 _raw_stream(dev.index))
    if rc:
        raise GdnError("gdn_decay_fwd", rc)
    return o, state_out


def decay_bwd(q, k, v, lg, state0, mask, dO, dS_final=None, *, scale=None, algo=ALGO_AUTO):
    """VJP of decay_fwd.  Returns dict(dq, dk, dv, dlg, dstate)."""
    d, wsb, states = _check_decay("gdn_decay_bwd_workspace_bytes", q, k, v, lg, state0, mask, algo)
    dev = q.device
    _check(dO, "dO", v.shape, q.dtype, dev)
    if dS_final is not None:
        _check(dS_final, "dS_final", states, torch.float32, dev)
    out = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
               dlg=torch.empty_like(lg),
               dstate=torch.empty(states, dtype=torch.float32, device=dev))
    ws = torch.empty((wsb,), dtype=torch.uint8, device=dev) if wsb else None
    with _on_device(dev):
        rc = lib().gdn_decay_bwd(d, _a(q), _a(k), _a(v), _a(lg), states[2] ** -0.5 if scale is None else scale,
                                 _a(state0), _a(mask), _a(dO), _a(dS_final),
                                 *[_a(out[n]) for n in ("dq", "dk", "dv", "dlg", "dstate")], _a(ws), wsb,
                                 _raw_stream(dev.index))
    if rc:
        raise GdnError("gdn_decay_bwd", rc)
    return out


class DecayAttention(torch.autograd.Function):
    """Autograd wrapper of decay_fwd / decay_bwd: forward(q, k, v, lg, state0,
    mask, scale) returns (o, state_out)."""

    @staticmethod
    def forward(ctx, q, k, v, lg, state0=None, mask=None, scale=None):
        o, st = decay_fwd(q, k, v, lg, state0, mask, scale=scale)
        ctx.save_for_backward(q, k, v, lg, state0, mask)
        ctx.scale = scale
        ctx.set_materialize_grads(False)  # a loss that does not use the state has no dS to read
        return o, st

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dO, dS):
        if dO is None and dS is None:
            return (None,) * 7
        q, k, v, lg, state0, mask = ctx.saved_tensors
        g = decay_bwd(q, k, v, lg, state0, mask, torch.zeros_like(v) if dO is None else _cotangent(dO),
                      None if dS is None else _cotangent(dS), scale=ctx.scale)
        return (g["dq"], g["dk"], g["dv"], g["dlg"], g["dstate"] if state0 is not None else None, None, None)


# ---- norm of queries and keys with rotation (gdn_norm_rope_fwd / gdn_norm_rope_bwd)

def rope_table(P, R, base=10000.0, device="cuda"):
    """The table of norm_rope: cos and sin of position * base^(-2i/R), computed
    in 64 bits, as [P, R] fp32 (R/2 cosines, then R/2 sines)."""
    f = base ** (-torch.arange(0, R, 2, dtype=torch.float64, device=device) / max(R, 1))
    a = torch.arange(P, dtype=torch.float64, device=device)[:, None] * f[None]
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def _token_stride(x, name):
    """Elements between the rows of consecutive tokens of [B, T, H, D]; the
    heads of a token are dense, the tokens evenly spaced over batch and time."""
    if x.is_contiguous():
        return 0
    B, T, H, D = x.shape
    sb, st, sh, sd = x.stride()
    if (D > 1 and sd != 1) or (H > 1 and sh != D):
        raise ValueError("%s: the heads of a token must be contiguous" % name)
    st = st if T > 1 else sb if B > 1 else H * D
    if st < H * D or (B > 1 and T > 1 and sb != T * st):
        raise ValueError("%s: tokens must be evenly spaced over batch and time, without overlap" % name)
    return st


def _norm_dims(q, k, wq, wk, rope, pos, eps, w_offset, interleaved):
    dev, dt = q.device, q.dtype
    if dev.type != "cuda":
        raise ValueError("gdn runs on the GPU; got device %s" % dev)
    if dt != torch.bfloat16 and dt != torch.float32:
        raise TypeError("q: expected float32 or bfloat16, got %s" % dt)
    B, T, Hq, D = q.shape
    Hk = k.shape[2]
    if k.dtype != dt:
        raise TypeError("k: expected %s, got %s" % (dt, k.dtype))
    if k.shape != (B, T, Hk, D) or k.device != dev:
        raise ValueError("k: expected shape %s on %s, got %s on %s" % ((B, T, Hk, D), dev, tuple(k.shape), k.device))
    for w, name in ((wq, "wq"), (wk, "wk")):
        if w is not None:
            _check(w, name, (D,), torch.float32, dev)
    P, R = 0, 0
    if rope is not None:
        P, R = rope.shape
        _check(rope, "rope", (P, R), torch.float32, dev)
    if pos is not None:
        _check(pos, "pos", (B, T), torch.int32, dev)
    return NormDims(B, T, Hq, Hk, D, R, P, _token_stride(q, "q"), _token_stride(k, "k"),
                    GDN_F32 if dt == torch.float32 else GDN_BF16, 1 if interleaved else 0, eps, w_offset)


def norm_rope(q, k, wq, wk, rope=None, pos=None, *, eps=1e-6, w_offset=0.0, interleaved=False):
    """RMS norm of every head of q [B,T,Hq,D] and k [B,T,Hk,D] with weights wq,
    wk [D] fp32 (plus w_offset) and rotation of their first R channels by the
    table rope [P,R] at positions pos [B,T] int32 (0 .. T-1 by default), in one
    pass.  q and k may be slices of a packed projection.  Returns dense (q, k)."""
    d = _norm_dims(q, k, wq, wk, rope, pos, eps, w_offset, interleaved)
    dev, dt = q.device, q.dtype
    oq = torch.empty((d.B, d.T, d.Hq, d.D), dtype=dt, device=dev)
    ok = torch.empty((d.B, d.T, d.Hk, d.D), dtype=dt, device=dev)
    with _on_device(dev):
        rc = lib().gdn_norm_rope_fwd(d, _a(q), _a(k), _a(wq), _a(wk), _a(rope), _a(pos), _a(oq), _a(ok),
                                     _raw_stream(dev.index))
    if rc:
        raise GdnError("gdn_norm_rope_fwd", rc)
    return oq, ok


def norm_rope_bwd(q, k, wq, wk, rope, pos, dyq, dyk, *, eps=1e-6, w_offset=0.0, interleaved=False):
    """VJP of norm_rope.  Returns dict(dq, dk, dwq, dwk), dq and dk dense."""
    d = _norm_dims(q, k, wq, wk, rope, pos, eps, w_offset, interleaved)
    dev = q.device
    _check(dyq, "dyq", q.shape, q.dtype, dev)
    _check(dyk, "dyk", k.shape, q.dtype, dev)
    out = dict(dq=torch.empty_like(dyq), dk=torch.empty_like(dyk), dwq=torch.empty_like(wq),
               dwk=torch.empty_like(wk))
    wsb = _query("gdn_norm_rope_bwd_workspace_bytes", d)
    ws = torch.empty((wsb,), dtype=torch.uint8, device=dev) if wsb else None
    with _on_device(dev):
        rc = lib().gdn_norm_rope_bwd(d, _a(q), _a(k), _a(wq), _a(wk), _a(rope), _a(pos), _a(dyq), _a(dyk),
                                     *[_a(out[n]) for n in ("dq", "dk", "dwq", "dwk")], _a(ws), wsb,
                                     _raw_stream(dev.index))
    if rc:
        raise GdnError("gdn_norm_rope_bwd", rc)
    return out


class NormRope(torch.autograd.Function):
    """Autograd wrapper of norm_rope / norm_rope_bwd: forward(q, k, wq, wk, rope,
    pos, eps, w_offset, interleaved) returns (q, k)."""

    @staticmethod
    def forward(ctx, q, k, wq, wk, rope=None, pos=None, eps=1e-6, w_offset=0.0, interleaved=False):
        ctx.save_for_backward(q, k, wq, wk, rope, pos)
        ctx.kw = dict(eps=eps, w_offset=w_offset, interleaved=interleaved)
        return norm_rope(q, k, wq, wk, rope, pos, **ctx.kw)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dyq, dyk):
        q, k, wq, wk, rope, pos = ctx.saved_tensors
        g = norm_rope_bwd(q, k, wq, wk, rope, pos, _cotangent(dyq), _cotangent(dyk), **ctx.kw)
        return (g["dq"], g["dk"], g["dwq"], g["dwk"]) + (None,) * 5


# ---- rotation with positions on several axes (gdn_norm_rope_axes_fwd / _bwd)

def axis_map(pairs, cycle=False, device="cuda"):
    """The axis of each pair for the operators below: pairs[a] pairs turn by axis
    a's position, in blocks (pairs of axis 0 first), or with cycle=True one of each
    axis in turn while it has any left."""
    if cycle:
        left, out = list(pairs), []
        while any(left):
            for a in range(len(left)):
                if left[a]:
                    out.append(a)
                    left[a] -= 1
    else:
        out = [a for a, n in enumerate(pairs) for _ in range(n)]
    return torch.tensor(out, dtype=torch.uint8, device=device)


def _axes_of(d, rope, axis, pos, tokens, dev):
    """The number of axes of checked positions and axis map (without positions, as many
    as there can be: they are the same on all)."""
    if axis is not None:
        _check(axis, "axis", (rope.shape[1] // 2 if rope is not None else 0,), torch.uint8, dev)
    if pos is None:
        return 4
    if pos.dim() != 1 + len(tokens) or not 1 <= pos.shape[0] <= 4:
        raise ValueError("pos: expected shape (1 .. 4 axes, %s), got %s" % (", ".join(map(str, tokens)), tuple(pos.shape)))
    _check(pos, "pos", (pos.shape[0], *tokens), torch.int32, dev)
    return pos.shape[0]


def norm_rope_axes(q, k, wq=None, wk=None, rope=None, axis=None, pos=None, *, eps=1e-6, w_offset=0.0,
                   interleaved=False):
    """norm_rope with positions on up to four axes: pos [A,B,T] int32, axis [R/2]
    uint8 the axis of each pair (axis_map).  Without wq and wk, the rotation alone."""
    if _calls is not None:
        out = _calls.norm_rope_axes(q, k, wq, wk, rope, axis, pos, eps, w_offset, interleaved)
        if out is not NotImplemented:
            return out
    d, A = _norm_axes_dims(q, k, wq, wk, rope, axis, pos, eps, w_offset, interleaved)
    dev, dt = q.device, q.dtype
    oq = torch.empty((d.B, d.T, d.Hq, d.D), dtype=dt, device=dev)
    ok = torch.empty((d.B, d.T, d.Hk, d.D), dtype=dt, device=dev)
    with _on_device(dev):
        rc = lib().gdn_norm_rope_axes_fwd(d, A, _a(q), _a(k), _a(wq), _a(wk), _a(rope), _a(axis), _a(pos), _a(oq),
                                          _a(ok), _raw_stream(dev.index))
    if rc:
        raise GdnError("gdn_norm_rope_axes_fwd", rc)
    return oq, ok


def _norm_axes_dims(q, k, wq, wk, rope, axis, pos, eps, w_offset, interleaved):
    if (wq is None) != (wk is None):
        raise ValueError("wq and wk: both, or neither")
    d = _norm_dims(q, k, wq, wk, rope, None, eps, w_offset, interleaved)
    return d, _axes_of(d, rope, axis, pos, (d.B, d.T), q.device)


def norm_rope_axes_bwd(q, k, wq, wk, rope, axis, pos, dyq, dyk, *, eps=1e-6, w_offset=0.0, interleaved=False):
    """VJP of norm_rope_axes.  Returns dict(dq, dk, dwq, dwk), dq and dk dense, dwq and
    dwk None without the norm, where of q and k only the shapes are used."""
    if _calls is not None:
        out = _calls.norm_rope_axes_bwd(q, k, wq, wk, rope, axis, pos, eps, w_offset, interleaved, dyq, dyk)
        if out is not NotImplemented:
            return out
    d, A = _norm_axes_dims(q, k, wq, wk, rope, axis, pos, eps, w_offset, interleaved)
    dev = q.device
    _check(dyq, "dyq", q.shape, q.dtype, dev)
    _check(dyk, "dyk", k.shape, q.dtype, dev)
    out = dict(dq=torch.empty_like(dyq), dk=torch.empty_like(dyk), dwq=None if wq is None else torch.empty_like(wq),
               dwk=None if wk is None else torch.empty_like(wk))
    wsb = 0 if wq is None else _query("gdn_norm_rope_bwd_workspace_bytes", d)
    ws = torch.empty((wsb,), dtype=torch.uint8, device=dev) if wsb else None
    with _on_device(dev):
        rc = lib().gdn_norm_rope_axes_bwd(d, A, _a(q), _a(k), _a(wq), _a(wk), _a(rope), _a(axis), _a(pos), _a(dyq),
                                          _a(dyk), *[_a(out[n]) for n in ("dq", "dk", "dwq", "dwk")], _a(ws), wsb,
                                          _raw_stream(dev.index))
    if rc:
        raise GdnError("gdn_norm_rope_axes_bwd", rc)
    return out


class NormRopeAxes(torch.autograd.Function):
    """Autograd wrapper of norm_rope_axes / norm_rope_axes_bwd: forward(q, k, wq, wk,
    rope, axis, pos, eps, w_offset, interleaved) returns (q, k).  To capture a step into
    a graph, drop what earlier eager steps of the same leaves returned first, and warm up
    on the capture's stream: torch adds a leaf's gradient on the stream of the graph that
    still holds it, which ends a capture on another one.  norm_rope_axes_bwd itself may
    be captured anywhere."""

    @staticmethod
    def forward(ctx, q, k, wq=None, wk=None, rope=None, axis=None, pos=None, eps=1e-6, w_offset=0.0, interleaved=False):
        # (without the norm the VJP reads neither q nor k)
        ctx.save_for_backward(*((q, k) if wq is not None else (None, None)), wq, wk, rope, axis, pos)
        ctx.kw = dict(eps=eps, w_offset=w_offset, interleaved=interleaved)
        return norm_rope_axes(q, k, wq, wk, rope, axis, pos, **ctx.kw)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dyq, dyk):
        q, k, wq, wk, rope, axis, pos = ctx.saved_tensors
        dyq, dyk = _cotangent(dyq), _cotangent(dyk)
        if wq is None:
            q, k = dyq, dyk  # for their shapes
        g = norm_rope_axes_bwd(q, k, wq, wk, rope, axis, pos, dyq, dyk, **ctx.kw)
        return (g["dq"], g["dk"], g["dwq"], g["dwk"]) + (None,) * 6


# ---- keys and values in pages (gdn_paged_append, gdn_prefix_attention)

class _NoBackward(torch.autograd.Function):
    """Results of an operator that has no backward pass, from inputs that require a
    gradient: whoever asks for one is told so.  forward(name, n, *n results, *inputs)."""

    @staticmethod
    def forward(ctx, name, n, *tensors):
        ctx.name = name
        ctx.mark_dirty(*tensors[:n])
        return tensors[:n]

    @staticmethod
    def backward(ctx, *_):
        raise NotImplementedError("%s has no backward pass (it serves from a cache)" % ctx.name)


def _wants_grad(tensors):
    return torch.is_grad_enabled() and any(x is not None and x.requires_grad for x in tensors)


def _without_backward(name, results, inputs):
    """The results, behind a node that raises where any of the inputs requires a gradient."""
    if not _wants_grad(inputs):
        return results
    return _NoBackward.apply(name, len(results), *results, *[x for x in inputs if x is not None])


def _no_out(name, inputs):
    if _wants_grad(inputs):
        raise RuntimeError("%s: out= with arguments that require a gradient (it has no backward pass; call it under "
                           "torch.no_grad())" % name)


def _rows_stride(x, name, shape):
    """Elements between the rows of consecutive tokens of [N, H, D] (0: dense)."""
    if tuple(x.shape) != shape:
        raise ValueError("%s: expected shape %s, got %s" % (name, shape, tuple(x.shape)))
    if x.is_contiguous():
        return 0
    N, H, D = shape
    sn, sh, sd = x.stride()
    if (D > 1 and sd != 1) or (H > 1 and sh != D) or (N > 1 and sn < H * D):
        raise ValueError("%s: the heads of a token must be contiguous, and tokens must not overlap" % name)
    return sn if N > 1 else 0


@functools.lru_cache(maxsize=256)
def _paged_dims(*dims):
    return PagedDims(*dims)


@functools.lru_cache(maxsize=256)
def _turn_dims(*dims):
    return Turn(*dims)


@functools.lru_cache(maxsize=256)
def _attention_ws(prefix, max_q, max_len, *dims):
    out = ctypes.c_size_t(0)
    rc = lib().gdn_prefix_attention_workspace_bytes(_paged_dims(*dims), prefix, max_q, max_len, ctypes.byref(out))
    if rc:
        hint = "; the launch goes by max_q = %d for each of %d sequences: give the longest one's tokens" % (max_q, dims[1])
        raise GdnError("gdn_prefix_attention_workspace_bytes", rc, hint if STATUS.get(rc) == "GDN_ERR_UNSUPPORTED" else "")
    return out.value


def _check_pool(k_pages, v_pages, table, cu, N, Hq, dt, dev):
    """The dims of a checked pool and table."""
    if dev.type != "cuda":
        raise ValueError("gdn runs on the GPU; got device %s" % dev)
    if dt != torch.bfloat16 and dt != torch.float32:
        raise TypeError("expected float32 or bfloat16, got %s" % dt)
    pages, Hk, page, D = k_pages.shape
    for x, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
        if x.dtype != dt:
            raise TypeError("%s: expected %s, got %s" % (name, dt, x.dtype))
        if x.shape != k_pages.shape or x.device != dev:
            raise ValueError("%s: expected shape %s on %s, got %s on %s" % (name, tuple(k_pages.shape), dev,
                                                                            tuple(x.shape), x.device))
    strides = k_pages.stride()
    if v_pages.stride() != strides or (D > 1 and strides[3] != 1):
        raise ValueError("k_pages and v_pages: expected the same strides, and contiguous rows")
    S, width = table.shape
    _check(table, "table", (S, width), torch.int32, dev)
    if S < 1:
        raise ValueError("table: expected a row for each sequence, got none")
    if cu is not None:
        _check(cu, "cu", (S + 1,), torch.int32, dev)
    return (N, S, Hq, Hk, D, pages, page, width, strides[0], strides[1], strides[2],
            GDN_F32 if dt == torch.float32 else GDN_BF16)


def paged_append(q, k, v, k_pages, v_pages, table, past, cu=None, *, wq=None, wk=None, rope=None, axis=None, pos=None,
                 first=0, eps=1e-6, w_offset=0.0, interleaved=False, out=None):
    """Appends the tokens of a call to a paged cache (gdn_paged_append): queries q
    [N,Hq,D] and keys k [N,Hk,D] with the norm and the rotation of norm_rope_axes,
    values v [N,Hk,D] as they are.  Keys and values go into k_pages, v_pages
    [pages,Hk,page,D] (any strides with contiguous rows, the same for both), to place
    past[s] + i of sequence s, whose pages are table[s].  Sequence s has the tokens
    cu[s] .. cu[s+1] - 1, or N / S tokens each.  q, k, v may be slices of a packed
    projection; q may be None.  Returns the turned queries (in out, if given).  There is no
    backward pass: one that reaches the result raises, and the pools hold values alone."""
    if _calls is not None:
        y = _calls.paged_append(q, k, v, k_pages, v_pages, table, past, cu, wq, wk, rope, axis, pos, first, eps, w_offset,
                                interleaved, out)
        if y is not NotImplemented:
            return y
    N, Hk, D = k.shape
    dev, dt = k.device, k.dtype
    Hq = 0 if q is None else q.shape[1]
    dims = _check_pool(k_pages, v_pages, table, cu, N, Hq, dt, dev)
    if dims[3] != Hk or dims[4] != D:
        raise ValueError("k: expected %d heads of %d, got %d of %d" % (dims[3], dims[4], Hk, D))
    for x, name in ((q, "q"), (v, "v")):
        if x is not None and x.dtype != dt:
            raise TypeError("%s: expected %s, got %s" % (name, dt, x.dtype))
        if x is not None and x.device != dev:
            raise ValueError("%s: expected device %s, got %s" % (name, dev, x.device))
    _check(past, "past", (dims[1],), torch.int32, dev)
    for x, name in ((wq, "wq"), (wk, "wk")):
        if x is not None:
            _check(x, name, (D,), torch.float32, dev)
    P, R = 0, 0
    if rope is not None:
        P, R = rope.shape
        _check(rope, "rope", (P, R), torch.float32, dev)
    A = _axes_of(None, rope, axis, pos, (N,), dev)
    given = False
    if q is None:
        qs = 0
        if out is not None:
            raise ValueError("out without q")
    else:
        qs = _rows_stride(q, "q", (N, Hq, D))
        if out is None:
            out = torch.empty((N, Hq, D), dtype=dt, device=dev)
        else:
            _check(out, "out", (N, Hq, D), dt, dev)
            _no_out("paged_append", (q, k, v, k_pages, v_pages, wq, wk, out))
            given = True
    turn = _turn_dims(P, R, qs, _rows_stride(k, "k", (N, Hk, D)), _rows_stride(v, "v", (N, Hk, D)), first, A,
                      1 if interleaved else 0, eps, w_offset)
    with _on_device(dev):
        rc = lib().gdn_paged_append(_paged_dims(*dims), turn, _a(q), _a(k), _a(v), _a(wq), _a(wk), _a(rope), _a(axis),
                                    _a(pos), _a(table), _a(past), _a(cu), _a(out), _a(k_pages), _a(v_pages),
                                    _raw_stream(dev.index))
    if rc:
        raise GdnError("gdn_paged_append", rc)
    if out is None or given:
        return out
    return _without_backward("paged_append", (out,), (q, k, v, k_pages, v_pages, wq, wk))[0]


def prefix_attention(q, k_pages, v_pages, table, lens, prefix_pages=None, prefix=0, cu=None, *, max_q=None,
                     max_len=None, scale=None, out=None, lse=False):
    """Softmax attention of new tokens over a shared prefix and their sequences' own
    pages (gdn_prefix_attention): q [N,Hq,D] the tokens' queries, sequence s's being the
    last of its lens[s] own tokens in the pages table[s]; the prefix's first `prefix`
    tokens lie in prefix_pages.  cu as in paged_append.  max_q (N by default, with cu)
    and max_len (the room of a table's row) bound a sequence's tokens in the call and its
    own length: the launch goes by them, and one of many sequences that are all taken to
    be as long as the batch may be refused.  scale: D^-1/2 by default.  Returns o [N,Hq,D]
    (in out, if given), with lse=True (o, lse [N,Hq] fp32).  There is no backward pass: one
    that reaches the result raises."""
    if _calls is not None:
        y = _calls.prefix_attention(q, k_pages, v_pages, table, lens, prefix_pages, prefix, cu, max_q, max_len, scale, out,
                                    lse)
        if y is not NotImplemented:
            return y
    N, Hq, D = q.shape
    dev, dt = q.device, q.dtype
    dims = _check_pool(k_pages, v_pages, table, cu, N, Hq, dt, dev)
    S, page = dims[1], dims[6]
    _check(q, "q", (N, Hq, dims[4]), dt, dev)
    _check(lens, "lens", (S,), torch.int32, dev)
    if prefix_pages is not None:
        _check(prefix_pages, "prefix_pages", prefix_pages.shape, torch.int32, dev)
    if prefix and (prefix_pages is None or prefix_pages.dim() != 1 or prefix_pages.shape[0] * page < prefix):
        raise ValueError("prefix_pages: %d tokens of a prefix need %d pages" % (prefix, -(-prefix // page)))
    if max_len is None:
        max_len = min(dims[7] * page, 1 << 30)
    if cu is None:
        if N % S:
            raise ValueError("%d tokens of %d sequences: cu is needed" % (N, S))
        max_q = N // S
    elif max_q is None or max_q > N:
        max_q = N
    given = out is not None
    if given:
        _check(out, "out", q.shape, dt, dev)
        _no_out("prefix_attention", (q, k_pages, v_pages, out))
    else:
        out = torch.empty_like(q)
    sums = torch.empty((N, Hq), dtype=torch.float32, device=dev) if lse else None
    wsb = _attention_ws(prefix, max_q, max_len, *dims)
    ws = torch.empty((wsb,), dtype=torch.uint8, device=dev) if wsb else None
    with _on_device(dev):
        rc = lib().gdn_prefix_attention(_paged_dims(*dims), _a(q), _a(k_pages), _a(v_pages), _a(table), _a(lens),
                                        _a(prefix_pages) if prefix else None, prefix, _a(cu), max_q, max_len,
                                        dims[4] ** -0.5 if scale is None else scale, _a(out), _a(sums), _a(ws), wsb,
                                        _raw_stream(dev.index))
    if rc:
        raise GdnError("gdn_prefix_attention", rc)
    results = (out, sums) if lse else (out,)
    if not given:
        results = _without_backward("prefix_attention", results, (q, k_pages, v_pages))
    return results if lse else results[0]
