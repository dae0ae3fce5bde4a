"""Thin ctypes binding of libdplr (argument marshalling only).

Every step of the forward runs in the CUDA kernels of libdplr.so; PyTorch only
provides device memory and the stream. If the library is missing the calls
raise: there is no CPU or PyTorch fallback.
"""

from __future__ import annotations

import ctypes
import operator
import os
import struct
import threading
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdplr.so")

DPLR_OK, DPLR_ERR_INVALID_ARG, DPLR_ERR_UNSUPPORTED, DPLR_ERR_WORKSPACE, DPLR_ERR_CUDA, DPLR_ERR_TIMEOUT = range(6)
DPLR_GDN, DPLR_HDLA, DPLR_GENERIC = 1, 2, 3
DPLR_F32, DPLR_BF16 = 0, 1
MODES = {"gdn": DPLR_GDN, "hdla": DPLR_HDLA, "generic": DPLR_GENERIC}


class dplr_desc(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("in_dtype", ctypes.c_int32), ("B", ctypes.c_int32),
                ("H", ctypes.c_int32), ("T", ctypes.c_int32), ("dk", ctypes.c_int32), ("dv", ctypes.c_int32),
                ("r_ab", ctypes.c_int32), ("r_kv", ctypes.c_int32), ("chunk", ctypes.c_int32)]


class dplr_hd_tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("sb", ctypes.c_int64), ("sh", ctypes.c_int64), ("st", ctypes.c_int64)]


class dplr_hd_desc(ctypes.Structure):
    _fields_ = [("in_dtype", ctypes.c_int32), ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("Hq", ctypes.c_int32),
                ("T", ctypes.c_int32), ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("per_head", ctypes.c_int32)]


class DplrError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)}")
        self.status = status


_lock = threading.Lock()
_lib = None
_vp = ctypes.c_void_p


def library() -> ctypes.CDLL:
    """Loads libdplr.so (built in-tree by ``__graft_entry__.build()``)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
            lib = ctypes.CDLL(LIB_PATH)
            dp = ctypes.POINTER(dplr_desc)
            lib.dplr_la_workspace_size.restype = ctypes.c_size_t
            lib.dplr_la_workspace_size.argtypes = [dp]
            lib.dplr_la_stage_workspace_size.restype = ctypes.c_size_t
            lib.dplr_la_stage_workspace_size.argtypes = [dp]
            lib.dplr_la_check.restype = ctypes.c_int
            lib.dplr_la_check.argtypes = [dp]
            lib.dplr_la_kernel_count.restype = ctypes.c_int
            lib.dplr_la_kernel_count.argtypes = [dp]
            lib.dplr_status_string.restype = ctypes.c_char_p
            lib.dplr_status_string.argtypes = [ctypes.c_int]
            lib.dplr_la_forward.restype = ctypes.c_int
            lib.dplr_la_forward.argtypes = [dp] + [_vp] * 12 + [_vp, ctypes.c_size_t, _vp]
            lib.dplr_la_chunk_maps.restype = ctypes.c_int
            lib.dplr_la_chunk_maps.argtypes = [dp] + [_vp] * 10 + [_vp, ctypes.c_size_t, _vp]
            lib.dplr_la_state_scan.restype = ctypes.c_int
            lib.dplr_la_state_scan.argtypes = [dp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
            lib.dplr_la_forward_noalloc.restype = ctypes.c_int
            lib.dplr_la_forward_noalloc.argtypes = [dp] + [_vp] * 12 + [_vp]
            lib.dplr_la_decode_step.restype = ctypes.c_int
            lib.dplr_la_decode_step.argtypes = [dp] + [_vp] * 11 + [_vp]
            lib.dplr_la_backward_workspace_size.restype = ctypes.c_size_t
            lib.dplr_la_backward_workspace_size.argtypes = [dp]
            lib.dplr_la_backward.restype = ctypes.c_int
            lib.dplr_la_backward.argtypes = [dp] + [_vp] * 22 + [_vp, ctypes.c_size_t, _vp]
            lib.dplr_hla_workspace_size.restype = ctypes.c_size_t
            lib.dplr_hla_workspace_size.argtypes = [dp, ctypes.c_int]
            lib.dplr_hla_forward.restype = ctypes.c_int
            lib.dplr_hla_forward.argtypes = [dp] + [_vp] * 6 + [ctypes.c_float, ctypes.c_int, _vp, _vp, ctypes.c_size_t, _vp]
            lib.dplr_hla_path.restype = ctypes.c_char_p
            lib.dplr_hla_path.argtypes = [dp, ctypes.c_int]
            lib.dplr_gdp_workspace_size.restype = ctypes.c_size_t
            lib.dplr_gdp_workspace_size.argtypes = [dp]
            lib.dplr_gdp_forward.restype = ctypes.c_int
            lib.dplr_gdp_forward.argtypes = [dp] + [_vp] * 8 + [_vp, ctypes.c_size_t, _vp]
            lib.dplr_gdp_path.restype = ctypes.c_char_p
            lib.dplr_gdp_path.argtypes = [dp]
            lib.dplr_la_path.restype = ctypes.c_char_p
            lib.dplr_la_path.argtypes = [dp]
            lib.dplr_la_set_wait_limit.restype = None
            lib.dplr_la_set_wait_limit.argtypes = [ctypes.c_longlong]
            lib.dplr_la_read_status.restype = ctypes.c_int
            lib.dplr_la_read_status.argtypes = [_vp, ctypes.c_size_t, ctypes.c_int, ctypes.POINTER(ctypes.c_int), _vp]
            lib.dplr_la_noalloc_status.restype = ctypes.c_int
            lib.dplr_la_noalloc_status.argtypes = [ctypes.POINTER(ctypes.c_int), _vp]
            lib.dplr_la_host_workspace_size.restype = ctypes.c_size_t
            lib.dplr_la_host_workspace_size.argtypes = [dp, ctypes.c_int, ctypes.c_int]
            lib.dplr_la_forward_host.restype = ctypes.c_int
            lib.dplr_la_forward_host.argtypes = [dp] + [_vp] * 12 + [_vp, ctypes.c_size_t, ctypes.c_int,
                                                                     ctypes.c_int, _vp]
            lib.dplr_la_host_seq_workspace_size.restype = ctypes.c_size_t
            lib.dplr_la_host_seq_workspace_size.argtypes = [dp, ctypes.c_int, ctypes.c_int]
            lib.dplr_la_forward_host_seq.restype = ctypes.c_int
            lib.dplr_la_forward_host_seq.argtypes = [dp] + [_vp] * 12 + [_vp, ctypes.c_size_t, ctypes.c_int,
                                                                         ctypes.c_int, _vp]
            hp, tp, i32 = ctypes.POINTER(dplr_hd_desc), ctypes.POINTER(dplr_hd_tensor), ctypes.c_int32
            lib.dplr_hd_check.restype = ctypes.c_int
            lib.dplr_hd_check.argtypes = [hp]
            lib.dplr_hd_path.restype = ctypes.c_char_p
            lib.dplr_hd_path.argtypes = [hp]
            lib.dplr_hd_workspace_size.restype = ctypes.c_size_t
            lib.dplr_hd_workspace_size.argtypes = [hp]
            lib.dplr_hd_forward.restype = ctypes.c_int
            lib.dplr_hd_forward.argtypes = [hp, tp, tp, tp, tp, _vp, tp, _vp, _vp, ctypes.c_size_t, _vp]
            lib.dplr_hd_backward_workspace_size.restype = ctypes.c_size_t
            lib.dplr_hd_backward_workspace_size.argtypes = [hp]
            lib.dplr_hd_backward.restype = ctypes.c_int
            lib.dplr_hd_backward.argtypes = [hp, tp, tp, tp, tp, _vp, tp, _vp, tp, tp, tp, _vp, _vp, _vp,
                                             ctypes.c_size_t, _vp]
            lib.dplr_hd_plan.restype = ctypes.c_int
            lib.dplr_hd_plan.argtypes = [i32, i32, i32, i32] + [_vp] * 10
            lib.dplr_hd_packed_workspace_size.restype = ctypes.c_size_t
            lib.dplr_hd_packed_workspace_size.argtypes = [hp, i32, i32]
            lib.dplr_hd_forward_packed.restype = ctypes.c_int
            lib.dplr_hd_forward_packed.argtypes = [hp, i32, i32, i32, _vp, _vp, _vp, _vp, tp, tp, tp, tp, _vp, tp, _vp,
                                                   ctypes.c_size_t, _vp]
            lib.dplr_hd_decode_step.restype = ctypes.c_int
            lib.dplr_hd_decode_step.argtypes = [hp, i32, _vp, tp, tp, tp, tp, _vp, tp, _vp, _vp]
            _lib = lib
    return _lib


def status_string(status: int) -> str:
    return library().dplr_status_string(int(status)).decode()


def make_desc(mode: str | int, in_dtype, B: int, H: int, T: int, dk: int, dv: int,
              r_ab: Optional[int] = None, r_kv: Optional[int] = None, chunk: int = 64) -> dplr_desc:
    m = MODES[mode] if isinstance(mode, str) else int(mode)
    if in_dtype in (torch.bfloat16, "bf16", DPLR_BF16):
        dt = DPLR_BF16
    elif in_dtype in (torch.float32, "f32", DPLR_F32):
        dt = DPLR_F32
    else:
        raise ValueError(f"unsupported input dtype {in_dtype}")
    if r_ab is None:
        r_ab = {DPLR_GDN: 1, DPLR_HDLA: 2}.get(m, 1)
    if r_kv is None:
        r_kv = 1
    return dplr_desc(m, dt, B, H, T, dk, dv, r_ab, r_kv, chunk)


# ----------------------------------------------------------------------------
# C-ABI mirrors (raw pointers as Python ints, stream as an int handle).
# ----------------------------------------------------------------------------

def dplr_la_workspace_size(desc: dplr_desc) -> int:
    return int(library().dplr_la_workspace_size(ctypes.byref(desc)))


def dplr_la_stage_workspace_size(desc: dplr_desc) -> int:
    return int(library().dplr_la_stage_workspace_size(ctypes.byref(desc)))


def dplr_la_check(desc: dplr_desc) -> int:
    return int(library().dplr_la_check(ctypes.byref(desc)))


def dplr_la_kernel_count(desc: dplr_desc) -> int:
    return int(library().dplr_la_kernel_count(ctypes.byref(desc)))


def dplr_la_decode_step(desc, q, k, v, decay, beta, A, Bm, K, V, S, o, stream) -> int:
    """One recurrent step (desc.T == 1): S updated in place, o = S^T q."""
    return int(library().dplr_la_decode_step(ctypes.byref(desc), q, k, v, decay, beta, A, Bm, K, V, S, o, stream))


def dplr_la_backward_workspace_size(desc: dplr_desc) -> int:
    return int(library().dplr_la_backward_workspace_size(ctypes.byref(desc)))


def dplr_la_backward(desc, q, k, v, decay, beta, A, Bm, K, V, S0, dO, dST, dq, dk, dv, ddecay, dbeta, dA, dBm, dK,
                     dV, dS0, workspace, ws_bytes, stream) -> int:
    """Gradients of every input given dO and dS_T (device pointers; see include/dplr.h)."""
    return int(library().dplr_la_backward(ctypes.byref(desc), q, k, v, decay, beta, A, Bm, K, V, S0, dO, dST, dq, dk,
                                          dv, ddecay, dbeta, dA, dBm, dK, dV, dS0, workspace, ws_bytes, stream))


def dplr_hla_workspace_size(desc: dplr_desc, L: int) -> int:
    return int(library().dplr_hla_workspace_size(ctypes.byref(desc), int(L)))


def dplr_hla_forward(desc, q, k, v, g, beta, W, theta, L, o, workspace, ws_bytes, stream) -> int:
    """HLA's query-gated composition of GDN chunk transitions (device pointers; see include/dplr.h)."""
    return int(library().dplr_hla_forward(ctypes.byref(desc), q, k, v, g, beta, W, float(theta), int(L), o, workspace,
                                          ws_bytes, stream))


def dplr_hla_path(desc, L: int) -> str:
    return library().dplr_hla_path(ctypes.byref(desc), int(L)).decode()


def dplr_gdp_workspace_size(desc: dplr_desc) -> int:
    return int(library().dplr_gdp_workspace_size(ctypes.byref(desc)))


def dplr_gdp_forward(desc, q, k, v, g, beta, S0, o, S_T, workspace, ws_bytes, stream) -> int:
    """Stacked-Householder (Gated DeltaProduct-style) forward (device pointers; see include/dplr.h)."""
    return int(library().dplr_gdp_forward(ctypes.byref(desc), q, k, v, g, beta, S0, o, S_T, workspace, ws_bytes, stream))


def dplr_gdp_path(desc: dplr_desc) -> str:
    return library().dplr_gdp_path(ctypes.byref(desc)).decode()


def dplr_la_path(desc: dplr_desc) -> str:
    return library().dplr_la_path(ctypes.byref(desc)).decode()


def dplr_la_forward(desc, q, k, v, decay, beta, A, Bm, K, V, S0, o, S_T, workspace, ws_bytes, stream) -> int:
    return int(library().dplr_la_forward(ctypes.byref(desc), q, k, v, decay, beta, A, Bm, K, V, S0, o, S_T,
                                         workspace, ctypes.c_size_t(ws_bytes), stream))


def dplr_la_forward_noalloc(desc, q, k, v, decay, beta, A, Bm, K, V, S0, o, S_T, stream) -> int:
    """dplr_la_forward with scratch from the library's fixed device array (no workspace argument)."""
    return int(library().dplr_la_forward_noalloc(ctypes.byref(desc), q, k, v, decay, beta, A, Bm, K, V, S0, o,
                                                 S_T, stream))


def dplr_la_set_wait_limit(cycles: int) -> None:
    """Limit (SM cycles) of the kernels' bounded device-side waits; <= 0 restores the default."""
    library().dplr_la_set_wait_limit(int(cycles))


def dplr_la_read_status(workspace, ws_bytes, clear, stream) -> Tuple[int, int]:
    """Synchronous read of a workspace's device status word: (call status, word)."""
    word = ctypes.c_int(-1)
    st = int(library().dplr_la_read_status(workspace, ctypes.c_size_t(ws_bytes), int(clear), ctypes.byref(word),
                                           stream))
    return st, int(word.value)


def dplr_la_noalloc_status(stream) -> Tuple[int, int]:
    """Synchronous read of the no-alloc scratch array's status word: (call status, word)."""
    word = ctypes.c_int(-1)
    st = int(library().dplr_la_noalloc_status(ctypes.byref(word), stream))
    return st, int(word.value)


def dplr_la_host_workspace_size(desc, groups: int, slots: int) -> int:
    return int(library().dplr_la_host_workspace_size(ctypes.byref(desc), int(groups), int(slots)))


def dplr_la_forward_host(desc, q, k, v, decay, beta, A, Bm, K, V, S0, o, S_T, staging, staging_bytes, groups,
                         slots, stream) -> int:
    """dplr_la_forward with host inputs and outputs; transfers overlapped over groups of heads."""
    return int(library().dplr_la_forward_host(ctypes.byref(desc), q, k, v, decay, beta, A, Bm, K, V, S0, o, S_T,
                                              staging, ctypes.c_size_t(staging_bytes), int(groups), int(slots),
                                              stream))

def dplr_la_host_seq_workspace_size(desc, segments: int, slots: int) -> int:
    return int(library().dplr_la_host_seq_workspace_size(ctypes.byref(desc), int(segments), int(slots)))


def dplr_la_forward_host_seq(desc, q, k, v, decay, beta, A, Bm, K, V, S0, o, S_T, staging, staging_bytes, segments,
                         slots, stream) -> int:
    """dplr_la_forward with host inputs and outputs; transfers overlapped over segments of heads."""
    return int(library().dplr_la_forward_host_seq(ctypes.byref(desc), q, k, v, decay, beta, A, Bm, K, V, S0, o, S_T,
                                              staging, ctypes.c_size_t(staging_bytes), int(segments), int(slots),
                                              stream))


def dplr_la_chunk_maps(desc, q, k, v, decay, beta, A, Bm, K, V, o, workspace, ws_bytes, stream) -> int:
    return int(library().dplr_la_chunk_maps(ctypes.byref(desc), q, k, v, decay, beta, A, Bm, K, V, o,
                                            workspace, ctypes.c_size_t(ws_bytes), stream))


def dplr_la_state_scan(desc, S0, o, S_T, workspace, ws_bytes, stream) -> int:
    return int(library().dplr_la_state_scan(ctypes.byref(desc), S0, o, S_T, workspace,
                                            ctypes.c_size_t(ws_bytes), stream))


# ----------------------------------------------------------------------------
# Tensor-level wrapper.
# ----------------------------------------------------------------------------

def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _need(t, name, device, dtype, shape):
    if t is None:
        raise ValueError(f"{name} is required")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


class Forward:
    """Prepared forward for one descriptor: owns the output and workspace tensors so that
    repeated calls (benchmarks, CUDA graphs) allocate nothing."""

    def __init__(self, mode: str, in_dtype: torch.dtype, B: int, H: int, T: int, dk: int, dv: int,
                 r_ab: Optional[int] = None, r_kv: Optional[int] = None, chunk: int = 64,
                 device: Optional[torch.device] = None):
        self.desc = make_desc(mode, in_dtype, B, H, T, dk, dv, r_ab, r_kv, chunk)
        st = dplr_la_check(self.desc)
        if st != DPLR_OK:
            raise DplrError(st, "dplr_la_check")
        self.mode, self.in_dtype = MODES[mode] if isinstance(mode, str) else mode, in_dtype
        self.B, self.H, self.T, self.dk, self.dv = B, H, T, dk, dv
        self.r_ab, self.r_kv = self.desc.r_ab, self.desc.r_kv
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.ws_bytes = dplr_la_workspace_size(self.desc)
        # zeroed once: on the fused path its first int32 is the device status word
        self.workspace = torch.zeros(max(self.ws_bytes, 256), dtype=torch.uint8, device=self.device)
        self.stage_ws_bytes = dplr_la_stage_workspace_size(self.desc)
        self._stage_ws = None
        self.o = torch.empty((B, H, T, dv), dtype=torch.float32, device=self.device)
        self.S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=self.device)
        self.kernels = dplr_la_kernel_count(self.desc)
        self.path = dplr_la_path(self.desc)

    def _check(self, q, k, v, decay, beta, A, Bm, K, V, S0):
        B, H, T, dk, dv, dev, dt = self.B, self.H, self.T, self.dk, self.dv, self.device, self.in_dtype
        _need(q, "q", dev, dt, (B, H, T, dk))
        if self.mode == DPLR_GENERIC:
            _need(decay, "decay", dev, torch.float32, (B, H, T, dk))
            _need(A, "A", dev, dt, (B, H, T, self.r_ab, dk))
            _need(Bm, "Bm", dev, dt, (B, H, T, self.r_ab, dk))
            if self.r_kv > 0:
                _need(K, "K", dev, dt, (B, H, T, self.r_kv, dk))
                _need(V, "V", dev, dt, (B, H, T, self.r_kv, dv))
        else:
            _need(k, "k", dev, dt, (B, H, T, dk))
            _need(v, "v", dev, dt, (B, H, T, dv))
            _need(decay, "decay", dev, torch.float32, (B, H, T) if self.mode == DPLR_GDN else (B, H, T, dk))
            _need(beta, "beta", dev, torch.float32, (B, H, T))
        if S0 is not None:
            _need(S0, "S0", dev, torch.float32, (B, H, dk, dv))

    def __call__(self, q, k=None, v=None, decay=None, beta=None, A=None, Bm=None, K=None, V=None, S0=None,
                 stream: Optional[torch.cuda.Stream] = None, check: bool = True) -> Tuple[torch.Tensor, torch.Tensor]:
        if check:
            self._check(q, k, v, decay, beta, A, Bm, K, V, S0)
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        st = dplr_la_forward(self.desc, _ptr(q), _ptr(k), _ptr(v), _ptr(decay), _ptr(beta), _ptr(A), _ptr(Bm),
                             _ptr(K), _ptr(V), _ptr(S0), _ptr(self.o), _ptr(self.S_T), _ptr(self.workspace),
                             self.ws_bytes, s.cuda_stream)
        if st != DPLR_OK:
            raise DplrError(st, "dplr_la_forward")
        return self.o, self.S_T

    def device_status(self, clear: bool = False) -> int:
        """The workspace's device status word (0, or DPLR_ERR_TIMEOUT after a bounded wait gave up),
        read synchronously through dplr_la_read_status."""
        s = torch.cuda.current_stream(self.device)
        st, word = dplr_la_read_status(_ptr(self.workspace), self.workspace.numel(), clear, s.cuda_stream)
        if st != DPLR_OK:
            raise DplrError(st, "dplr_la_read_status")
        return word

    def _stage_workspace(self):
        if self._stage_ws is None:
            self._stage_ws = torch.empty(max(self.stage_ws_bytes, 256), dtype=torch.uint8, device=self.device)
        return self._stage_ws

    def chunk_maps(self, q, k=None, v=None, decay=None, beta=None, A=None, Bm=None, K=None, V=None,
                   stream: Optional[torch.cuda.Stream] = None):
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        st = dplr_la_chunk_maps(self.desc, _ptr(q), _ptr(k), _ptr(v), _ptr(decay), _ptr(beta), _ptr(A), _ptr(Bm),
                                _ptr(K), _ptr(V), _ptr(self.o), _ptr(self._stage_workspace()), self.stage_ws_bytes,
                                s.cuda_stream)
        if st != DPLR_OK:
            raise DplrError(st, "dplr_la_chunk_maps")

    def state_scan(self, S0=None, stream: Optional[torch.cuda.Stream] = None):
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        st = dplr_la_state_scan(self.desc, _ptr(S0), _ptr(self.o), _ptr(self.S_T), _ptr(self._stage_workspace()),
                                self.stage_ws_bytes, s.cuda_stream)
        if st != DPLR_OK:
            raise DplrError(st, "dplr_la_state_scan")
        return self.o, self.S_T


def default_groups(desc: dplr_desc) -> int:
    """Head groups for dplr_la_forward_host: enough groups to overlap the copies, while each
    group keeps enough heads to occupy the GPU (the fused kernel runs one CTA per head for the
    whole sequence, the two-stage kernels parallelise over chunks and want more heads)."""
    bh = desc.B * desc.H
    min_heads = 16 if dplr_la_kernel_count(desc) == 1 else 32
    best = 1
    for g in range(1, 17):
        if bh % g == 0 and bh // g >= min_heads:
            best = g
    return best


class ForwardHost:
    """Prepared forward from host (pinned) tensors through dplr_la_forward_host: owns the device
    staging area and pinned host outputs, so repeated calls allocate nothing."""

    def __init__(self, mode: str, in_dtype: torch.dtype, B: int, H: int, T: int, dk: int, dv: int,
                 r_ab: Optional[int] = None, r_kv: Optional[int] = None, chunk: int = 64,
                 groups: Optional[int] = None, slots: int = 8, device: Optional[torch.device] = None):
        self.desc = make_desc(mode, in_dtype, B, H, T, dk, dv, r_ab, r_kv, chunk)
        st = dplr_la_check(self.desc)
        if st != DPLR_OK:
            raise DplrError(st, "dplr_la_check")
        self.groups = groups if groups is not None else default_groups(self.desc)
        self.slots = slots
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.staging_bytes = dplr_la_host_workspace_size(self.desc, self.groups, self.slots)
        if self.staging_bytes == 0:
            raise DplrError(DPLR_ERR_INVALID_ARG, "dplr_la_host_workspace_size")
        self.staging = torch.empty(self.staging_bytes, dtype=torch.uint8, device=self.device)
        self.o = torch.empty((B, H, T, dv), dtype=torch.float32).pin_memory()
        self.S_T = torch.empty((B, H, dk, dv), dtype=torch.float32).pin_memory()

    def __call__(self, q, k=None, v=None, decay=None, beta=None, A=None, Bm=None, K=None, V=None, S0=None,
                 stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """Host tensors in, host tensors out (valid once `stream` has been synchronised)."""
        for name, t in (("q", q), ("k", k), ("v", v), ("decay", decay), ("beta", beta), ("A", A), ("Bm", Bm),
                        ("K", K), ("V", V), ("S0", S0)):
            if t is not None and (t.device.type != "cpu" or not t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous host tensor")
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        st = dplr_la_forward_host(self.desc, _ptr(q), _ptr(k), _ptr(v), _ptr(decay), _ptr(beta), _ptr(A), _ptr(Bm),
                                  _ptr(K), _ptr(V), _ptr(S0), _ptr(self.o), _ptr(self.S_T), _ptr(self.staging),
                                  self.staging_bytes, self.groups, self.slots, s.cuda_stream)
        if st != DPLR_OK:
            raise DplrError(st, "dplr_la_forward_host")
        return self.o, self.S_T


def default_segments(T: int) -> int:
    """Sequence segments for dplr_la_forward_host_seq: 4 up to 32K tokens, then one per 8K tokens (at most 16).
    Shorter segments shorten the tail after the last copy in, but each head's row of a 2-D copy shrinks
    with them, and rows well under ~0.5 MB copy slowly."""
    return 4 if T < 32768 else max(4, min(16, T // 8192))


class ForwardHostSeq:
    """Prepared forward from host (pinned) tensors through dplr_la_forward_host_seq (the sequence split
    into segments whose forwards carry the state on the device): owns the device staging area and pinned
    host outputs, so repeated calls allocate nothing."""

    def __init__(self, mode: str, in_dtype: torch.dtype, B: int, H: int, T: int, dk: int, dv: int,
                 r_ab: Optional[int] = None, r_kv: Optional[int] = None, chunk: int = 64,
                 segments: Optional[int] = None, slots: int = 4, device: Optional[torch.device] = None):
        self.desc = make_desc(mode, in_dtype, B, H, T, dk, dv, r_ab, r_kv, chunk)
        st = dplr_la_check(self.desc)
        if st != DPLR_OK:
            raise DplrError(st, "dplr_la_check")
        self.segments = segments if segments is not None else default_segments(T)
        self.slots = slots
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.staging_bytes = dplr_la_host_seq_workspace_size(self.desc, self.segments, self.slots)
        if self.staging_bytes == 0:
            raise DplrError(DPLR_ERR_INVALID_ARG, "dplr_la_host_seq_workspace_size")
        self.staging = torch.empty(self.staging_bytes, dtype=torch.uint8, device=self.device)
        self.o = torch.empty((B, H, T, dv), dtype=torch.float32).pin_memory()
        self.S_T = torch.empty((B, H, dk, dv), dtype=torch.float32).pin_memory()

    def __call__(self, q, k=None, v=None, decay=None, beta=None, A=None, Bm=None, K=None, V=None, S0=None,
                 stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """Host tensors in, host tensors out (valid once `stream` has been synchronised)."""
        for name, t in (("q", q), ("k", k), ("v", v), ("decay", decay), ("beta", beta), ("A", A), ("Bm", Bm),
                        ("K", K), ("V", V), ("S0", S0)):
            if t is not None and (t.device.type != "cpu" or not t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous host tensor")
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        st = dplr_la_forward_host_seq(self.desc, _ptr(q), _ptr(k), _ptr(v), _ptr(decay), _ptr(beta), _ptr(A),
                                      _ptr(Bm), _ptr(K), _ptr(V), _ptr(S0), _ptr(self.o), _ptr(self.S_T),
                                      _ptr(self.staging), self.staging_bytes, self.segments, self.slots,
                                      s.cuda_stream)
        if st != DPLR_OK:
            raise DplrError(st, "dplr_la_forward_host_seq")
        return self.o, self.S_T


def forward(mode: str, q, k=None, v=None, decay=None, beta=None, A=None, Bm=None, K=None, V=None, S0=None,
            chunk: int = 64) -> Tuple[torch.Tensor, torch.Tensor]:
    """One-shot forward on device tensors; returns fresh (o [B,H,T,dv] fp32, S_T [B,H,dk,dv] fp32)."""
    B, H, T, dk = q.shape
    if mode == "generic":
        r_ab, r_kv = A.shape[3], (K.shape[3] if K is not None else 0)
        dv = V.shape[4] if V is not None else S0.shape[3]
    else:
        r_ab, r_kv, dv = None, None, v.shape[3]
    f = Forward(mode, q.dtype, B, H, T, dk, dv, r_ab, r_kv, chunk, device=q.device)
    return f(q, k, v, decay, beta, A, Bm, K, V, S0)


class Decode:
    """Prepared one-token step for B x H heads (dplr_la_decode_step): owns the state S and the output o."""

    def __init__(self, mode: str, in_dtype: torch.dtype, B: int, H: int, dk: int, dv: int,
                 r_ab: Optional[int] = None, r_kv: Optional[int] = None, S0: Optional[torch.Tensor] = None,
                 device: Optional[torch.device] = None):
        self.desc = make_desc(mode, in_dtype, B, H, 1, dk, dv, r_ab, r_kv)
        st = dplr_la_check(self.desc)
        if st != DPLR_OK:
            raise DplrError(st, "dplr_la_check")
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.S = torch.zeros((B, H, dk, dv), dtype=torch.float32, device=self.device)
        if S0 is not None:
            self.S.copy_(S0)
        self.o = torch.empty((B, H, 1, dv), dtype=torch.float32, device=self.device)

    def __call__(self, q, k=None, v=None, decay=None, beta=None, A=None, Bm=None, K=None, V=None,
                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """One token (tensors with T = 1, contiguous, on the device). Returns o [B,H,1,dv]."""
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        st = dplr_la_decode_step(self.desc, _ptr(q), _ptr(k), _ptr(v), _ptr(decay), _ptr(beta), _ptr(A), _ptr(Bm),
                                 _ptr(K), _ptr(V), _ptr(self.S), _ptr(self.o), s.cuda_stream)
        if st != DPLR_OK:
            raise DplrError(st, "dplr_la_decode_step")
        return self.o


class Backward:
    """Prepared backward for one descriptor (dplr_la_backward): owns the workspace and the fp32 gradients."""

    def __init__(self, mode: str, in_dtype: torch.dtype, B: int, H: int, T: int, dk: int, dv: int,
                 r_ab: Optional[int] = None, r_kv: Optional[int] = None, chunk: int = 64,
                 device: Optional[torch.device] = None):
        self.mode = mode
        self.desc = make_desc(mode, in_dtype, B, H, T, dk, dv, r_ab, r_kv, chunk)
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        nbytes = dplr_la_backward_workspace_size(self.desc)
        if nbytes == 0:
            raise DplrError(dplr_la_check(self.desc) or 2, "dplr_la_backward_workspace_size")
        self.ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=self.device)
        off = (-self.ws.data_ptr()) % 256
        self.ws_ptr, self.ws_bytes = self.ws.data_ptr() + off, nbytes
        r, p = self.desc.r_ab, self.desc.r_kv
        f = lambda *shape: torch.zeros(shape, dtype=torch.float32, device=self.device)
        g = {"q": f(B, H, T, dk), "S0": f(B, H, dk, dv)}
        if mode == "generic":
            g.update(decay=f(B, H, T, dk), A=f(B, H, T, r, dk), Bm=f(B, H, T, r, dk))
            if p > 0:
                g.update(K=f(B, H, T, p, dk), V=f(B, H, T, p, dv))
        else:
            g.update(k=f(B, H, T, dk), v=f(B, H, T, dv), beta=f(B, H, T),
                     decay=f(B, H, T) if mode == "gdn" else f(B, H, T, dk))
        self.grads = g

    def __call__(self, dO, dST=None, q=None, k=None, v=None, decay=None, beta=None, A=None, Bm=None, K=None,
                 V=None, S0=None, stream: Optional[torch.cuda.Stream] = None) -> dict:
        """Gradients of the forward's inputs (dict of fp32 tensors, also kept in .grads)."""
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        g = self.grads
        st = dplr_la_backward(self.desc, _ptr(q), _ptr(k), _ptr(v), _ptr(decay), _ptr(beta), _ptr(A), _ptr(Bm),
                              _ptr(K), _ptr(V), _ptr(S0), _ptr(dO), _ptr(dST), _ptr(g["q"]), _ptr(g.get("k")),
                              _ptr(g.get("v")), _ptr(g["decay"]), _ptr(g.get("beta")), _ptr(g.get("A")),
                              _ptr(g.get("Bm")), _ptr(g.get("K")), _ptr(g.get("V")), _ptr(g["S0"]), self.ws_ptr,
                              self.ws_bytes, s.cuda_stream)
        if st != DPLR_OK:
            raise DplrError(st, "dplr_la_backward")
        return g


class HLA:
    """Prepared HLA forward (dplr_hla_forward) for one GDN descriptor and chunk length: owns workspace and output."""

    def __init__(self, in_dtype: torch.dtype, B: int, H: int, T: int, dk: int, dv: int, L: int = 256,
                 device: Optional[torch.device] = None):
        self.desc = make_desc("gdn", in_dtype, B, H, T, dk, dv)
        self.L = int(L)
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        nbytes = dplr_hla_workspace_size(self.desc, self.L)
        if nbytes == 0:
            raise DplrError(2, "dplr_hla_workspace_size")
        self.ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=self.device)
        off = (-self.ws.data_ptr()) % 256
        self.ws_ptr, self.ws_bytes = self.ws.data_ptr() + off, nbytes
        self.o = torch.empty((B, H, T, dv), dtype=torch.float32, device=self.device)
        self.path = dplr_hla_path(self.desc, self.L)

    def device_status(self, clear: bool = False) -> int:
        """The workspace's status word (0, or DPLR_ERR_TIMEOUT after a bounded wait gave up), read synchronously."""
        s = torch.cuda.current_stream(self.device)
        st, word = dplr_la_read_status(self.ws_ptr, self.ws_bytes, clear, s.cuda_stream)
        if st != DPLR_OK:
            raise DplrError(st, "dplr_la_read_status")
        return word

    def __call__(self, q, k, v, g, beta, W, theta: float = 0.0,
                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        st = dplr_hla_forward(self.desc, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(W), theta, self.L,
                              _ptr(self.o), self.ws_ptr, self.ws_bytes, s.cuda_stream)
        if st != DPLR_OK:
            raise DplrError(st, "dplr_hla_forward")
        return self.o


class GDP:
    """Prepared stacked-Householder forward (dplr_gdp_forward) with n_h steps per token: owns workspace and outputs."""

    def __init__(self, in_dtype: torch.dtype, B: int, H: int, T: int, dk: int, dv: int, nh: int,
                 device: Optional[torch.device] = None):
        self.desc = make_desc("generic", in_dtype, B, H, T, dk, dv, nh, nh)
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        nbytes = dplr_gdp_workspace_size(self.desc)
        if nbytes == 0:
            raise DplrError(2, "dplr_gdp_workspace_size")
        self.ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=self.device)
        off = (-self.ws.data_ptr()) % 256
        self.ws_ptr, self.ws_bytes = self.ws.data_ptr() + off, nbytes
        self.o = torch.empty((B, H, T, dv), dtype=torch.float32, device=self.device)
        self.S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=self.device)
        self.path = dplr_gdp_path(self.desc)

    def __call__(self, q, k, v, g, beta, S0=None, stream: Optional[torch.cuda.Stream] = None):
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        st = dplr_gdp_forward(self.desc, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S0), _ptr(self.o),
                              _ptr(self.S_T), self.ws_ptr, self.ws_bytes, s.cuda_stream)
        if st != DPLR_OK:
            raise DplrError(st, "dplr_gdp_forward")
        return self.o, self.S_T


# ----------------------------------------------------------------------------
# Linear attention with one decay per head (dplr_hd_*).
# ----------------------------------------------------------------------------

def make_hd_desc(in_dtype, B: int, H: int, T: int, dk: int, dv: int, q_heads: Optional[int] = None,
                 per_head: bool = False) -> dplr_hd_desc:
    if in_dtype in (torch.bfloat16, "bf16", DPLR_BF16):
        dt = DPLR_BF16
    elif in_dtype in (torch.float32, "f32", DPLR_F32):
        dt = DPLR_F32
    else:
        raise ValueError(f"unsupported input dtype {in_dtype}")
    sizes = _int32(B=B, H=H, q_heads=H if q_heads is None else q_heads, T=T, dk=dk, dv=dv)
    return dplr_hd_desc(dt, *sizes, int(bool(per_head)))


def _int32(**sizes):
    """The sizes as ints, refused beyond the C interface's 32 bits (ctypes would drop the bits above)."""
    for name, n in sizes.items():
        if not -2 ** 31 <= operator.index(n) < 2 ** 31:
            raise ValueError(f"{name} is {n}, which does not fit 32 bits")
    return [operator.index(n) for n in sizes.values()]


def dplr_hd_check(desc: dplr_hd_desc) -> int:
    return int(library().dplr_hd_check(ctypes.byref(desc)))


def dplr_hd_path(desc: dplr_hd_desc) -> str:
    return library().dplr_hd_path(ctypes.byref(desc)).decode()


def dplr_hd_workspace_size(desc: dplr_hd_desc) -> int:
    return int(library().dplr_hd_workspace_size(ctypes.byref(desc)))


def dplr_hd_backward_workspace_size(desc: dplr_hd_desc) -> int:
    return int(library().dplr_hd_backward_workspace_size(ctypes.byref(desc)))


def dplr_hd_packed_workspace_size(desc: dplr_hd_desc, R: int, block: int) -> int:
    return int(library().dplr_hd_packed_workspace_size(ctypes.byref(desc), int(R), int(block)))


def _ref(t: Optional[dplr_hd_tensor]):
    return None if t is None else ctypes.byref(t)


def dplr_hd_forward(desc, q, k, v, decay, S0, o, S_T, workspace, ws_bytes, stream) -> int:
    """q, k, v, decay, o: dplr_hd_tensor (or None); the states and the workspace: device pointers."""
    return int(library().dplr_hd_forward(ctypes.byref(desc), _ref(q), _ref(k), _ref(v), _ref(decay), S0, _ref(o), S_T,
                                         workspace, ctypes.c_size_t(ws_bytes), stream))


def dplr_hd_backward(desc, q, k, v, decay, S0, dO, dST, dq, dk, dv, ddecay, dS0, workspace, ws_bytes, stream) -> int:
    return int(library().dplr_hd_backward(ctypes.byref(desc), _ref(q), _ref(k), _ref(v), _ref(decay), S0, _ref(dO), dST,
                                          _ref(dq), _ref(dk), _ref(dv), ddecay, dS0, workspace,
                                          ctypes.c_size_t(ws_bytes), stream))


def dplr_hd_plan(R, capacity, block, n_slots, lengths, slots, context, starts, blocks, block_starts, token_slot,
                 token_pos, status, stream) -> int:
    return int(library().dplr_hd_plan(R, capacity, block, n_slots, lengths, slots, context, starts, blocks,
                                      block_starts, token_slot, token_pos, status, stream))


def dplr_hd_forward_packed(desc, R, block, n_slots, blocks, block_starts, slots, context, q, k, v, decay, S, o,
                           workspace, ws_bytes, stream) -> int:
    return int(library().dplr_hd_forward_packed(ctypes.byref(desc), R, block, n_slots, blocks, block_starts, slots,
                                                context, _ref(q), _ref(k), _ref(v), _ref(decay), S, _ref(o), workspace,
                                                ctypes.c_size_t(ws_bytes), stream))


def dplr_hd_decode_step(desc, n_slots, slots, q, k, v, decay, S, o, status, stream) -> int:
    return int(library().dplr_hd_decode_step(ctypes.byref(desc), n_slots, slots, _ref(q), _ref(k), _ref(v), _ref(decay),
                                             S, _ref(o), status, stream))


class _Slots:
    """The dplr_hd_tensor arguments of one prepared call, in one buffer that each call fills anew: a call's host time is
    its launches', and building a ctypes structure per tensor and call took longer than those. `turn` is held from filling
    it to the end of the C call, which reads it: another thread may call the same object."""

    def __init__(self, n: int):
        self.buf = ctypes.create_string_buffer(32 * n)
        at = ctypes.addressof(self.buf)
        self.refs = [ctypes.cast(at + 32 * i, ctypes.POINTER(dplr_hd_tensor)) for i in range(n)]
        self.fill = struct.Struct(f"={4 * n}q").pack_into
        self.turn = threading.Lock()

    def __call__(self, *values):
        self.fill(self.buf, 0, *values)


def _refuse(t, name, device, dtype, shape):
    """Says what is wrong with a tensor that _bad found wrong."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous along its last axis, start on a 16-byte boundary and have strides that "
                     "are positive multiples of 16 bytes")


class _HeadDecayBase:
    def _setup(self, in_dtype, B, H, T, dk, dv, q_heads, per_head, device):
        self.desc = make_hd_desc(in_dtype, B, H, T, dk, dv, q_heads, per_head)
        st = dplr_hd_check(self.desc)
        if st != DPLR_OK:
            raise DplrError(st, "dplr_hd_check")
        self.B, self.H, self.Hq, self.T, self.dk, self.dv = B, H, self.desc.Hq, T, dk, dv
        self.in_dtype = torch.bfloat16 if self.desc.in_dtype == DPLR_BF16 else torch.float32
        self.per_head = bool(per_head)
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.path = dplr_hd_path(self.desc)
        self._unit = 16 // self.in_dtype.itemsize       # strides are multiples of this
        self._desc_ref = ctypes.byref(self.desc)

    def _workspace(self, nbytes, name):
        if nbytes == 0:
            raise DplrError(DPLR_ERR_INVALID_ARG, name)
        self.ws_bytes = nbytes
        self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)   # status word zeroed once

    def _rows(self, heads, d, token_major, dtype=None):
        B, T = self.B, self.T
        dt = self.in_dtype if dtype is None else dtype
        if token_major:
            return torch.zeros((B, T, heads, d), dtype=dt, device=self.device).transpose(1, 2)
        return torch.zeros((B, heads, T, d), dtype=dt, device=self.device)

    def _at(self, t, name, shape):
        """Address and strides of a row tensor (features last), checked."""
        if t is None or t.dtype is not self.in_dtype or t.shape != shape or t.device != self.device:
            _refuse(t, name, self.device, self.in_dtype, shape)
        p = t.data_ptr()
        if p & 15 or not t.is_contiguous():
            st, u = t.stride(), self._unit
            if t.numel() and (st[-1] != 1 or p & 15):
                _refuse(t, name, self.device, self.in_dtype, shape)
            for n, s in zip(shape, st[:-1]):
                if n > 1 and (s <= 0 or s % u) and t.numel():
                    _refuse(t, name, self.device, self.in_dtype, shape)
            return p, st
        return p, t.stride()

    def _gates(self, t, shape):
        """Address and strides of the log-gates, checked (all strides 0 with per_head)."""
        want = (self.H,) if self.per_head else shape
        if t is None or t.dtype is not torch.float32 or t.shape != want or t.device != self.device:
            _refuse(t, "decay", self.device, torch.float32, want)
        st = t.stride()
        if self.per_head:
            if self.H > 1 and st[0] != 1:
                raise ValueError("decay must be contiguous")
            return t.data_ptr(), (0, 0, 0)
        if min(st) < 0:
            raise ValueError("decay needs non-negative strides")
        return t.data_ptr(), st

    def _state(self, t, name, shape):
        if t is None:
            return None
        if t.dtype is not torch.float32 or t.shape != shape or t.device != self.device or not t.is_contiguous():
            _need(t, name, self.device, torch.float32, shape)
        return t.data_ptr()

    def _call(self, fn, name, stream, *args):
        """The C call on this object's device and a stream, as its last argument."""
        i = self.device.index
        s = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(i)
        if torch._C._cuda_getDevice() == i:
            st = fn(self._desc_ref, *args, s)
        else:
            with torch.cuda.device(i):
                st = fn(self._desc_ref, *args, s)
        if st != DPLR_OK:
            raise DplrError(st, name)

    def device_status(self, clear: bool = False) -> int:
        """The workspace's device status word (0, DPLR_ERR_TIMEOUT after a bounded wait gave up, or DPLR_ERR_INVALID_ARG
        after a ragged forward found a slot out of range), read synchronously through dplr_la_read_status."""
        with torch.cuda.device(self.device):
            s = torch.cuda.current_stream(self.device)
            st, word = dplr_la_read_status(_ptr(self.workspace), self.workspace.numel(), clear, s.cuda_stream)
        if st != DPLR_OK:
            raise DplrError(st, "dplr_la_read_status")
        return word


class HeadDecay(_HeadDecayBase):
    """Prepared forward of linear attention with one decay per head (dplr_hd_forward): S_t = exp(g_t) S_{t-1} + k_t v_t^T,
    o_t = S_t^T q_t. Owns the outputs o [B,H,T,dv] (the inputs' type; stored with the tokens before the heads if
    `token_major`), S_T [B,H,dk,dv] fp32, and the workspace, so that repeated calls allocate nothing."""

    def __init__(self, in_dtype, B: int, H: int, T: int, dk: int, dv: int, q_heads: Optional[int] = None,
                 per_head: bool = False, token_major: bool = False, device: Optional[torch.device] = None):
        self._setup(in_dtype, B, H, T, dk, dv, q_heads, per_head, device)
        with torch.cuda.device(self.device):
            self._workspace(dplr_hd_workspace_size(self.desc), "dplr_hd_workspace_size")
            self.o = self._rows(H, dv, token_major)
            self.S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=self.device)
        self._fn, self._slots = library().dplr_hd_forward, _Slots(5)

    def __call__(self, q, k, v, decay, S0=None,
                 stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """q, k [B,Hq,T,dk], v [B,H,T,dv], strided as they are; decay [B,H,T] fp32, or [H] with per_head."""
        B, H, T = self.B, self.H, self.T
        qk = (B, self.Hq, T, self.dk)
        (pq, sq), (pk, sk) = self._at(q, "q", qk), self._at(k, "k", qk)
        pv, sv = self._at(v, "v", (B, H, T, self.dv))
        pg, sg = self._gates(decay, (B, H, T))
        o, so = self.o, self.o.stride()
        f = self._slots
        with f.turn:
            f(pq, sq[0], sq[1], sq[2], pk, sk[0], sk[1], sk[2], pv, sv[0], sv[1], sv[2], pg, sg[0], sg[1], sg[2],
              o.data_ptr(), so[0], so[1], so[2])
            r = f.refs
            self._call(self._fn, "dplr_hd_forward", stream, r[0], r[1], r[2], r[3],
                       self._state(S0, "S0", (B, H, self.dk, self.dv)), r[4], self.S_T.data_ptr(),
                       self.workspace.data_ptr(), self.ws_bytes)
        return o, self.S_T


class HeadDecayBackward(_HeadDecayBase):
    """Prepared backward of HeadDecay (dplr_hd_backward): owns the workspace and the gradients, q, k, v in the inputs'
    type (token-major if asked for), decay ([B,H,T], or [H] with per_head) and S0 in fp32."""

    def __init__(self, in_dtype, B: int, H: int, T: int, dk: int, dv: int, q_heads: Optional[int] = None,
                 per_head: bool = False, token_major: bool = False, device: Optional[torch.device] = None):
        self._setup(in_dtype, B, H, T, dk, dv, q_heads, per_head, device)
        with torch.cuda.device(self.device):
            self._workspace(dplr_hd_backward_workspace_size(self.desc), "dplr_hd_backward_workspace_size")
            f = lambda *shape: torch.zeros(shape, dtype=torch.float32, device=self.device)  # noqa: E731
            self.grads = {"q": self._rows(self.Hq, dk, token_major), "k": self._rows(self.Hq, dk, token_major),
                          "v": self._rows(H, dv, token_major), "decay": f(H) if per_head else f(B, H, T),
                          "S0": f(B, H, dk, dv)}
        self._fn, self._slots = library().dplr_hd_backward, _Slots(8)

    def __call__(self, dO, dST, q, k, v, decay, S0=None, decay_grad: bool = True,
                 stream: Optional[torch.cuda.Stream] = None) -> dict:
        """Gradients of HeadDecay's inputs (a dict, also kept in .grads) given dO [B,H,T,dv] in the inputs' type and
        dST (fp32 or None: zero). Without `decay_grad` the gradient of the gates is not computed (and not returned), and on
        the tensor cores those of q and k come from operands rounded to bf16 once instead of split in two parts: in less
        time and with other bits, 2.4e-3 instead of 1.7e-3 of their 2-norm."""
        B, H, T = self.B, self.H, self.T
        qk, vo, state = (B, self.Hq, T, self.dk), (B, H, T, self.dv), (B, H, self.dk, self.dv)
        at = [self._at(q, "q", qk), self._at(k, "k", qk), self._at(v, "v", vo), self._gates(decay, (B, H, T)),
              self._at(dO, "dO", vo)]
        G = self.grads
        at += [(G[n].data_ptr(), G[n].stride()) for n in ("q", "k", "v")]
        f = self._slots
        with f.turn:
            f(*[x for p, st in at for x in (p, st[0], st[1], st[2])])
            r = f.refs
            self._call(self._fn, "dplr_hd_backward", stream, r[0], r[1], r[2], r[3], self._state(S0, "S0", state), r[4],
                       self._state(dST, "dST", state), r[5], r[6], r[7], G["decay"].data_ptr() if decay_grad else None,
                       G["S0"].data_ptr(), self.workspace.data_ptr(), self.ws_bytes)
        return G if decay_grad else {n: t for n, t in G.items() if n != "decay"}


class RequestPlan:
    """Tables of a ragged batch of `requests` requests with up to `capacity` tokens, built on the GPU from their lengths
    (dplr_hd_plan). Owns the tables: starts [R+1], blocks [capacity // block + R, 4], block_starts [R+1], token_slot and
    token_pos [capacity], all int32."""

    def __init__(self, requests: int, capacity: int, slots: int, block: int = 128,
                 device: Optional[torch.device] = None):
        self.R, self.capacity, self.n_slots, self.block = _int32(requests=int(requests), capacity=int(capacity),
                                                                 slots=int(slots), block=int(block))
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        if self.R < 1 or self.capacity < 0 or self.block < 32 or self.block % 32 or self.n_slots < 1:
            raise ValueError("RequestPlan needs requests >= 1, capacity >= 0, slots >= 1 and a block that is a multiple of 32")
        f = lambda *shape: torch.full(shape, -1, dtype=torch.int32, device=self.device)  # noqa: E731
        self.starts, self.block_starts = f(self.R + 1), f(self.R + 1)
        self.blocks = f(self.capacity // self.block + self.R, 4)
        self.token_slot, self.token_pos = f(self.capacity), f(self.capacity)
        self.status = f(1)
        self.tables = {"starts": self.starts, "blocks": self.blocks, "block_starts": self.block_starts,
                       "token_slot": self.token_slot, "token_pos": self.token_pos}
        self._fn = library().dplr_hd_plan

    def __call__(self, lengths, slots, context, stream: Optional[torch.cuda.Stream] = None) -> dict:
        """lengths, slots, context: int32 [R] on the device. Returns the tables (see device_status for refused input). A packed
        forward of this plan reads `slots` and `context` again: leave them as they are until it has run."""
        dev, i = self.device, self.device.index
        for t, name in ((lengths, "lengths"), (slots, "slots"), (context, "context")):
            if t is None or t.dtype is not torch.int32 or t.shape != (self.R,) or t.device != dev or not t.is_contiguous():
                _need(t, name, dev, torch.int32, (self.R,))
        s = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(i)
        args = (self.R, self.capacity, self.block, self.n_slots, lengths.data_ptr(), slots.data_ptr(), context.data_ptr(),
                self.starts.data_ptr(), self.blocks.data_ptr(), self.block_starts.data_ptr(), self.token_slot.data_ptr(),
                self.token_pos.data_ptr(), self.status.data_ptr(), s)
        if torch._C._cuda_getDevice() == i:
            st = self._fn(*args)
        else:
            with torch.cuda.device(i):
                st = self._fn(*args)
        if st != DPLR_OK:
            raise DplrError(st, "dplr_hd_plan")
        self.slots, self.context = slots, context     # the packed forward reads them
        return self.tables

    def device_status(self) -> int:
        """The last call's status word (DPLR_OK or DPLR_ERR_INVALID_ARG), read synchronously."""
        return int(self.status.item())


class HeadDecayPacked(_HeadDecayBase):
    """Prepared forward of a ragged batch (dplr_hd_forward_packed) on a pool of states: `plan` (a RequestPlan; one is made
    if none is given) says which rows belong to which request. Owns the output o [capacity,H,dv] (rows behind the last
    token stay as they were) and the workspace."""

    def __init__(self, in_dtype, requests: int, capacity: int, slots: int, H: int, dk: int, dv: int,
                 q_heads: Optional[int] = None, per_head: bool = False, plan: Optional[RequestPlan] = None,
                 device: Optional[torch.device] = None):
        self._setup(in_dtype, 1, H, capacity, dk, dv, q_heads, per_head, device)
        if plan is None:
            plan = RequestPlan(requests, capacity, slots, default_block(self.desc), self.device)
        elif (plan.R, plan.capacity, plan.n_slots, plan.device) != (requests, capacity, slots, self.device):
            raise ValueError("the plan is for another number of requests, capacity, slots or device")
        self.plan, self.n_slots = plan, int(slots)
        with torch.cuda.device(self.device):
            self._workspace(dplr_hd_packed_workspace_size(self.desc, plan.R, plan.block), "dplr_hd_packed_workspace_size")
            self.o = torch.zeros((capacity, H, dv), dtype=self.in_dtype, device=self.device)
        self._fn, self._slots = library().dplr_hd_forward_packed, _Slots(5)

    def __call__(self, q, k, v, decay, S, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """q, k [capacity,Hq,dk], v [capacity,H,dv], decay [capacity,H] fp32 or [H]; S [slots,H,dk,dv] fp32 is updated."""
        p, n, H = self.plan, self.T, self.H
        if not hasattr(p, "slots"):
            raise ValueError("call the plan first: it makes the tables")
        qk, o = (n, self.Hq, self.dk), self.o
        at = [self._at(q, "q", qk), self._at(k, "k", qk), self._at(v, "v", (n, H, self.dv)),
              self._gates(decay, (n, H)), (o.data_ptr(), o.stride())]
        if S is None:
            raise ValueError("S is required")
        f = self._slots
        with f.turn:
            f(*[x for ptr, st in at for x in (ptr, 0, st[1], st[0])])
            r = f.refs
            self._call(self._fn, "dplr_hd_forward_packed", stream, p.R, p.block, self.n_slots, p.blocks.data_ptr(),
                       p.block_starts.data_ptr(), p.slots.data_ptr(), p.context.data_ptr(), r[0], r[1], r[2], r[3],
                       self._state(S, "S", (self.n_slots, H, self.dk, self.dv)), r[4], self.workspace.data_ptr(),
                       self.ws_bytes)
        return o


def default_block(desc: dplr_hd_desc) -> int:
    """Tokens per block of a ragged batch. Every block but a request's last costs a pass more over its keys and values, and
    the longest block decides when the call ends: so blocks are about as long as the tokens and heads that an SM gets, up
    to the next power of two on the tensor cores (bf16 H16 128 x 128, 16 requests of up to 1900 tokens: 2048 83 us, 512
    132 us; one of 3000: 512 39 us, 2048 86 us), down to it on the CUDA cores, whose extra pass is the smaller part (fp32,
    one of 3000: 256 250 us, 512 318 us).

    The tokens are those of a full batch (`desc.T`, the capacity): a step's own are not known when the workspace is made.
    Where steps stay far below the capacity, a plan with a shorter block is the better choice (H16 128 x 128, tables and
    forward: one request of 3000 tokens in a capacity of 16384 97 us, with blocks of 512 49 us; one of 8000 in a capacity
    of 55165 189 and 78 us)."""
    per_sm = desc.T * desc.H // 152
    if dplr_hd_path(desc) == "hd_tcgen05":
        return max(512, 1 << max(per_sm - 1, 0).bit_length())
    return max(128, 1 << max(per_sm.bit_length() - 1, 0))


class HeadDecayDecode(_HeadDecayBase):
    """Prepared one-token step for `rows` rows on a pool of states (dplr_hd_decode_step): owns the output o [rows,H,dv]."""

    def __init__(self, in_dtype, rows: int, H: int, dk: int, dv: int, slots: int, q_heads: Optional[int] = None,
                 per_head: bool = False, device: Optional[torch.device] = None):
        self._setup(in_dtype, rows, H, 1, dk, dv, q_heads, per_head, device)
        self.n_slots, = _int32(slots=int(slots))
        self.o = torch.zeros((rows, H, dv), dtype=self.in_dtype, device=self.device)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._fn, self._slots = library().dplr_hd_decode_step, _Slots(5)

    def device_status(self, clear: bool = False) -> int:
        """DPLR_ERR_INVALID_ARG if a row's slot was out of range or an earlier row's since the word was cleared."""
        word = int(self.status.item())
        if clear:
            self.status.zero_()
        return word

    def __call__(self, q, k, v, decay, S, slots, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """q, k [rows,Hq,dk], v [rows,H,dv], decay [rows,H] fp32 or [H]; S [slots,H,dk,dv] fp32 is updated in place;
        slots [rows] int32: each row's state, -1 for a row without one."""
        n, H = self.B, self.H
        qk, o = (n, self.Hq, self.dk), self.o
        (pq, sq), (pk, sk) = self._at(q, "q", qk), self._at(k, "k", qk)
        pv, sv = self._at(v, "v", (n, H, self.dv))
        pg, sg = self._gates(decay, (n, H))
        if S is None:
            raise ValueError("S is required")
        if slots is None or slots.dtype is not torch.int32 or slots.shape != (n,) or slots.device != self.device or \
                not slots.is_contiguous():
            _need(slots, "slots", self.device, torch.int32, (n,))
        f = self._slots
        with f.turn:
            f(pq, sq[0], sq[1], 0, pk, sk[0], sk[1], 0, pv, sv[0], sv[1], 0, pg, sg[0], sg[1], 0, o.data_ptr(), H * self.dv,
              self.dv, 0)
            r = f.refs
            self._call(self._fn, "dplr_hd_decode_step", stream, self.n_slots, slots.data_ptr(), r[0], r[1], r[2], r[3],
                       self._state(S, "S", (self.n_slots, H, self.dk, self.dv)), r[4], self.status.data_ptr())
        return o
