"""Thin ctypes binding of ``libsscan.so`` (the C ABI in include/sscan.h).

Argument marshalling only: every step of the scan runs in the library's HIP
kernels.  PyTorch supplies device memory (inputs, outputs, the workspace) and the
current stream.  If the library is missing this module raises; there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsscan.so")

SSCAN_F32 = 0
SSCAN_BF16 = 1
DSTATE = 16
PROFILE_EVENTS = 5  # step boundaries: start, staged B/C, aggregates, carry, output
PROFILE_STEPS = ("stage_bc", "aggregate", "carry", "output")
BWD_PROFILE_EVENTS = 6  # start, staged B/C, window states, window adjoints, window pass, sums
BWD_PROFILE_STEPS = ("stage_bc", "window_states", "window_adjoints", "window_pass", "param_sums")

_DT_CODE = {torch.float32: SSCAN_F32, torch.bfloat16: SSCAN_BF16}


class SScanError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: status {status} ({strerror(status)})")
        self.status = status


class DirParams(ctypes.Structure):
    _fields_ = [("delta", ctypes.c_void_p), ("delta_bias", ctypes.c_void_p), ("A", ctypes.c_void_p),
                ("B", ctypes.c_void_p), ("C", ctypes.c_void_p), ("D", ctypes.c_void_p)]


class ConvParams(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("width", ctypes.c_int),
                ("same", ctypes.c_int), ("silu", ctypes.c_int)]


class DirGrads(ctypes.Structure):
    _fields_ = [("ddelta", ctypes.c_void_p), ("ddelta_bias", ctypes.c_void_p), ("dA", ctypes.c_void_p),
                ("dB", ctypes.c_void_p), ("dC", ctypes.c_void_p), ("dD", ctypes.c_void_p)]


class DeltaParams(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("g", ctypes.c_void_p),
                ("beta", ctypes.c_void_p), ("lengths", ctypes.c_void_p), ("h0", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64 * 3), ("k_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3),
                ("g_stride", ctypes.c_int64 * 3), ("beta_stride", ctypes.c_int64 * 3), ("batch", ctypes.c_int64),
                ("len", ctypes.c_int64), ("qk_heads", ctypes.c_int64), ("v_heads", ctypes.c_int64),
                ("dk", ctypes.c_int64), ("dv", ctypes.c_int64), ("scale", ctypes.c_float), ("qk_norm", ctypes.c_int),
                ("io_dtype", ctypes.c_int)]


class DeltaGrads(ctypes.Structure):
    _fields_ = [("dq", ctypes.c_void_p), ("dk", ctypes.c_void_p), ("dv", ctypes.c_void_p), ("dg", ctypes.c_void_p),
                ("dbeta", ctypes.c_void_p), ("dh0", ctypes.c_void_p)]


class GatedNormParams(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("z", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("x_stride", ctypes.c_int64 * 2), ("z_stride", ctypes.c_int64 * 2), ("rows", ctypes.c_int64),
                ("heads", ctypes.c_int64), ("size", ctypes.c_int64), ("eps", ctypes.c_float),
                ("gate_first", ctypes.c_int), ("per_head", ctypes.c_int), ("io_dtype", ctypes.c_int)]


class AddNormParams(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("scale", ctypes.c_void_p), ("post_weight", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("size", ctypes.c_int64), ("eps", ctypes.c_float), ("io_dtype", ctypes.c_int),
                ("residual_dtype", ctypes.c_int)]


# The parameter structs packed in one go: small calls are bound by the host, and a
# ctypes.Structure of thirty fields takes several microseconds to fill.
_DELTA = struct.Struct("7P21qfii4x")
_GATED = struct.Struct("3P7qfiii")
_ADD = struct.Struct("5P2qfii4x")


_lib = None


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Loads (once) and returns the shared library; raises if it is not built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with `python -m selective_state_space_sscan_amd.build`")
    lib = ctypes.CDLL(p)
    V, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    DP = ctypes.POINTER(DirParams)
    lib.sscan_fwd.argtypes = [V, V, V, I, V, V, V, V, V, V, I64, I64, I64, I64, I, V, I, I, V, SZ]
    lib.sscan_fwd.restype = I
    lib.sscan_bidir.argtypes = [V, V, V, DP, DP, I, I64, I64, I64, I64, V, I, I, V, SZ]
    lib.sscan_bidir.restype = I
    lib.sscan_fwd_noalloc.argtypes = lib.sscan_fwd.argtypes[:-2]
    lib.sscan_fwd_noalloc.restype = I
    lib.sscan_fwd_profiled.argtypes = lib.sscan_fwd.argtypes + [V]
    lib.sscan_fwd_profiled.restype = I
    lib.sscan_bidir_profiled.argtypes = lib.sscan_bidir.argtypes + [V]
    lib.sscan_bidir_profiled.restype = I
    lib.sscan_validate_fwd.argtypes = [V, V, V, I, V, V, V, V, V, V, I64, I64, I64, I64, I, I, I, V, SZ]
    lib.sscan_validate_fwd.restype = I
    lib.sscan_validate_bidir.argtypes = [V, V, V, DP, DP, I, I64, I64, I64, I64, I, I, V, SZ]
    lib.sscan_validate_bidir.restype = I
    lib.sscan_fwd_state.argtypes = [V, V, V, I, V, V, V, V, V, V, V, V, I64, I64, I64, I64, I, V, I, I, V, SZ]
    lib.sscan_fwd_state.restype = I
    lib.sscan_validate_fwd_state.argtypes = [V, V, V, I, V, V, V, V, V, V, V, V, I64, I64, I64, I64, I, I, I, V, SZ]
    lib.sscan_validate_fwd_state.restype = I
    lib.sscan_step.argtypes = [V, V, V, V, I, V, V, V, V, V, V, I64, I64, I64, V, I, I]
    lib.sscan_step.restype = I
    lib.sscan_validate_step.argtypes = [V, V, V, V, I, V, V, V, V, V, V, I64, I64, I64, I, I]
    lib.sscan_validate_step.restype = I
    CPP = ctypes.POINTER(ConvParams)
    DGP = ctypes.POINTER(DirGrads)
    lib.sscan_bwd_conv.argtypes = [V, CPP, V, V, I, V, V, V, V, V, V, V, V, DGP, V, V, I64, I64, I64, I64, I, V, I, I,
                                   V, SZ]
    lib.sscan_bwd_conv.restype = I
    lib.sscan_bidir_bwd_conv.argtypes = [V, CPP, V, V, V, V, DP, DP, DGP, DGP, V, V, I, I64, I64, I64, I64, V, I, I, V,
                                         SZ]
    lib.sscan_bidir_bwd_conv.restype = I
    lib.sscan_validate_bwd_conv.argtypes = [V, CPP, V, V, I, V, V, V, V, V, V, V, V, DGP, V, V, I64, I64, I64, I64, I,
                                            I, I, V, SZ]
    lib.sscan_validate_bwd_conv.restype = I
    lib.sscan_bwd_conv_workspace_bytes.argtypes = [I64, I64, I64, I64, I, I]
    lib.sscan_bwd_conv_workspace_bytes.restype = SZ
    lib.sscan_step_conv.argtypes = [V, V, V, CPP, V, V, I, V, V, V, V, V, V, I64, I64, I64, V, I, I]
    lib.sscan_step_conv.restype = I
    lib.sscan_validate_step_conv.argtypes = [V, V, V, CPP, V, V, I, V, V, V, V, V, V, I64, I64, I64, I, I]
    lib.sscan_validate_step_conv.restype = I
    DG = ctypes.POINTER(DirGrads)
    lib.sscan_bwd.argtypes = [V, V, V, I, V, V, V, V, V, V, V, V, DG, I64, I64, I64, I64, I, V, I, I, V, SZ]
    lib.sscan_bwd.restype = I
    lib.sscan_bidir_bwd.argtypes = [V, V, V, V, V, DP, DP, DG, DG, I, I64, I64, I64, I64, V, I, I, V, SZ]
    lib.sscan_bidir_bwd.restype = I
    lib.sscan_validate_bwd.argtypes = [V, V, V, I, V, V, V, V, V, V, V, V, DG, I64, I64, I64, I64, I, I, I, V, SZ]
    lib.sscan_validate_bwd.restype = I
    lib.sscan_validate_bidir_bwd.argtypes = [V, V, V, V, V, DP, DP, DG, DG, I, I64, I64, I64, I64, I, I, V, SZ]
    lib.sscan_validate_bidir_bwd.restype = I
    lib.sscan_bwd_state.argtypes = [V, V, V, I, V, V, V, V, V, V, V, V, V, V, DG, V, I64, I64, I64, I64, I, V, I, I,
                                    V, SZ]
    lib.sscan_bwd_state.restype = I
    lib.sscan_validate_bwd_state.argtypes = [V, V, V, I, V, V, V, V, V, V, V, V, V, V, DG, V, I64, I64, I64, I64, I,
                                             I, I, V, SZ]
    lib.sscan_validate_bwd_state.restype = I
    lib.sscan_bwd_profiled.argtypes = lib.sscan_bwd.argtypes + [V]
    lib.sscan_bwd_profiled.restype = I
    lib.sscan_bidir_bwd_profiled.argtypes = lib.sscan_bidir_bwd.argtypes + [V]
    lib.sscan_bidir_bwd_profiled.restype = I
    lib.sscan_bwd_workspace_bytes.argtypes = [I64, I64, I64, I64, I]
    lib.sscan_bwd_workspace_bytes.restype = SZ
    CP = ctypes.POINTER(ConvParams)
    lib.sscan_conv1d.argtypes = [V, CP, V, I64, I64, I64, V, I]
    lib.sscan_conv1d.restype = I
    lib.sscan_validate_conv1d.argtypes = [V, CP, V, I64, I64, I64, I]
    lib.sscan_validate_conv1d.restype = I
    lib.sscan_fwd_conv.argtypes = [V, CP, V, V, I, V, V, V, V, V, V, I64, I64, I64, I64, I, V, I, I, V, SZ]
    lib.sscan_fwd_conv.restype = I
    lib.sscan_bidir_conv.argtypes = [V, CP, V, V, DP, DP, I, I64, I64, I64, I64, V, I, I, V, SZ]
    lib.sscan_bidir_conv.restype = I
    lib.sscan_fwd_conv_profiled.argtypes = lib.sscan_fwd_conv.argtypes + [V]
    lib.sscan_fwd_conv_profiled.restype = I
    lib.sscan_bidir_conv_profiled.argtypes = lib.sscan_bidir_conv.argtypes + [V]
    lib.sscan_bidir_conv_profiled.restype = I
    IP = ctypes.POINTER(ctypes.c_int)
    lib.sscan_multi.argtypes = [V, V, V, DP, IP, I, V, I, I64, I64, I64, I64, I64, V, I, I, V, SZ]
    lib.sscan_multi.restype = I
    lib.sscan_validate_multi.argtypes = [V, V, V, DP, IP, I, V, I, I64, I64, I64, I64, I64, I, I, V, SZ]
    lib.sscan_validate_multi.restype = I
    lib.sscan_multi_workspace_bytes.argtypes = [I64, I64, I64, I64, I64, IP, I, I, I]
    lib.sscan_multi_workspace_bytes.restype = SZ
    lib.sscan_multi_bwd.argtypes = [V, V, V, V, V, DP, DG, IP, I, V, I, I64, I64, I64, I64, I64, V, I, I, V, SZ]
    lib.sscan_multi_bwd.restype = I
    lib.sscan_validate_multi_bwd.argtypes = [V, V, V, V, V, DP, DG, IP, I, V, I, I64, I64, I64, I64, I64, I, I, V,
                                             SZ]
    lib.sscan_validate_multi_bwd.restype = I
    lib.sscan_multi_bwd_workspace_bytes.argtypes = [I64, I64, I64, I64, I64, IP, I, I, I]
    lib.sscan_multi_bwd_workspace_bytes.restype = SZ
    lib.sscan_spiral_order.argtypes = [I64, I64, V]
    lib.sscan_spiral_order.restype = I
    lib.sscan_workspace_bytes.argtypes = [I64, I64, I64, I64, I]
    lib.sscan_workspace_bytes.restype = SZ
    lib.sscan_scan_plan.argtypes = [I64, I64, I64, I64, I, ctypes.POINTER(ctypes.c_int64)]
    lib.sscan_scan_plan.restype = I
    lib.sscan_bwd_plan.argtypes = [I64, I64, I64, I64, I, ctypes.POINTER(ctypes.c_int64)]
    lib.sscan_bwd_plan.restype = I
    PP = NP = AP = V  # packed bytes, or a reference to the struct
    GP = ctypes.POINTER(DeltaGrads)
    lib.sscan_delta_fwd.argtypes = [PP, V, V, V, V, SZ]
    lib.sscan_delta_step.argtypes = [PP, V, V, V]
    lib.sscan_delta_bwd.argtypes = [PP, V, V, GP, V, V, SZ]
    lib.sscan_validate_delta_fwd.argtypes = [PP, V, V, V, SZ]
    lib.sscan_validate_delta_step.argtypes = [PP, V, V]
    lib.sscan_validate_delta_bwd.argtypes = [PP, V, V, GP, V, SZ]
    lib.sscan_gated_norm.argtypes = [NP, V, V]
    lib.sscan_gated_norm_bwd.argtypes = [NP, V, V, V, V, V, V, SZ]
    lib.sscan_validate_gated_norm.argtypes = [NP, V]
    lib.sscan_validate_gated_norm_bwd.argtypes = [NP, V, V, V, V, V, SZ]
    lib.sscan_add_norm.argtypes = [AP, V, V, V]
    lib.sscan_add_norm_bwd.argtypes = [AP, V, V, V, V, V, V, V, V, V, SZ]
    lib.sscan_validate_add_norm.argtypes = [AP, V, V]
    lib.sscan_validate_add_norm_bwd.argtypes = [AP, V, V, V, V, V, V, V, V, SZ]
    for name in ("delta_fwd", "delta_step", "delta_bwd", "gated_norm", "gated_norm_bwd", "add_norm", "add_norm_bwd"):
        getattr(lib, "sscan_" + name).restype = I
        getattr(lib, "sscan_validate_" + name).restype = I
    for name in ("sscan_delta_workspace_bytes", "sscan_delta_bwd_workspace_bytes"):
        getattr(lib, name).argtypes = [I64] * 6 + [I]
        getattr(lib, name).restype = SZ
    lib.sscan_delta_plan.argtypes = [I64] * 6 + [I, ctypes.POINTER(ctypes.c_int64)]
    lib.sscan_delta_plan.restype = I
    lib.sscan_gated_norm_bwd_workspace_bytes.argtypes = [I64, I64, I64]
    lib.sscan_gated_norm_bwd_workspace_bytes.restype = SZ
    lib.sscan_add_norm_bwd_workspace_bytes.argtypes = [I64, I64]
    lib.sscan_add_norm_bwd_workspace_bytes.restype = SZ
    lib.sscan_strerror.argtypes = [I]
    lib.sscan_strerror.restype = ctypes.c_char_p
    lib.sscan_version.argtypes = []
    lib.sscan_version.restype = I
    if path is None:
        _lib = lib
    return lib


class HipEvents:
    """Timing events of the HIP runtime the library runs on, for the profiled entry
    points (one set per call in flight): one event per boundary of ``steps``
    (PROFILE_STEPS for the forward calls, BWD_PROFILE_STEPS for the backward)."""

    _hip = None

    def __init__(self, steps=PROFILE_STEPS):
        self.steps = tuple(steps)
        nev = len(self.steps) + 1
        if HipEvents._hip is None:
            hip = ctypes.CDLL("libamdhip64.so.7")  # the runtime already mapped by torch and libsscan
            hip.hipEventCreate.argtypes = [ctypes.POINTER(ctypes.c_void_p)]
            hip.hipEventElapsedTime.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.c_void_p, ctypes.c_void_p]
            hip.hipEventSynchronize.argtypes = [ctypes.c_void_p]
            hip.hipEventDestroy.argtypes = [ctypes.c_void_p]
            HipEvents._hip = hip
        self._ev = (ctypes.c_void_p * nev)()
        for i in range(nev):
            h = ctypes.c_void_p()
            if HipEvents._hip.hipEventCreate(ctypes.byref(h)) != 0:
                raise RuntimeError("hipEventCreate failed")
            self._ev[i] = h

    @property
    def handles(self):
        return self._ev

    def step_ms(self):
        """Milliseconds of each step (dict keyed by PROFILE_STEPS); waits for the last event."""
        hip = HipEvents._hip
        hip.hipEventSynchronize(self._ev[len(self.steps)])
        out = {}
        for i, name in enumerate(self.steps):
            ms = ctypes.c_float()
            if hip.hipEventElapsedTime(ctypes.byref(ms), self._ev[i], self._ev[i + 1]) != 0:
                raise RuntimeError("hipEventElapsedTime failed")
            out[name] = float(ms.value)
        return out

    def total_ms(self) -> float:
        """Milliseconds from the first to the last event (the whole call)."""
        hip = HipEvents._hip
        hip.hipEventSynchronize(self._ev[len(self.steps)])
        ms = ctypes.c_float()
        if hip.hipEventElapsedTime(ctypes.byref(ms), self._ev[0], self._ev[len(self.steps)]) != 0:
            raise RuntimeError("hipEventElapsedTime failed")
        return float(ms.value)

    def __del__(self):
        # through the instance's class: at interpreter exit the module's globals may
        # already be gone when the last events are collected
        hip = getattr(type(self), "_hip", None)
        if hip is not None:
            for h in self._ev:
                if h:
                    hip.hipEventDestroy(h)


def strerror(status: int) -> str:
    return load_library().sscan_strerror(int(status)).decode()


def workspace_bytes(batch: int, dim: int, length: int, dstate: int = DSTATE, bidir: bool = False) -> int:
    return int(load_library().sscan_workspace_bytes(batch, dim, length, dstate, int(bool(bidir))))


def scan_plan(batch: int, dim: int, length: int, dstate: int = DSTATE, bidir: bool = False) -> dict:
    """How a scan of these sizes is split (sscan_scan_plan): segment length, segments
    per row, segments per aggregate run, runs per row."""
    out = (ctypes.c_int64 * 4)()
    st = load_library().sscan_scan_plan(batch, dim, length, dstate, int(bool(bidir)), out)
    if st != 0:
        raise SScanError(st, "sscan_scan_plan")
    return dict(seg_len=out[0], nseg=out[1], run_len=out[2], nrun=out[3])


def bwd_plan(batch: int, dim: int, length: int, dstate: int = DSTATE, bidir: bool = False) -> dict:
    """How a backward call of these sizes is split (sscan_bwd_plan): windows per
    row, blocks per window, channel groups per block, windows per chain run, runs
    per row."""
    out = (ctypes.c_int64 * 5)()
    st = load_library().sscan_bwd_plan(batch, dim, length, dstate, int(bool(bidir)), out)
    if st != 0:
        raise SScanError(st, "sscan_bwd_plan")
    return dict(nwin=out[0], csplit=out[1], gps=out[2], run_len=out[3], nrun=out[4])


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(t: Optional[torch.Tensor], name: str, device, dtype=None, shape=None):
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _workspace(nbytes: int, device, workspace: Optional[torch.Tensor]):
    if nbytes == 0:
        return None, 0
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    _check(workspace, "workspace", device)
    return workspace, workspace.numel() * workspace.element_size()


def _stream(device) -> ctypes.c_void_p:
    if device.index is None:
        return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)
    # the handle alone, without a Stream object: 2 us less a call
    return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(device.index))


def fwd(u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus: bool = True, reverse: bool = False,
        out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
        events: Optional[HipEvents] = None) -> torch.Tensor:
    """One-direction scan (``sscan_fwd``).  u, delta, z: [batch, dim, len] f32/bf16;
    B, C: [batch, 16, len] f32/bf16; A: [dim, 16] f32; D, delta_bias: [dim] f32.
    Returns the gated output, same dtype as u, enqueued on the current stream.
    With ``events`` the profiled entry point also records the step boundaries."""
    lib = load_library()
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("sscan.fwd needs CUDA (HIP) tensors")
    if u.dtype not in _DT_CODE or B.dtype not in _DT_CODE:
        raise TypeError("u/delta/z and B/C must be float32 or bfloat16")
    b, d, L = u.shape
    _check(u, "u", dev)
    _check(delta, "delta", dev, u.dtype, u.shape)
    _check(z, "z", dev, u.dtype, u.shape)
    _check(A, "A", dev, torch.float32, (d, DSTATE))
    _check(B, "B", dev, None, (b, DSTATE, L))
    _check(C, "C", dev, B.dtype, (b, DSTATE, L))
    _check(D, "D", dev, torch.float32, (d,))
    _check(delta_bias, "delta_bias", dev, torch.float32, (d,))
    if out is None:
        out = torch.empty_like(u)
    _check(out, "out", dev, u.dtype, u.shape)
    if u.numel() == 0:
        return out
    ws, ws_bytes = _workspace(workspace_bytes(b, d, L, DSTATE, False), dev, workspace)
    args = [_ptr(u), _ptr(delta), _ptr(delta_bias), int(bool(softplus)), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
            _ptr(out), b, d, L, DSTATE, int(bool(reverse)), _stream(dev), _DT_CODE[u.dtype], _DT_CODE[B.dtype],
            _ptr(ws), ws_bytes]
    if events is None:
        st = lib.sscan_fwd(*args)
    else:
        if events.steps != PROFILE_STEPS:
            raise ValueError("sscan.fwd needs HipEvents(PROFILE_STEPS)")
        st = lib.sscan_fwd_profiled(*args, ctypes.cast(events.handles, ctypes.c_void_p))
    if st != 0:
        raise SScanError(st, "sscan_fwd")
    return out


NOALLOC_SCRATCH_BYTES = 64 << 20  # SSCAN_NOALLOC_SCRATCH_BYTES


def fwd_noalloc(u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus: bool = True, reverse: bool = False,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``sscan_fwd_noalloc``: ``fwd`` with the library's fixed scratch array of the
    current device as its workspace (for callers that cannot allocate).  Allocates
    only ``out`` when it is not given."""
    lib = load_library()
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("sscan.fwd_noalloc needs CUDA (HIP) tensors")
    if u.dtype not in _DT_CODE or B.dtype not in _DT_CODE:
        raise TypeError("u/delta/z and B/C must be float32 or bfloat16")
    b, d, L = u.shape
    _check(u, "u", dev)
    _check(delta, "delta", dev, u.dtype, u.shape)
    _check(z, "z", dev, u.dtype, u.shape)
    _check(A, "A", dev, torch.float32, (d, DSTATE))
    _check(B, "B", dev, None, (b, DSTATE, L))
    _check(C, "C", dev, B.dtype, (b, DSTATE, L))
    _check(D, "D", dev, torch.float32, (d,))
    _check(delta_bias, "delta_bias", dev, torch.float32, (d,))
    if out is None:
        out = torch.empty_like(u)
    _check(out, "out", dev, u.dtype, u.shape)
    st = lib.sscan_fwd_noalloc(_ptr(u), _ptr(delta), _ptr(delta_bias), int(bool(softplus)), _ptr(A), _ptr(B), _ptr(C),
                               _ptr(D), _ptr(z), _ptr(out), b, d, L, DSTATE, int(bool(reverse)), _stream(dev),
                               _DT_CODE[u.dtype], _DT_CODE[B.dtype])
    if st != 0:
        raise SScanError(st, "sscan_fwd_noalloc")
    return out


def fwd_state(u, delta, A, B, C, D=None, z=None, delta_bias=None, h0: Optional[torch.Tensor] = None,
              h_last: Optional[torch.Tensor] = None, softplus: bool = True, reverse: bool = False,
              out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """One-direction scan with state I/O (``sscan_fwd_state``).  h0 (optional) is
    the state before the first scanned token, [batch, dim, 16] f32; the state after
    the last scanned token is written to ``h_last`` (allocated if None, may be h0
    itself).  Returns (out, h_last)."""
    lib = load_library()
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("sscan.fwd_state needs CUDA (HIP) tensors")
    if u.dtype not in _DT_CODE or B.dtype not in _DT_CODE:
        raise TypeError("u/delta/z and B/C must be float32 or bfloat16")
    b, d, L = u.shape
    _check(u, "u", dev)
    _check(delta, "delta", dev, u.dtype, u.shape)
    _check(z, "z", dev, u.dtype, u.shape)
    _check(A, "A", dev, torch.float32, (d, DSTATE))
    _check(B, "B", dev, None, (b, DSTATE, L))
    _check(C, "C", dev, B.dtype, (b, DSTATE, L))
    _check(D, "D", dev, torch.float32, (d,))
    _check(delta_bias, "delta_bias", dev, torch.float32, (d,))
    _check(h0, "h0", dev, torch.float32, (b, d, DSTATE))
    if h_last is None:
        h_last = torch.empty((b, d, DSTATE), dtype=torch.float32, device=dev)
    _check(h_last, "h_last", dev, torch.float32, (b, d, DSTATE))
    if out is None:
        out = torch.empty_like(u)
    _check(out, "out", dev, u.dtype, u.shape)
    if b * d == 0:
        return out, h_last
    ws, ws_bytes = _workspace(workspace_bytes(b, d, L, DSTATE, False), dev, workspace)
    st = lib.sscan_fwd_state(_ptr(u), _ptr(delta), _ptr(delta_bias), int(bool(softplus)), _ptr(A), _ptr(B), _ptr(C),
                             _ptr(D), _ptr(z), _ptr(out), _ptr(h0), _ptr(h_last), b, d, L, DSTATE,
                             int(bool(reverse)), _stream(dev), _DT_CODE[u.dtype], _DT_CODE[B.dtype], _ptr(ws),
                             ws_bytes)
    if st != 0:
        raise SScanError(st, "sscan_fwd_state")
    return out, h_last


def step(state, u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus: bool = True,
         out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token from a stored state (``sscan_step``), updating ``state``
    [batch, dim, 16] f32 in place.  u, delta, z: [batch, dim]; B, C: [batch, 16].
    Returns y [batch, dim] in u's dtype."""
    lib = load_library()
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("sscan.step needs CUDA (HIP) tensors")
    if u.dtype not in _DT_CODE or B.dtype not in _DT_CODE:
        raise TypeError("u/delta/z and B/C must be float32 or bfloat16")
    b, d = u.shape
    _check(state, "state", dev, torch.float32, (b, d, DSTATE))
    _check(u, "u", dev)
    _check(delta, "delta", dev, u.dtype, u.shape)
    _check(z, "z", dev, u.dtype, u.shape)
    _check(A, "A", dev, torch.float32, (d, DSTATE))
    _check(B, "B", dev, None, (b, DSTATE))
    _check(C, "C", dev, B.dtype, (b, DSTATE))
    _check(D, "D", dev, torch.float32, (d,))
    _check(delta_bias, "delta_bias", dev, torch.float32, (d,))
    if out is None:
        out = torch.empty_like(u)
    _check(out, "out", dev, u.dtype, u.shape)
    if u.numel() == 0:
        return out
    st = lib.sscan_step(_ptr(state), _ptr(u), _ptr(delta), _ptr(delta_bias), int(bool(softplus)), _ptr(A), _ptr(B),
                        _ptr(C), _ptr(D), _ptr(z), _ptr(out), b, d, DSTATE, _stream(dev), _DT_CODE[u.dtype],
                        _DT_CODE[B.dtype])
    if st != 0:
        raise SScanError(st, "sscan_step")
    return out


def step_conv(state, conv_state, x, conv: dict, delta, A, B, C, D=None, z=None, delta_bias=None,
              softplus: bool = True, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token through the causal convolution and the scan (``sscan_step_conv``):
    ``conv_state`` [batch, dim, width - 1] (x's dtype, may be None for width 1) and
    ``state`` [batch, dim, 16] f32 are updated in place; x, delta, z [batch, dim];
    B, C [batch, 16]; ``conv`` holds weight [dim, width] f32 and optional bias and
    silu.  Returns y [batch, dim] in x's dtype."""
    lib = load_library()
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("sscan.step_conv needs CUDA (HIP) tensors")
    if x.dtype not in _DT_CODE or B.dtype not in _DT_CODE:
        raise TypeError("x/delta/z and B/C must be float32 or bfloat16")
    if conv.get("same", False):
        raise ValueError("the decode step needs a causal convolution")
    b, d = x.shape
    cp = _conv_params(dict(conv, same=False), d, dev)
    _check(state, "state", dev, torch.float32, (b, d, DSTATE))
    _check(conv_state, "conv_state", dev, x.dtype, (b, d, cp.width - 1))
    _check(x, "x", dev)
    _check(delta, "delta", dev, x.dtype, x.shape)
    _check(z, "z", dev, x.dtype, x.shape)
    _check(A, "A", dev, torch.float32, (d, DSTATE))
    _check(B, "B", dev, None, (b, DSTATE))
    _check(C, "C", dev, B.dtype, (b, DSTATE))
    _check(D, "D", dev, torch.float32, (d,))
    _check(delta_bias, "delta_bias", dev, torch.float32, (d,))
    if out is None:
        out = torch.empty_like(x)
    _check(out, "out", dev, x.dtype, x.shape)
    if x.numel() == 0:
        return out
    st = lib.sscan_step_conv(_ptr(state), _ptr(conv_state) if conv_state is not None and conv_state.numel() else None,
                             _ptr(x), ctypes.byref(cp), _ptr(delta), _ptr(delta_bias), int(bool(softplus)), _ptr(A),
                             _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(out), b, d, DSTATE, _stream(dev),
                             _DT_CODE[x.dtype], _DT_CODE[B.dtype])
    if st != 0:
        raise SScanError(st, "sscan_step_conv")
    return out


def _dir(p: dict, name: str, dev, u, bdtype):
    b, d, L = u.shape
    _check(p["delta"], f"{name}.delta", dev, u.dtype, u.shape)
    _check(p["A"], f"{name}.A", dev, torch.float32, (d, DSTATE))
    _check(p["B"], f"{name}.B", dev, bdtype, (b, DSTATE, L))
    _check(p["C"], f"{name}.C", dev, bdtype, (b, DSTATE, L))
    _check(p.get("D"), f"{name}.D", dev, torch.float32, (d,))
    _check(p.get("delta_bias"), f"{name}.delta_bias", dev, torch.float32, (d,))
    return DirParams(p["delta"].data_ptr(), p["delta_bias"].data_ptr() if p.get("delta_bias") is not None else None,
                     p["A"].data_ptr(), p["B"].data_ptr(), p["C"].data_ptr(),
                     p["D"].data_ptr() if p.get("D") is not None else None)


def bidir(u, z, fwd: dict, rev: dict, softplus: bool = True, out: Optional[torch.Tensor] = None,
          workspace: Optional[torch.Tensor] = None, events: Optional[HipEvents] = None) -> torch.Tensor:
    """Bidirectional scan (``sscan_bidir``): ``fwd`` and ``rev`` are dicts with
    delta, A, B, C and optional D, delta_bias.  Returns (y_fwd + y_rev) * silu(z)."""
    lib = load_library()
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("sscan.bidir needs CUDA (HIP) tensors")
    if u.dtype not in _DT_CODE or fwd["B"].dtype not in _DT_CODE:
        raise TypeError("u/delta/z and B/C must be float32 or bfloat16")
    b, d, L = u.shape
    _check(u, "u", dev)
    _check(z, "z", dev, u.dtype, u.shape)
    pf = _dir(fwd, "fwd", dev, u, fwd["B"].dtype)
    pr = _dir(rev, "rev", dev, u, fwd["B"].dtype)
    if out is None:
        out = torch.empty_like(u)
    _check(out, "out", dev, u.dtype, u.shape)
    if u.numel() == 0:
        return out
    ws, ws_bytes = _workspace(workspace_bytes(b, d, L, DSTATE, True), dev, workspace)
    args = [_ptr(u), _ptr(z), _ptr(out), ctypes.byref(pf), ctypes.byref(pr), int(bool(softplus)), b, d, L, DSTATE,
            _stream(dev), _DT_CODE[u.dtype], _DT_CODE[fwd["B"].dtype], _ptr(ws), ws_bytes]
    if events is None:
        st = lib.sscan_bidir(*args)
    else:
        if events.steps != PROFILE_STEPS:
            raise ValueError("sscan.bidir needs HipEvents(PROFILE_STEPS)")
        st = lib.sscan_bidir_profiled(*args, ctypes.cast(events.handles, ctypes.c_void_p))
    if st != 0:
        raise SScanError(st, "sscan_bidir")
    return out


def _conv_params(conv: dict, dim: int, dev) -> ConvParams:
    w = conv["weight"]
    _check(w, "conv weight", dev, torch.float32)
    if w.dim() != 2 or w.shape[0] != dim:
        raise ValueError(f"conv weight must be [dim={dim}, width]")
    _check(conv.get("bias"), "conv bias", dev, torch.float32, (dim,))
    b = conv.get("bias")
    return ConvParams(w.data_ptr(), b.data_ptr() if b is not None else None, int(w.shape[1]),
                      int(bool(conv.get("same", False))), int(bool(conv.get("silu", False))))


def conv1d(x, weight, bias=None, same: bool = False, silu: bool = False,
           out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Depthwise convolution of each channel (``sscan_conv1d``): x [batch, dim, len]
    f32/bf16, weight [dim, width] f32 (causal, or centred when ``same``), optional
    bias [dim] f32, optional silu."""
    lib = load_library()
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("sscan.conv1d needs CUDA (HIP) tensors")
    if x.dtype not in _DT_CODE:
        raise TypeError("x must be float32 or bfloat16")
    b, d, L = x.shape
    _check(x, "x", dev)
    cp = _conv_params(dict(weight=weight, bias=bias, same=same, silu=silu), d, dev)
    if out is None:
        out = torch.empty_like(x)
    _check(out, "out", dev, x.dtype, x.shape)
    st = lib.sscan_conv1d(_ptr(x), ctypes.byref(cp), _ptr(out), b, d, L, _stream(dev), _DT_CODE[x.dtype])
    if st != 0:
        raise SScanError(st, "sscan_conv1d")
    return out


def _fwd_events(events: Optional[HipEvents]):
    if events is None:
        return None
    if events.steps != PROFILE_STEPS:
        raise ValueError("the forward calls need HipEvents(PROFILE_STEPS)")
    return ctypes.cast(events.handles, ctypes.c_void_p)


def fwd_conv(x, conv: dict, delta, A, B, C, D=None, z=None, delta_bias=None, softplus: bool = True,
             reverse: bool = False, out: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None, events: Optional[HipEvents] = None) -> torch.Tensor:
    """``sscan_fwd_conv``: the scan of u = conv(x), the convolution computed inside
    the scan kernels.  ``conv`` holds weight [dim, width] f32 and optional bias,
    same, silu."""
    lib = load_library()
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("sscan.fwd_conv needs CUDA (HIP) tensors")
    if x.dtype not in _DT_CODE or B.dtype not in _DT_CODE:
        raise TypeError("x/delta/z and B/C must be float32 or bfloat16")
    b, d, L = x.shape
    _check(x, "x", dev)
    _check(delta, "delta", dev, x.dtype, x.shape)
    _check(z, "z", dev, x.dtype, x.shape)
    _check(A, "A", dev, torch.float32, (d, DSTATE))
    _check(B, "B", dev, None, (b, DSTATE, L))
    _check(C, "C", dev, B.dtype, (b, DSTATE, L))
    _check(D, "D", dev, torch.float32, (d,))
    _check(delta_bias, "delta_bias", dev, torch.float32, (d,))
    cp = _conv_params(conv, d, dev)
    if out is None:
        out = torch.empty_like(x)
    _check(out, "out", dev, x.dtype, x.shape)
    if x.numel() == 0:
        return out
    ws, ws_bytes = _workspace(workspace_bytes(b, d, L, DSTATE, False), dev, workspace)
    args = [_ptr(x), ctypes.byref(cp), _ptr(delta), _ptr(delta_bias), int(bool(softplus)), _ptr(A), _ptr(B), _ptr(C),
            _ptr(D), _ptr(z), _ptr(out), b, d, L, DSTATE, int(bool(reverse)), _stream(dev), _DT_CODE[x.dtype],
            _DT_CODE[B.dtype], _ptr(ws), ws_bytes]
    ev = _fwd_events(events)
    st = lib.sscan_fwd_conv(*args) if ev is None else lib.sscan_fwd_conv_profiled(*args, ev)
    if st != 0:
        raise SScanError(st, "sscan_fwd_conv")
    return out


def bidir_conv(x, conv: dict, z, fwd: dict, rev: dict, softplus: bool = True, out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, events: Optional[HipEvents] = None) -> torch.Tensor:
    """``sscan_bidir_conv``: both directions over u = conv(x), summed, gated once."""
    lib = load_library()
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("sscan.bidir_conv needs CUDA (HIP) tensors")
    if x.dtype not in _DT_CODE or fwd["B"].dtype not in _DT_CODE:
        raise TypeError("x/delta/z and B/C must be float32 or bfloat16")
    b, d, L = x.shape
    _check(x, "x", dev)
    _check(z, "z", dev, x.dtype, x.shape)
    pf = _dir(fwd, "fwd", dev, x, fwd["B"].dtype)
    pr = _dir(rev, "rev", dev, x, fwd["B"].dtype)
    cp = _conv_params(conv, d, dev)
    if out is None:
        out = torch.empty_like(x)
    _check(out, "out", dev, x.dtype, x.shape)
    if x.numel() == 0:
        return out
    ws, ws_bytes = _workspace(workspace_bytes(b, d, L, DSTATE, True), dev, workspace)
    args = [_ptr(x), ctypes.byref(cp), _ptr(z), _ptr(out), ctypes.byref(pf), ctypes.byref(pr), int(bool(softplus)), b,
            d, L, DSTATE, _stream(dev), _DT_CODE[x.dtype], _DT_CODE[fwd["B"].dtype], _ptr(ws), ws_bytes]
    ev = _fwd_events(events)
    st = lib.sscan_bidir_conv(*args) if ev is None else lib.sscan_bidir_conv_profiled(*args, ev)
    if st != 0:
        raise SScanError(st, "sscan_bidir_conv")
    return out


ORDER_ROW, ORDER_ROW_REV, ORDER_COL, ORDER_COL_REV, ORDER_INDEX, ORDER_INDEX_REV = range(6)


def spiral_order(height: int, width: int) -> torch.Tensor:
    """The centre-out clockwise spiral over a [height, width] map (``sscan_spiral_order``,
    host code): int32 CPU tensor of row-major token indices."""
    out = torch.empty(height * width, dtype=torch.int32)
    st = load_library().sscan_spiral_order(height, width, ctypes.c_void_p(out.data_ptr()) if out.numel() else None)
    if st != 0:
        raise SScanError(st, "sscan_spiral_order")
    return out


def multi_workspace_bytes(batch, dim, height, width, kinds, io_dtype=torch.float32, bc_dtype=torch.float32) -> int:
    k = (ctypes.c_int * len(kinds))(*kinds)
    return int(load_library().sscan_multi_workspace_bytes(batch, dim, height, width, DSTATE, k, len(kinds),
                                                          _DT_CODE[io_dtype], _DT_CODE[bc_dtype]))


def multi(u, z, dirs, kinds, height: int, width: int, index: Optional[torch.Tensor] = None, softplus: bool = True,
          out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``sscan_multi``: the map [height, width] (flattened row-major in u's last
    axis) scanned along the orders ``kinds`` (ORDER_*), one parameter dict per
    direction (delta, A, B, C, optional D, delta_bias, all in token layout); the
    directions' outputs are summed and gated once.  ``index`` (device int32
    permutation) is needed by the index orders."""
    lib = load_library()
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("sscan.multi needs CUDA (HIP) tensors")
    if u.dtype not in _DT_CODE or dirs[0]["B"].dtype not in _DT_CODE:
        raise TypeError("u/delta/z and B/C must be float32 or bfloat16")
    b, d, L = u.shape
    if L != height * width:
        raise ValueError("u's last axis must be height * width")
    if len(dirs) != len(kinds):
        raise ValueError("one parameter dict per order")
    _check(u, "u", dev)
    _check(z, "z", dev, u.dtype, u.shape)
    _check(index, "index", dev, torch.int32, (L,))
    bdt = dirs[0]["B"].dtype
    ps = [_dir(p, f"dirs[{k}]", dev, u, bdt) for k, p in enumerate(dirs)]
    arr = (DirParams * len(ps))(*ps)
    kk = (ctypes.c_int * len(kinds))(*kinds)
    if out is None:
        out = torch.empty_like(u)
    _check(out, "out", dev, u.dtype, u.shape)
    if u.numel() == 0:
        return out
    nbytes = multi_workspace_bytes(b, d, height, width, kinds, u.dtype, bdt)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _check(workspace, "workspace", dev)
    st = lib.sscan_multi(_ptr(u), _ptr(z), _ptr(out), arr, kk, len(kinds), _ptr(index), int(bool(softplus)), b, d,
                         height, width, DSTATE, _stream(dev), _DT_CODE[u.dtype], _DT_CODE[bdt], _ptr(workspace),
                         workspace.numel())
    if st != 0:
        raise SScanError(st, "sscan_multi")
    return out


def multi_bwd_workspace_bytes(batch, dim, height, width, kinds, io_dtype=torch.float32,
                              bc_dtype=torch.float32) -> int:
    k = (ctypes.c_int * len(kinds))(*kinds)
    return int(load_library().sscan_multi_bwd_workspace_bytes(batch, dim, height, width, DSTATE, k, len(kinds),
                                                              _DT_CODE[io_dtype], _DT_CODE[bc_dtype]))


def multi_bwd(u, z, dout, dirs, kinds, height: int, width: int, index: Optional[torch.Tensor] = None,
              softplus: bool = True, workspace: Optional[torch.Tensor] = None) -> dict:
    """Backward pass of ``multi`` (``sscan_multi_bwd``): gradients of
    sum(dout * out).  Returns {"du", "dz" (None without z), "dirs": [one dict per
    direction with ddelta, ddelta_bias, dA, dB, dC, dD as in ``bwd``]}."""
    lib = load_library()
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("sscan.multi_bwd needs CUDA (HIP) tensors")
    if u.dtype not in _DT_CODE or dirs[0]["B"].dtype not in _DT_CODE:
        raise TypeError("u/delta/z and B/C must be float32 or bfloat16")
    b, d, L = u.shape
    if L != height * width:
        raise ValueError("u's last axis must be height * width")
    if len(dirs) != len(kinds):
        raise ValueError("one parameter dict per order")
    _check(u, "u", dev)
    _check(z, "z", dev, u.dtype, u.shape)
    _check(dout, "dout", dev, u.dtype, u.shape)
    _check(index, "index", dev, torch.int32, (L,))
    bdt = dirs[0]["B"].dtype
    ps = [_dir(p, f"dirs[{k}]", dev, u, bdt) for k, p in enumerate(dirs)]
    gs = [_grads_for(p, u) for p in dirs]
    arr = (DirParams * len(ps))(*ps)
    garr = (DirGrads * len(gs))(*[g[1] for g in gs])
    kk = (ctypes.c_int * len(kinds))(*kinds)
    du = torch.empty_like(u)
    dz = torch.empty_like(u) if z is not None else None
    nbytes = multi_bwd_workspace_bytes(b, d, height, width, kinds, u.dtype, bdt)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    _check(workspace, "workspace", dev)
    st = lib.sscan_multi_bwd(_ptr(u), _ptr(z), _ptr(dout), _ptr(du), _ptr(dz), arr, garr, kk, len(kinds), _ptr(index),
                             int(bool(softplus)), b, d, height, width, DSTATE, _stream(dev), _DT_CODE[u.dtype],
                             _DT_CODE[bdt], _ptr(workspace), workspace.numel())
    if st != 0:
        raise SScanError(st, "sscan_multi_bwd")
    return {"du": du, "dz": dz, "dirs": [g[0] for g in gs]}


def bwd_workspace_bytes(batch: int, dim: int, length: int, dstate: int = DSTATE, bidir: bool = False) -> int:
    return int(load_library().sscan_bwd_workspace_bytes(batch, dim, length, dstate, int(bool(bidir))))


def _grads_for(p: dict, u):
    """Output tensors for one direction's gradients (shapes and dtypes of its inputs)."""
    d = u.shape[1]
    dev = u.device
    g = {"ddelta": torch.empty_like(p["delta"]), "dA": torch.empty_like(p["A"]),
         "dB": torch.empty_like(p["B"]), "dC": torch.empty_like(p["C"]),
         "ddelta_bias": torch.empty(d, dtype=torch.float32, device=dev) if p.get("delta_bias") is not None else None,
         "dD": torch.empty(d, dtype=torch.float32, device=dev) if p.get("D") is not None else None}
    st = DirGrads(g["ddelta"].data_ptr(), g["ddelta_bias"].data_ptr() if g["ddelta_bias"] is not None else None,
                  g["dA"].data_ptr(), g["dB"].data_ptr(), g["dC"].data_ptr(),
                  g["dD"].data_ptr() if g["dD"] is not None else None)
    return g, st


def _bwd_events(events: Optional[HipEvents]):
    if events is None:
        return None
    if events.steps != BWD_PROFILE_STEPS:
        raise ValueError("the backward calls need HipEvents(BWD_PROFILE_STEPS)")
    return ctypes.cast(events.handles, ctypes.c_void_p)


def bwd(u, delta, A, B, C, dout, D=None, z=None, delta_bias=None, softplus: bool = True, reverse: bool = False,
        workspace: Optional[torch.Tensor] = None, events: Optional[HipEvents] = None) -> dict:
    """Backward pass of ``fwd`` (``sscan_bwd``): gradients of sum(dout * out).
    Returns a dict with du, dz (None without z), ddelta, ddelta_bias, dA, dB, dC, dD
    (None for an absent optional input), in the dtypes of the matching inputs."""
    lib = load_library()
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("sscan.bwd needs CUDA (HIP) tensors")
    if u.dtype not in _DT_CODE or B.dtype not in _DT_CODE:
        raise TypeError("u/delta/z and B/C must be float32 or bfloat16")
    b, d, L = u.shape
    _check(u, "u", dev)
    _check(delta, "delta", dev, u.dtype, u.shape)
    _check(z, "z", dev, u.dtype, u.shape)
    _check(dout, "dout", dev, u.dtype, u.shape)
    _check(A, "A", dev, torch.float32, (d, DSTATE))
    _check(B, "B", dev, None, (b, DSTATE, L))
    _check(C, "C", dev, B.dtype, (b, DSTATE, L))
    _check(D, "D", dev, torch.float32, (d,))
    _check(delta_bias, "delta_bias", dev, torch.float32, (d,))
    p = dict(delta=delta, A=A, B=B, C=C, D=D, delta_bias=delta_bias)
    g, gst = _grads_for(p, u)
    du = torch.empty_like(u)
    dz = torch.empty_like(u) if z is not None else None
    ws, ws_bytes = _workspace(bwd_workspace_bytes(b, d, L, DSTATE, False), dev, workspace)
    args = [_ptr(u), _ptr(delta), _ptr(delta_bias), int(bool(softplus)), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
            _ptr(z), _ptr(dout), _ptr(du), _ptr(dz), ctypes.byref(gst), b, d, L, DSTATE, int(bool(reverse)),
            _stream(dev), _DT_CODE[u.dtype], _DT_CODE[B.dtype], _ptr(ws), ws_bytes]
    ev = _bwd_events(events)
    st = lib.sscan_bwd(*args) if ev is None else lib.sscan_bwd_profiled(*args, ev)
    if st != 0:
        raise SScanError(st, "sscan_bwd")
    return dict(g, du=du, dz=dz)


def bwd_state(u, delta, A, B, C, dout, D=None, z=None, delta_bias=None, h0=None, dh_last=None,
              softplus: bool = True, reverse: bool = False, workspace: Optional[torch.Tensor] = None) -> dict:
    """Backward pass of ``fwd_state`` (``sscan_bwd_state``): the gradients of
    sum(dout * out) + sum(dh_last * h_last) given the forward's entry state ``h0``;
    returns ``bwd``'s dict plus "dh0" [batch, dim, 16] f32."""
    lib = load_library()
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("sscan.bwd_state needs CUDA (HIP) tensors")
    if u.dtype not in _DT_CODE or B.dtype not in _DT_CODE:
        raise TypeError("u/delta/z and B/C must be float32 or bfloat16")
    b, d, L = u.shape
    _check(u, "u", dev)
    _check(delta, "delta", dev, u.dtype, u.shape)
    _check(z, "z", dev, u.dtype, u.shape)
    _check(dout, "dout", dev, u.dtype, u.shape)
    _check(A, "A", dev, torch.float32, (d, DSTATE))
    _check(B, "B", dev, None, (b, DSTATE, L))
    _check(C, "C", dev, B.dtype, (b, DSTATE, L))
    _check(D, "D", dev, torch.float32, (d,))
    _check(delta_bias, "delta_bias", dev, torch.float32, (d,))
    _check(h0, "h0", dev, torch.float32, (b, d, DSTATE))
    _check(dh_last, "dh_last", dev, torch.float32, (b, d, DSTATE))
    g, gst = _grads_for(dict(delta=delta, A=A, B=B, C=C, D=D, delta_bias=delta_bias), u)
    du = torch.empty_like(u)
    dz = torch.empty_like(u) if z is not None else None
    dh0 = torch.empty((b, d, DSTATE), dtype=torch.float32, device=dev)
    ws, ws_bytes = _workspace(bwd_workspace_bytes(b, d, L, DSTATE, False), dev, workspace)
    st = lib.sscan_bwd_state(_ptr(u), _ptr(delta), _ptr(delta_bias), int(bool(softplus)), _ptr(A), _ptr(B), _ptr(C),
                             _ptr(D), _ptr(z), _ptr(dout), _ptr(h0), _ptr(dh_last), _ptr(du), _ptr(dz),
                             ctypes.byref(gst), _ptr(dh0), b, d, L, DSTATE, int(bool(reverse)), _stream(dev),
                             _DT_CODE[u.dtype], _DT_CODE[B.dtype], _ptr(ws), ws_bytes)
    if st != 0:
        raise SScanError(st, "sscan_bwd_state")
    return dict(g, du=du, dz=dz, dh0=dh0)


def bidir_bwd(u, z, dout, fwd: dict, rev: dict, softplus: bool = True,
              workspace: Optional[torch.Tensor] = None, events: Optional[HipEvents] = None) -> dict:
    """Backward pass of ``bidir`` (``sscan_bidir_bwd``).  Returns {"du", "dz",
    "fwd": {...}, "rev": {...}} with each direction's gradients as in ``bwd``."""
    lib = load_library()
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("sscan.bidir_bwd needs CUDA (HIP) tensors")
    if u.dtype not in _DT_CODE or fwd["B"].dtype not in _DT_CODE:
        raise TypeError("u/delta/z and B/C must be float32 or bfloat16")
    b, d, L = u.shape
    _check(u, "u", dev)
    _check(z, "z", dev, u.dtype, u.shape)
    _check(dout, "dout", dev, u.dtype, u.shape)
    pf = _dir(fwd, "fwd", dev, u, fwd["B"].dtype)
    pr = _dir(rev, "rev", dev, u, fwd["B"].dtype)
    gf, gfs = _grads_for(fwd, u)
    gr, grs = _grads_for(rev, u)
    du = torch.empty_like(u)
    dz = torch.empty_like(u) if z is not None else None
    ws, ws_bytes = _workspace(bwd_workspace_bytes(b, d, L, DSTATE, True), dev, workspace)
    args = [_ptr(u), _ptr(z), _ptr(dout), _ptr(du), _ptr(dz), ctypes.byref(pf), ctypes.byref(pr),
            ctypes.byref(gfs), ctypes.byref(grs), int(bool(softplus)), b, d, L, DSTATE, _stream(dev),
            _DT_CODE[u.dtype], _DT_CODE[fwd["B"].dtype], _ptr(ws), ws_bytes]
    ev = _bwd_events(events)
    st = lib.sscan_bidir_bwd(*args) if ev is None else lib.sscan_bidir_bwd_profiled(*args, ev)
    if st != 0:
        raise SScanError(st, "sscan_bidir_bwd")
    return {"du": du, "dz": dz, "fwd": gf, "rev": gr}


def bwd_conv_workspace_bytes(batch: int, dim: int, length: int, dstate: int = DSTATE, bidir: bool = False,
                             io_dtype=torch.float32) -> int:
    return int(load_library().sscan_bwd_conv_workspace_bytes(batch, dim, length, dstate, int(bool(bidir)),
                                                             _DT_CODE[io_dtype]))


def _conv_grads(conv: dict, dim: int, dev):
    dw = torch.empty((dim, conv["weight"].shape[1]), dtype=torch.float32, device=dev)
    db = torch.empty(dim, dtype=torch.float32, device=dev) if conv.get("bias") is not None else None
    return dw, db


def bwd_conv(x, conv: dict, delta, A, B, C, dout, D=None, z=None, delta_bias=None, softplus: bool = True,
             reverse: bool = False, workspace: Optional[torch.Tensor] = None) -> dict:
    """Backward of ``fwd_conv`` (``sscan_bwd_conv``): the gradients of ``bwd`` with
    dx in place of du, plus dconv_w [dim, width] and dconv_b [dim] (None without a
    convolution bias)."""
    lib = load_library()
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("sscan.bwd_conv needs CUDA (HIP) tensors")
    if x.dtype not in _DT_CODE or B.dtype not in _DT_CODE:
        raise TypeError("x/delta/z and B/C must be float32 or bfloat16")
    b, d, L = x.shape
    _check(x, "x", dev)
    _check(delta, "delta", dev, x.dtype, x.shape)
    _check(z, "z", dev, x.dtype, x.shape)
    _check(dout, "dout", dev, x.dtype, x.shape)
    _check(A, "A", dev, torch.float32, (d, DSTATE))
    _check(B, "B", dev, None, (b, DSTATE, L))
    _check(C, "C", dev, B.dtype, (b, DSTATE, L))
    _check(D, "D", dev, torch.float32, (d,))
    _check(delta_bias, "delta_bias", dev, torch.float32, (d,))
    cp = _conv_params(conv, d, dev)
    g, gst = _grads_for(dict(delta=delta, A=A, B=B, C=C, D=D, delta_bias=delta_bias), x)
    dx = torch.empty_like(x)
    dz = torch.empty_like(x) if z is not None else None
    dw, db = _conv_grads(conv, d, dev)
    nbytes = bwd_conv_workspace_bytes(b, d, L, DSTATE, False, x.dtype)
    ws, ws_bytes = _workspace(nbytes, dev, workspace)
    st = lib.sscan_bwd_conv(_ptr(x), ctypes.byref(cp), _ptr(delta), _ptr(delta_bias), int(bool(softplus)), _ptr(A),
                            _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(dout), _ptr(dx), _ptr(dz), ctypes.byref(gst),
                            _ptr(dw), _ptr(db), b, d, L, DSTATE, int(bool(reverse)), _stream(dev), _DT_CODE[x.dtype],
                            _DT_CODE[B.dtype], _ptr(ws), ws_bytes)
    if st != 0:
        raise SScanError(st, "sscan_bwd_conv")
    return dict(g, dx=dx, dz=dz, dconv_w=dw, dconv_b=db)


def bidir_bwd_conv(x, conv: dict, z, dout, fwd: dict, rev: dict, softplus: bool = True,
                   workspace: Optional[torch.Tensor] = None) -> dict:
    """Backward of ``bidir_conv`` (``sscan_bidir_bwd_conv``): {"dx", "dz", "dconv_w",
    "dconv_b", "fwd": {...}, "rev": {...}}."""
    lib = load_library()
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("sscan.bidir_bwd_conv needs CUDA (HIP) tensors")
    if x.dtype not in _DT_CODE or fwd["B"].dtype not in _DT_CODE:
        raise TypeError("x/delta/z and B/C must be float32 or bfloat16")
    b, d, L = x.shape
    _check(x, "x", dev)
    _check(z, "z", dev, x.dtype, x.shape)
    _check(dout, "dout", dev, x.dtype, x.shape)
    pf = _dir(fwd, "fwd", dev, x, fwd["B"].dtype)
    pr = _dir(rev, "rev", dev, x, fwd["B"].dtype)
    cp = _conv_params(conv, d, dev)
    gf, gfs = _grads_for(fwd, x)
    gr, grs = _grads_for(rev, x)
    dx = torch.empty_like(x)
    dz = torch.empty_like(x) if z is not None else None
    dw, db = _conv_grads(conv, d, dev)
    nbytes = bwd_conv_workspace_bytes(b, d, L, DSTATE, True, x.dtype)
    ws, ws_bytes = _workspace(nbytes, dev, workspace)
    st = lib.sscan_bidir_bwd_conv(_ptr(x), ctypes.byref(cp), _ptr(z), _ptr(dout), _ptr(dx), _ptr(dz),
                                  ctypes.byref(pf), ctypes.byref(pr), ctypes.byref(gfs), ctypes.byref(grs), _ptr(dw),
                                  _ptr(db), int(bool(softplus)), b, d, L, DSTATE, _stream(dev), _DT_CODE[x.dtype],
                                  _DT_CODE[fwd["B"].dtype], _ptr(ws), ws_bytes)
    if st != 0:
        raise SScanError(st, "sscan_bidir_bwd_conv")
    return {"dx": dx, "dz": dz, "dconv_w": dw, "dconv_b": db, "fwd": gf, "rev": gr}


def run_inputs(x, softplus: bool = True, out=None, workspace=None, events: Optional[HipEvents] = None) -> torch.Tensor:
    """Runs the scan on a ``ScanInputs`` already on the device (one or two directions)."""
    if len(x.dirs) == 1:
        p = x.dirs[0]
        return fwd(x.u, x.delta, p.A, p.B, p.C, p.D, x.z, p.delta_bias, softplus=softplus, out=out,
                   workspace=workspace, events=events)
    f, r = x.dirs
    mk = lambda p: dict(delta=x.delta, delta_bias=p.delta_bias, A=p.A, B=p.B, C=p.C, D=p.D)
    return bidir(x.u, x.z, mk(f), mk(r), softplus=softplus, out=out, workspace=workspace, events=events)


# ---- autograd ---------------------------------------------------------------------
# torch.autograd.Function wrappers: the forward call, and in backward the matching
# backward entry point (the forward states are recomputed there, nothing beyond the
# inputs is kept).  Argument marshalling only, like the functions above.

class _ScanFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, delta, A, B, C, D, z, delta_bias, softplus, reverse):
        ctx.save_for_backward(u, delta, A, B, C, D, z, delta_bias)
        ctx.softplus, ctx.reverse = softplus, reverse
        return fwd(u, delta, A, B, C, D, z, delta_bias, softplus=softplus, reverse=reverse)

    @staticmethod
    def backward(ctx, dout):
        u, delta, A, B, C, D, z, delta_bias = ctx.saved_tensors
        g = bwd(u, delta, A, B, C, dout.contiguous(), D=D, z=z, delta_bias=delta_bias, softplus=ctx.softplus,
                reverse=ctx.reverse)
        return (g["du"], g["ddelta"], g["dA"], g["dB"], g["dC"], g["dD"], g["dz"], g["ddelta_bias"], None, None)


def selective_scan(u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus: bool = True,
                   reverse: bool = False) -> torch.Tensor:
    """``fwd`` with gradients: differentiable in every tensor argument (``sscan_bwd``
    in the backward pass)."""
    return _ScanFn.apply(u, delta, A, B, C, D, z, delta_bias, softplus, reverse)


class _BidirFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, z, d_f, A_f, B_f, C_f, D_f, bias_f, d_r, A_r, B_r, C_r, D_r, bias_r, softplus):
        ctx.save_for_backward(u, z, d_f, A_f, B_f, C_f, D_f, bias_f, d_r, A_r, B_r, C_r, D_r, bias_r)
        ctx.softplus = softplus
        pf = dict(delta=d_f, A=A_f, B=B_f, C=C_f, D=D_f, delta_bias=bias_f)
        pr = dict(delta=d_r, A=A_r, B=B_r, C=C_r, D=D_r, delta_bias=bias_r)
        return bidir(u, z, pf, pr, softplus=softplus)

    @staticmethod
    def backward(ctx, dout):
        u, z, d_f, A_f, B_f, C_f, D_f, bias_f, d_r, A_r, B_r, C_r, D_r, bias_r = ctx.saved_tensors
        pf = dict(delta=d_f, A=A_f, B=B_f, C=C_f, D=D_f, delta_bias=bias_f)
        pr = dict(delta=d_r, A=A_r, B=B_r, C=C_r, D=D_r, delta_bias=bias_r)
        g = bidir_bwd(u, z, dout.contiguous(), pf, pr, softplus=ctx.softplus)
        gf, gr = g["fwd"], g["rev"]
        # a delta tensor shared by the two directions appears twice in the inputs, and
        # autograd adds the two gradients it receives for it
        return (g["du"], g["dz"],
                gf["ddelta"], gf["dA"], gf["dB"], gf["dC"], gf["dD"], gf["ddelta_bias"],
                gr["ddelta"], gr["dA"], gr["dB"], gr["dC"], gr["dD"], gr["ddelta_bias"], None)


def selective_scan_bidir(u, z, fwd_params: dict, rev_params: dict, softplus: bool = True) -> torch.Tensor:
    """``bidir`` with gradients (``sscan_bidir_bwd`` in the backward pass); each
    parameter dict holds delta, A, B, C and optional D, delta_bias."""
    f, r = fwd_params, rev_params
    return _BidirFn.apply(u, z, f["delta"], f["A"], f["B"], f["C"], f.get("D"), f.get("delta_bias"),
                          r["delta"], r["A"], r["B"], r["C"], r.get("D"), r.get("delta_bias"), softplus)


# ---- the gated delta rule ---------------------------------------------------------

# Tells autograd that kernels wrote to a tensor: a backward pass that saved it before raises
# instead of using what it holds now.
_bump = torch.autograd.graph.increment_version


def _written(*tensors) -> None:
    """``_bump`` of the caller's tensors that the kernels wrote to (None: not given)."""
    for t in tensors:
        if t is not None:
            _bump(t)


def _aligned(t):
    """A state at a 16-byte boundary, as the kernels take them: a copy of a slice of a pool
    whose states' sizes are no multiple of four."""
    return t.clone() if isinstance(t, torch.Tensor) and t.data_ptr() % 16 else t


def _apart(state, out) -> None:
    """Refuses an output over a state that is written through a copy, of which the C checks
    do not know."""
    a, b = state.data_ptr(), out.data_ptr()
    if a < b + out.numel() * out.element_size() and b < a + state.numel() * 4:
        raise ValueError("out and the state overlap")


class _NoSecond(torch.autograd.Function):
    """Gradients as they are, whose own backward pass raises."""

    @staticmethod
    def forward(ctx, n, *tensors):
        return tuple(t.view_as(t) for t in tensors[:n])

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("the gated delta rule and the norms around a mixer have no second derivatives")


def _first_order(backward):
    """A backward pass whose gradients cannot be differentiated again: where a graph of them
    is made (``create_graph``) they say so when it is used, instead of counting as constants
    (torch's once_differentiable leaves them constants where only the saved inputs require
    gradients, as those of a sum of the outputs do)."""

    @functools.wraps(backward)
    def run(ctx, *grads):
        with torch.no_grad():
            r = backward(ctx, *grads)
        if not torch.is_grad_enabled():
            return r
        at = [i for i, t in enumerate(r) if t is not None]
        on = [t for t in (*ctx.saved_tensors, *grads) if t is not None and t.requires_grad]
        marked = dict(zip(at, _NoSecond.apply(len(at), *(r[i] for i in at), *on)))
        return tuple(marked.get(i) for i in range(len(r)))

    return run


def _strided(t, name: str, device, dtype, shape, unit: bool = True):
    """A tensor the kernels read through its own strides: only the last dimension has
    to be contiguous (``unit``; the gates have none)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if unit and shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")


def _delta_check(what, q, k, v, g, beta, lengths, tokens: bool):
    """Raises what is wrong with the inputs of a delta call (its fast test failed)."""
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    dev = q.device
    if dev.type != "cuda":
        raise ValueError(f"sscan.{what} needs CUDA (HIP) tensors")
    if q.dtype not in _DT_CODE:
        raise TypeError("q/k/v must be float32 or bfloat16")
    if q.dim() != 3 + tokens or v.dim() != 3 + tokens:
        raise ValueError("q, k are [batch, len, qk_heads, dk] and v is [batch, len, v_heads, dv]" if tokens else
                         "q, k are [batch, qk_heads, dk] and v is [batch, v_heads, dv]")
    lead, (hk, dk), (hv, dv) = q.shape[:-2], q.shape[-2:], v.shape[-2:]
    if hv % max(hk, 1) or (hk == 0) != (hv == 0):
        raise ValueError(f"v_heads ({hv}) must be a multiple of qk_heads ({hk})")
    _strided(q, "q", dev, q.dtype, (*lead, hk, dk))
    _strided(k, "k", dev, q.dtype, (*lead, hk, dk))
    _strided(v, "v", dev, q.dtype, (*lead, hv, dv))
    _strided(g, "g", dev, torch.float32, (*lead, hv), unit=False)
    _strided(beta, "beta", dev, torch.float32, (*lead, hv), unit=False)
    _check(lengths, "lengths", dev, torch.int32, (q.shape[0],))


def _delta_pack(what, q, k, v, g, beta, h0, lengths, scale, qk_norm, tokens: bool = True):
    """Checks the inputs of a delta call; (packed params, device, sizes (b, L, hk, hv, dk, dv), dtype code)."""
    try:
        qs, vs, dt, di = q.shape, v.shape, q.dtype, q.get_device()
        qt, kt, vt, gt, bt = q.stride(), k.stride(), v.stride(), g.stride(), beta.stride()
    except AttributeError:
        _delta_check(what, q, k, v, g, beta, lengths, tokens)  # says which of them is no tensor
        raise
    code = _DT_CODE.get(dt)
    # one test of everything that is wrong only in a wrong call; _delta_check says what
    if not (code is not None and di >= 0 and len(qs) == 3 + tokens and k.shape == qs and len(vs) == len(qs)
            and vs[:-2] == qs[:-2] and g.shape == vs[:-1] and beta.shape == g.shape and k.dtype == dt
            and v.dtype == dt and g.dtype == torch.float32 and beta.dtype == torch.float32
            and k.get_device() == di and v.get_device() == di and g.get_device() == di and beta.get_device() == di
            and qt[-1] == 1 and kt[-1] == 1 and vt[-1] == 1 and lengths is None and qs[-2] and not vs[-2] % qs[-2]):
        _delta_check(what, q, k, v, g, beta, lengths, tokens)
    dev = q.device
    if tokens:
        b, L, hk, dk = qs
        strides = (*qt[:3], *kt[:3], *vt[:3], *gt, *bt)
    else:
        (b, hk, dk), L = qs, 1
        strides = (qt[0], 0, qt[1], kt[0], 0, kt[1], vt[0], 0, vt[1], gt[0], 0, gt[1], bt[0], 0, bt[1])
    hv, dv = vs[-2:]
    if h0 is not None:
        _check(h0, "h0", dev, torch.float32, (b, hv, dk, dv))
    if scale is None:
        scale = dk ** -0.5 if dk else 1.0
    p = _DELTA.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
                    0 if lengths is None else lengths.data_ptr(), 0 if h0 is None else h0.data_ptr(), *strides,
                    b, L, hk, hv, dk, dv, scale, 1 if qk_norm else 0, code)
    return p, dev, (b, L, hk, hv, dk, dv), code


def delta_workspace_bytes(batch: int, length: int, qk_heads: int, v_heads: int, dk: int, dv: int,
                          io_dtype=torch.bfloat16, backward: bool = False) -> int:
    lib = load_library()
    f = lib.sscan_delta_bwd_workspace_bytes if backward else lib.sscan_delta_workspace_bytes
    return int(f(batch, length, qk_heads, v_heads, dk, dv, _DT_CODE[io_dtype]))


def delta_plan(batch: int, length: int, qk_heads: int, v_heads: int, dk: int, dv: int,
               io_dtype=torch.bfloat16) -> dict:
    """How rows of these sizes are walked (``sscan_delta_plan``): chunks per row (0: token
    by token), segments walked at once, chunks per segment, waves per block."""
    out = (ctypes.c_int64 * 4)()
    st = load_library().sscan_delta_plan(batch, length, qk_heads, v_heads, dk, dv, _DT_CODE[io_dtype], out)
    if st != 0:
        raise SScanError(st, "sscan_delta_plan")
    return dict(nchunk=out[0], nseg=out[1], seg_chunks=out[2], waves=out[3])


def delta_fwd(q, k, v, g, beta, h0: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
              scale: Optional[float] = None, qk_norm: bool = False, out: Optional[torch.Tensor] = None,
              h_last: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """The gated delta rule over whole sequences (``sscan_delta_fwd``).  q, k: [batch,
    len, qk_heads, dk], v: [batch, len, v_heads, dv], f32/bf16; g (log decay), beta:
    [batch, len, v_heads] f32; any strides with the last dimension of q, k, v
    contiguous.  h0: [batch, v_heads, dk, dv] f32; lengths: int32 [batch].  scale
    defaults to dk ** -0.5.  Returns (out, h_last); h_last may be given as h0."""
    lib = load_library()
    h0 = _aligned(h0)
    p, dev, (b, L, hk, hv, dk, dv), code = _delta_pack("delta_fwd", q, k, v, g, beta, h0, lengths, scale, qk_norm)
    given = out, h_last
    if out is None:
        out = torch.empty((b, L, hv, dv), dtype=q.dtype, device=dev)
    else:
        _check(out, "out", dev, q.dtype, (b, L, hv, dv))
    if h_last is None:
        h_last = torch.empty((b, hv, dk, dv), dtype=torch.float32, device=dev)
    else:
        _check(h_last, "h_last", dev, torch.float32, (b, hv, dk, dv))
    if b * hv == 0:
        return out, h_last
    last = h_last
    if h_last.data_ptr() % 16:
        _apart(h_last, out)
        last = torch.empty_like(h_last)
    ws, ws_bytes = _workspace(lib.sscan_delta_workspace_bytes(b, L, hk, hv, dk, dv, code), dev, workspace)
    st = lib.sscan_delta_fwd(p, out.data_ptr(), last.data_ptr(), _stream(dev), _ptr(ws), ws_bytes)
    if st != 0:
        raise SScanError(st, "sscan_delta_fwd")
    if last is not h_last:
        h_last.copy_(last)
    _written(*given)
    return out, h_last


def delta_step(state, q, k, v, g, beta, lengths: Optional[torch.Tensor] = None, scale: Optional[float] = None,
               qk_norm: bool = False, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token from a stored state (``sscan_delta_step``), updating ``state``
    [batch, v_heads, dk, dv] f32 in place.  q, k: [batch, qk_heads, dk]; v: [batch,
    v_heads, dv]; g, beta: [batch, v_heads] f32.  Rows of ``lengths`` 0 keep their
    state and answer 0.  Returns [batch, v_heads, dv] in q's dtype."""
    lib = load_library()
    p, dev, (b, _, hk, hv, dk, dv), code = _delta_pack("delta_step", q, k, v, g, beta, None, lengths, scale, qk_norm,
                                                       tokens=False)
    if state is None:
        raise ValueError("state is required")
    _check(state, "state", dev, torch.float32, (b, hv, dk, dv))
    given = out
    if out is None:
        out = torch.empty((b, hv, dv), dtype=q.dtype, device=dev)
    else:
        _check(out, "out", dev, q.dtype, (b, hv, dv))
    if b * hv == 0:
        return out
    s, at = state, state.data_ptr()
    if at % 16:
        _apart(state, out)
        s = state.clone()
        at = s.data_ptr()
    st = lib.sscan_delta_step(p, at, out.data_ptr(), _stream(dev))
    if st != 0:
        raise SScanError(st, "sscan_delta_step")
    if s is not state:
        state.copy_(s)
    _bump(state if given is None else [state, given])
    return out


def delta_bwd(q, k, v, g, beta, dout, h0: Optional[torch.Tensor] = None, dh_last: Optional[torch.Tensor] = None,
              lengths: Optional[torch.Tensor] = None, scale: Optional[float] = None, qk_norm: bool = False,
              workspace: Optional[torch.Tensor] = None) -> dict:
    """Backward pass of ``delta_fwd`` (``sscan_delta_bwd``): the gradients of
    sum(dout * out) + sum(dh_last * h_last) as {"dq", "dk", "dv" (q's dtype), "dg",
    "dbeta", "dh0" (f32)}, contiguous; the states are recomputed."""
    lib = load_library()
    h0 = _aligned(h0)
    p, dev, (b, L, hk, hv, dk, dv), code = _delta_pack("delta_bwd", q, k, v, g, beta, h0, lengths, scale, qk_norm)
    _check(dout, "dout", dev, q.dtype, (b, L, hv, dv))
    _check(dh_last, "dh_last", dev, torch.float32, (b, hv, dk, dv))

    def new(shape, dtype):
        return torch.empty(shape, dtype=dtype, device=dev)

    r = dict(dq=new((b, L, hk, dk), q.dtype), dk=new((b, L, hk, dk), q.dtype), dv=new((b, L, hv, dv), q.dtype),
             dg=new((b, L, hv), torch.float32), dbeta=new((b, L, hv), torch.float32),
             dh0=new((b, hv, dk, dv), torch.float32))
    if b * hv == 0:
        return r
    ws, ws_bytes = _workspace(lib.sscan_delta_bwd_workspace_bytes(b, L, hk, hv, dk, dv, code), dev, workspace)
    gst = DeltaGrads(*(r[n].data_ptr() for n in ("dq", "dk", "dv", "dg", "dbeta", "dh0")))
    st = lib.sscan_delta_bwd(p, _ptr(dout), _ptr(dh_last), ctypes.byref(gst), _stream(dev), _ptr(ws),
                             ws_bytes)
    if st != 0:
        raise SScanError(st, "sscan_delta_bwd")
    return r


class _DeltaFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, h0, lengths, scale, qk_norm):
        ctx.save_for_backward(q, k, v, g, beta, h0, lengths)
        ctx.scale, ctx.qk_norm = scale, qk_norm
        ctx.set_materialize_grads(False)
        return delta_fwd(q, k, v, g, beta, h0, lengths, scale, qk_norm)

    @staticmethod
    @_first_order
    def backward(ctx, dout, dh_last):
        q, k, v, g, beta, h0, lengths = ctx.saved_tensors
        if dout is None:
            dout = torch.zeros(v.shape, dtype=v.dtype, device=v.device)
        r = delta_bwd(q, k, v, g, beta, dout.contiguous(), h0, None if dh_last is None else dh_last.contiguous(),
                      lengths, ctx.scale, ctx.qk_norm)
        return (r["dq"], r["dk"], r["dv"], r["dg"], r["dbeta"], None if h0 is None else r["dh0"], None, None, None)


def gated_delta(q, k, v, g, beta, h0: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
                scale: Optional[float] = None, qk_norm: bool = False):
    """``delta_fwd`` with gradients in q, k, v, g, beta and h0 (``sscan_delta_bwd`` in
    the backward pass; no second derivatives).  Returns (out, h_last)."""
    return _DeltaFn.apply(q, k, v, g, beta, h0, lengths, scale, qk_norm)


# ---- RMS norms around a mixer -----------------------------------------------------

# More "heads" than this are the tokens of [batch, len, size]: rows, where their strides and
# a shared weight allow it.  (The workspace of the gradients is sized for a weight each.)
_ROW_HEADS = 1024


def _row_stride(shape, stride, keep: int):
    """The one stride between the rows that the first ``keep`` dimensions collapse to, or None."""
    if keep == 1:
        return stride[0] if shape[0] > 1 else 0
    row = reach = None
    for i in range(keep - 1, -1, -1):  # innermost first: each must continue the one inside
        if shape[i] <= 1:
            continue
        if row is None:
            row = stride[i]
        elif stride[i] != reach:
            return None
        reach = stride[i] * shape[i]
    return row or 0


def _gated_params(what, x, z, weight, eps, gate_first):
    """(packed params, device, (rows, heads, size)): x and z are [..., size] or [..., heads, size]; all
    leading dimensions but the last one (the heads, where there are two or more)
    collapse to rows."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    dev, xs, dt = x.device, x.shape, x.dtype
    if dev.type != "cuda":
        raise ValueError(f"sscan.{what} needs CUDA (HIP) tensors")
    if dt not in _DT_CODE:
        raise TypeError("x/z must be float32 or bfloat16")
    if not xs:
        raise ValueError("x needs at least one dimension")
    size = xs[-1]
    _strided(x, "x", dev, dt, xs)
    _strided(z, "z", dev, dt, xs)
    heads = xs[-2] if len(xs) >= 3 else 1
    keep = len(xs) - 2 if len(xs) >= 3 else len(xs) - 1  # dimensions that collapse to rows
    per_head = isinstance(weight, torch.Tensor) and weight.dim() == 2
    if weight is not None:
        _check(weight, "weight", dev, torch.float32, (heads, size) if per_head else (size,))
    n = x.numel()
    if heads > _ROW_HEADS and not per_head and None not in (_row_stride(xs, x.stride(), keep + 1),
                                                            _row_stride(xs, z.stride(), keep + 1)):
        heads, keep = 1, keep + 1
    rows = n // (heads * size) if n else 0

    def strides(t, name):
        row = _row_stride(xs, t.stride(), keep)
        if row is None:
            raise ValueError(f"the leading dimensions of {name} must collapse to rows of one stride")
        return row, t.stride(-2) if heads > 1 else 0

    p = _GATED.pack(x.data_ptr(), z.data_ptr(), 0 if weight is None else weight.data_ptr(), *strides(x, "x"),
                    *strides(z, "z"), rows, heads, size, eps, 1 if gate_first else 0, 1 if per_head else 0,
                    _DT_CODE[dt])
    return p, dev, (rows, heads, size)


def gated_norm(x, z, weight: Optional[torch.Tensor] = None, eps: float = 1e-6, gate_first: bool = False,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """RMS norm over the last dimension fused with a silu gate (``sscan_gated_norm``):
    x / rms(x) * weight * silu(z), or with ``gate_first`` m / rms(m) * weight of m = x *
    silu(z).  x, z: [..., size] or [..., heads, size] f32/bf16 (rows and heads may be
    strided); weight: [size] or [heads, size] f32.  Returns a contiguous tensor."""
    lib = load_library()
    p, dev, _ = _gated_params("gated_norm", x, z, weight, eps, gate_first)
    given = out
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    else:
        _check(out, "out", dev, x.dtype, x.shape)
    st = lib.sscan_gated_norm(p, out.data_ptr(), _stream(dev))
    if st != 0:
        raise SScanError(st, "sscan_gated_norm")
    _written(given)
    return out


def gated_norm_bwd(x, z, dout, weight: Optional[torch.Tensor] = None, eps: float = 1e-6, gate_first: bool = False,
                   workspace: Optional[torch.Tensor] = None) -> dict:
    """Backward pass of ``gated_norm`` (``sscan_gated_norm_bwd``): {"dx", "dz",
    "dweight" (f32, None without a weight)}."""
    lib = load_library()
    p, dev, sizes = _gated_params("gated_norm_bwd", x, z, weight, eps, gate_first)
    _check(dout, "dout", dev, x.dtype, x.shape)
    dx, dz = (torch.empty(x.shape, dtype=x.dtype, device=dev) for _ in range(2))
    dw = None if weight is None else torch.empty_like(weight)
    ws, ws_bytes = _workspace(lib.sscan_gated_norm_bwd_workspace_bytes(*sizes), dev, workspace)
    st = lib.sscan_gated_norm_bwd(p, _ptr(dout), _ptr(dx), _ptr(dz), _ptr(dw), _stream(dev), _ptr(ws),
                                  ws_bytes)
    if st != 0:
        raise SScanError(st, "sscan_gated_norm_bwd")
    return dict(dx=dx, dz=dz, dweight=dw)


def _add_params(what, x, residual, residual_dtype, weight, scale, post_weight, eps):
    try:
        return _add_pack(what, x, residual, residual_dtype, weight, scale, post_weight, eps)
    except AttributeError:
        for name, t in (("x", x), ("residual", residual), ("weight", weight), ("scale", scale),
                        ("post_weight", post_weight)):
            if not isinstance(t, torch.Tensor) and (t is not None or name == "x"):
                raise TypeError(f"{name} must be a torch.Tensor") from None
        raise


def _add_pack(what, x, residual, residual_dtype, weight, scale, post_weight, eps):
    """(packed params, device, (rows, size))"""
    dev = x.device
    if dev.type != "cuda":
        raise ValueError(f"sscan.{what} needs CUDA (HIP) tensors")
    if x.dtype not in _DT_CODE or residual_dtype not in _DT_CODE:
        raise TypeError("x and the residual must be float32 or bfloat16")
    if x.dim() < 1:
        raise ValueError("x needs at least one dimension")
    size = x.shape[-1]
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if residual is not None and not (residual.dtype == residual_dtype and residual.shape == x.shape
                                     and residual.is_contiguous() and residual.device == dev):
        _check(residual, "residual", dev, residual_dtype, x.shape)
    for name, t in (("weight", weight), ("scale", scale), ("post_weight", post_weight)):
        if t is not None and not (t.dtype == torch.float32 and t.dim() == 1 and t.shape[0] == size
                                  and t.is_contiguous() and t.device == dev):
            _check(t, name, dev, torch.float32, (size,))
    addr = [0 if t is None else t.data_ptr() for t in (x, residual, weight, scale, post_weight)]
    rows = x.numel() // size if size else 0
    return _ADD.pack(*addr, rows, size, eps, _DT_CODE[x.dtype], _DT_CODE[residual_dtype]), dev, (rows, size)


def add_norm(x, residual: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
             scale: Optional[torch.Tensor] = None, post_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
             residual_dtype=None, out: Optional[torch.Tensor] = None, residual_out: Optional[torch.Tensor] = None):
    """A block's output added to the residual stream, and the next block's RMS norm
    (``sscan_add_norm``): total = residual + scale * x (x normed by ``post_weight``
    first where given), out = total / rms(total) * weight.  x: [..., size] f32/bf16;
    residual: f32/bf16 of the same shape (None: 0, stored as ``residual_dtype`` or x's
    dtype); weight, scale, post_weight: [size] f32 or None.  Returns (out, total);
    ``residual_out`` may be ``residual`` itself."""
    lib = load_library()
    if residual_dtype is None:
        residual_dtype = getattr(x if residual is None else residual, "dtype", None)
    p, dev, _ = _add_params("add_norm", x, residual, residual_dtype, weight, scale, post_weight, eps)
    given = out, residual_out
    if out is None:
        out = torch.empty_like(x)
    else:
        _check(out, "out", dev, x.dtype, x.shape)
    if residual_out is None:
        residual_out = torch.empty_like(x if residual is None else residual, dtype=residual_dtype)
    else:
        _check(residual_out, "residual_out", dev, residual_dtype, x.shape)
    st = lib.sscan_add_norm(p, out.data_ptr(), residual_out.data_ptr(), _stream(dev))
    if st != 0:
        raise SScanError(st, "sscan_add_norm")
    _written(*given)
    return out, residual_out


def add_norm_bwd(x, residual_out, dout, weight: Optional[torch.Tensor] = None,
                 dresidual_out: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                 post_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 workspace: Optional[torch.Tensor] = None) -> dict:
    """Backward pass of ``add_norm`` (``sscan_add_norm_bwd``) from the total it stored:
    {"dx", "dresidual", "dweight", "dscale", "dpost_weight"} (the last three f32, None
    for a vector that was not given)."""
    lib = load_library()
    p, dev, sizes = _add_params("add_norm_bwd", x, residual_out, getattr(residual_out, "dtype", None), weight, scale,
                                post_weight, eps)
    _check(dout, "dout", dev, x.dtype, x.shape)
    _check(dresidual_out, "dresidual_out", dev, residual_out.dtype, x.shape)
    dx, dres = torch.empty_like(x), torch.empty_like(residual_out)
    dw, ds, dp = (None if t is None else torch.empty_like(t) for t in (weight, scale, post_weight))
    ws, ws_bytes = _workspace(lib.sscan_add_norm_bwd_workspace_bytes(*sizes), dev, workspace)
    st = lib.sscan_add_norm_bwd(p, _ptr(dout), _ptr(dresidual_out), _ptr(dx), _ptr(dres), _ptr(dw),
                                _ptr(ds), _ptr(dp), _stream(dev), _ptr(ws), ws_bytes)
    if st != 0:
        raise SScanError(st, "sscan_add_norm_bwd")
    return dict(dx=dx, dresidual=dres, dweight=dw, dscale=ds, dpost_weight=dp)


class _GatedNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, z, weight, eps, gate_first):
        ctx.save_for_backward(x, z, weight)
        ctx.eps, ctx.gate_first = eps, gate_first
        return gated_norm(x, z, weight, eps, gate_first)

    @staticmethod
    @_first_order
    def backward(ctx, dout):
        x, z, weight = ctx.saved_tensors
        r = gated_norm_bwd(x, z, dout.contiguous(), weight, ctx.eps, ctx.gate_first)
        return r["dx"], r["dz"], r["dweight"], None, None


def gated_rms_norm(x, z, weight: Optional[torch.Tensor] = None, eps: float = 1e-6, gate_first: bool = False):
    """``gated_norm`` with gradients in x, z and weight (no second derivatives)."""
    return _GatedNormFn.apply(x, z, weight, eps, gate_first)


class _AddNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, scale, post_weight, eps, residual_dtype):
        out, total = add_norm(x, residual, weight, scale, post_weight, eps, residual_dtype)
        ctx.save_for_backward(x, total, weight, scale, post_weight)
        ctx.eps, ctx.has_residual = eps, residual is not None
        ctx.set_materialize_grads(False)
        return out, total

    @staticmethod
    @_first_order
    def backward(ctx, dout, dtotal):
        x, total, weight, scale, post_weight = ctx.saved_tensors
        dout = torch.zeros_like(x) if dout is None else dout.contiguous()
        r = add_norm_bwd(x, total, dout, weight, None if dtotal is None else dtotal.contiguous(), scale, post_weight,
                         ctx.eps)
        return (r["dx"], r["dresidual"] if ctx.has_residual else None, r["dweight"], r["dscale"], r["dpost_weight"],
                None, None)


def add_rms_norm(x, residual: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                 scale: Optional[torch.Tensor] = None, post_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 residual_dtype=None):
    """``add_norm`` with gradients in x, residual, weight, scale and post_weight (no second
    derivatives).  Returns (out, total)."""
    return _AddNormFn.apply(x, residual, weight, scale, post_weight, eps, residual_dtype)
