"""ctypes handle on the in-tree CUDA library ``libgla.so`` (C ABI in include/gla.h).

Loading never falls back to anything: if the library is missing or cannot be
loaded the error says so and names the build command.
"""

from __future__ import annotations

import ctypes
import os
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgla.so")

# Status codes (enum gla_status in include/gla.h).
GLA_OK = 0
GLA_ERR_ARG = 1
GLA_ERR_SHAPE = 2
GLA_ERR_DEVICE = 3
GLA_ERR_LAUNCH = 4
GLA_ERR_TIMEOUT = 5
GLA_ERR_ALLOC = 6
GLA_ERR_SCRATCH = 7

EXPORTED = ("gla_chunk_fwd", "gla_chunk_fwd_ex", "gla_chunk_fwd_plan", "gla_chunk_fwd_noalloc",
            "gla_chunk_fwd_debug",
            "gla_chunk_fwd_host", "gla_chunk_fwd_varlen", "gla_chunk_fwd_varlen_ex",
            "gla_chunk_fwd_varlen_plan", "gla_chunk_bwd", "gla_chunk_bwd_ex",
            "gla_chunk_bwd_plan", "gla_chunk_bwd_varlen", "gla_chunk_bwd_varlen_ex",
            "gla_gdn_fwd", "gla_gdn_chunk_fwd", "gla_recurrent_step",
            "gla_scan_fwd", "gla_scan_bwd", "gla_scan_fwd_varlen", "gla_scan_bwd_varlen",
            "gla_scan_step", "gla_qk_norm_rope_fwd", "gla_qk_norm_rope_bwd",
            "gla_qk_norm_rope_bwd_scratch", "gla_headgate_fwd_varlen",
            "gla_headgate_fwd_varlen_scratch", "gla_headgate_step", "gla_group_norm_act_fwd",
            "gla_group_norm_act_bwd", "gla_group_norm_act_bwd_scratch", "gla_status_string",
            "gla_last_device_status", "gla_version")


# Element types (enum gla_dtype) and norms (enum gla_norm).
GLA_BF16 = 0
GLA_F32 = 1
GLA_NORM_RMS = 0
GLA_NORM_L2 = 1
GLA_NORM_LAYER = 2
# Activations (enum gla_activation).
GLA_ACT_SILU = 0
GLA_ACT_SIGMOID = 1
# Tokens of one block of a scan's checkpoints (GLA_SCAN_BLOCK).
SCAN_BLOCK = 64


class GlaChunkOptions(ctypes.Structure):
    _fields_ = [("segments", ctypes.c_int), ("dv_tile", ctypes.c_int),
                ("force_exact", ctypes.c_int), ("cta_pair", ctypes.c_int),
                ("gate_per_head", ctypes.c_int), ("reserved", ctypes.c_int * 3)]


class GlaChunkDebug(ctypes.Structure):
    """gla_chunk_debug (include/gla.h): test instrumentation of the chunked forward."""
    _fields_ = [("gamma", ctypes.c_void_p), ("block_len", ctypes.c_void_p),
                ("wait_limit_us", ctypes.c_uint), ("withhold_v", ctypes.c_int)]


class GlaQkLayout(ctypes.Structure):
    """gla_qk_layout (include/gla.h): strides of q, k and the positions, in elements."""
    _fields_ = [(n, ctypes.c_longlong) for n in ("q_sb", "q_st", "q_sh", "k_sb", "k_st", "k_sh",
                                                 "pos_sb")]


class GlaQkOptions(ctypes.Structure):
    """gla_qk_options (include/gla.h)."""
    _fields_ = [("dtype", ctypes.c_int), ("norm", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("eps", ctypes.c_float)]


class GlaHeadgateLayout(ctypes.Structure):
    """gla_headgate_layout (include/gla.h): strides of q, k, v and log_alpha, in elements."""
    _fields_ = [(n, ctypes.c_longlong) for n in ("q_st", "q_sh", "k_st", "k_sh", "v_st", "v_sh",
                                                 "a_st", "a_sh")]


class GlaNormActLayout(ctypes.Structure):
    """gla_norm_act_layout (include/gla.h): strides of x, gate and grad_x, in elements."""
    _fields_ = [(n, ctypes.c_longlong) for n in ("x_sb", "x_st", "x_sh", "g_sb", "g_st", "g_sh",
                                                 "dx_sb", "dx_st", "dx_sh")]


class GlaNormActOptions(ctypes.Structure):
    """gla_norm_act_options (include/gla.h)."""
    _fields_ = [("dtype", ctypes.c_int), ("norm", ctypes.c_int), ("activation", ctypes.c_int),
                ("per_channel", ctypes.c_int), ("eps", ctypes.c_float)]


class GlaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


_lock = threading.Lock()
_lib: ctypes.CDLL | None = None


def _bind(lib: ctypes.CDLL) -> ctypes.CDLL:
    vp, fp, i, f = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.gla_chunk_fwd.argtypes = [vp, vp, vp, fp, f, fp, vp, fp, i, i, i, i, i, vp]
    lib.gla_chunk_fwd.restype = i
    lib.gla_chunk_fwd_ex.argtypes = [vp, vp, vp, fp, f, fp, vp, fp, i, i, i, i, i,
                                     ctypes.POINTER(GlaChunkOptions), vp]
    lib.gla_chunk_fwd_ex.restype = i
    lib.gla_chunk_fwd_noalloc.argtypes = [vp, vp, vp, fp, f, fp, vp, fp, i, i, i, i, i,
                                          ctypes.POINTER(GlaChunkOptions), vp]
    lib.gla_chunk_fwd_noalloc.restype = i
    lib.gla_chunk_fwd_debug.argtypes = [vp, vp, vp, fp, f, fp, vp, fp, i, i, i, i, i,
                                        ctypes.POINTER(GlaChunkOptions),
                                        ctypes.POINTER(GlaChunkDebug), vp]
    lib.gla_chunk_fwd_debug.restype = i
    lib.gla_chunk_fwd_host.argtypes = [vp, vp, vp, fp, f, fp, vp, fp, i, i, i, i, i, vp]
    lib.gla_chunk_fwd_host.restype = i
    ip = ctypes.POINTER(ctypes.c_int)
    lib.gla_chunk_fwd_varlen_plan.argtypes = [ip, i, i, i, i, i, ctypes.POINTER(GlaChunkOptions),
                                              ip, ip, ip, ctypes.POINTER(ctypes.c_ulong)]
    lib.gla_chunk_fwd_varlen_plan.restype = i
    lib.gla_chunk_fwd_varlen.argtypes = [vp, vp, vp, fp, f, fp, vp, fp, ip, i, i, i, i, i, vp]
    lib.gla_chunk_fwd_varlen.restype = i
    lib.gla_chunk_fwd_varlen_ex.argtypes = [vp, vp, vp, fp, f, fp, vp, fp, ip, i, i, i, i, i,
                                            ctypes.POINTER(GlaChunkOptions), vp]
    lib.gla_chunk_fwd_varlen_ex.restype = i
    lib.gla_chunk_fwd_plan.argtypes = [i, i, i, i, i, ctypes.POINTER(GlaChunkOptions), ip, ip, ip,
                                       ctypes.POINTER(ctypes.c_ulong)]
    lib.gla_chunk_fwd_plan.restype = i
    bwd = [vp, vp, vp, fp, f, fp, vp, fp, vp, vp, vp, fp, fp, i, i, i, i, i]
    lib.gla_chunk_bwd.argtypes = bwd + [vp]
    lib.gla_chunk_bwd.restype = i
    lib.gla_chunk_bwd_ex.argtypes = bwd + [ctypes.POINTER(GlaChunkOptions), vp]
    lib.gla_chunk_bwd_ex.restype = i
    lib.gla_chunk_bwd_plan.argtypes = [i, i, i, i, i, ip, ip, ctypes.POINTER(ctypes.c_ulong)]
    bwdv = [vp, vp, vp, fp, f, fp, vp, fp, vp, vp, vp, fp, fp, ip, i, i, i, i, i]
    lib.gla_chunk_bwd_varlen.argtypes = bwdv + [vp]
    lib.gla_chunk_bwd_varlen.restype = i
    lib.gla_chunk_bwd_varlen_ex.argtypes = bwdv + [ctypes.POINTER(GlaChunkOptions), vp]
    lib.gla_chunk_bwd_varlen_ex.restype = i
    lib.gla_chunk_bwd_plan.restype = i
    lib.gla_gdn_fwd.argtypes = [vp, vp, vp, fp, fp, f, fp, vp, fp, i, i, i, i, i, vp]
    lib.gla_gdn_fwd.restype = i
    lib.gla_gdn_chunk_fwd.argtypes = [vp, vp, vp, fp, fp, f, fp, vp, fp, i, i, i, i, i, vp]
    lib.gla_gdn_chunk_fwd.restype = i
    lib.gla_recurrent_step.argtypes = [vp, vp, vp, fp, f, fp, vp, i, i, i, i, vp]
    lib.gla_recurrent_step.restype = i
    lib.gla_scan_fwd.argtypes = [vp, fp, fp, vp, fp, fp, i, i, i, i, vp]
    lib.gla_scan_fwd.restype = i
    lib.gla_scan_bwd.argtypes = [vp, fp, fp, vp, fp, vp, fp, fp, i, i, i, i, vp]
    lib.gla_scan_bwd.restype = i
    lib.gla_scan_fwd_varlen.argtypes = [vp, fp, fp, vp, fp, fp, ip, i, i, i, i, i, vp]
    lib.gla_scan_fwd_varlen.restype = i
    lib.gla_scan_bwd_varlen.argtypes = [vp, fp, fp, vp, fp, vp, fp, fp, ip, i, i, i, i, i, vp]
    lib.gla_scan_bwd_varlen.restype = i
    lib.gla_scan_step.argtypes = [vp, fp, fp, vp, i, i, i, vp]
    lib.gla_scan_step.restype = i
    qk = [i, i, i, i, i, i, ctypes.POINTER(GlaQkLayout), ctypes.POINTER(GlaQkOptions)]
    lib.gla_qk_norm_rope_fwd.argtypes = [vp, vp, fp, fp, vp, vp, vp, vp] + qk + [vp]
    lib.gla_qk_norm_rope_fwd.restype = i
    lib.gla_qk_norm_rope_bwd.argtypes = ([vp, vp, fp, fp, vp, vp, vp, vp, vp, vp, fp, fp] + qk +
                                         [vp, ctypes.c_ulong, vp])
    lib.gla_qk_norm_rope_bwd.restype = i
    lib.gla_qk_norm_rope_bwd_scratch.argtypes = [i]
    lib.gla_qk_norm_rope_bwd_scratch.restype = ctypes.c_ulong
    ul, lay = ctypes.c_ulong, ctypes.POINTER(GlaHeadgateLayout)
    lib.gla_headgate_fwd_varlen_scratch.argtypes = [ip, i, i, i, i]
    lib.gla_headgate_fwd_varlen_scratch.restype = ul
    lib.gla_headgate_fwd_varlen.argtypes = [vp, vp, vp, fp, f, fp, vp, fp, ip, i, i, i, i, i, i,
                                            lay, vp, ul, vp]
    lib.gla_headgate_fwd_varlen.restype = i
    lib.gla_headgate_step.argtypes = [vp, vp, vp, fp, f, fp, vp, vp, i, i, i, i, i, i, lay, i, vp]
    lib.gla_headgate_step.restype = i
    norm = [i, i, i, i, ctypes.POINTER(GlaNormActLayout), ctypes.POINTER(GlaNormActOptions)]
    lib.gla_group_norm_act_fwd.argtypes = [vp, vp, fp, fp, vp] + norm + [vp]
    lib.gla_group_norm_act_fwd.restype = i
    lib.gla_group_norm_act_bwd_scratch.argtypes = [i, i, i, i]
    lib.gla_group_norm_act_bwd_scratch.restype = ul
    lib.gla_group_norm_act_bwd.argtypes = [vp, vp, fp, fp, vp, vp, vp, fp, fp] + norm + [vp, ul, vp]
    lib.gla_group_norm_act_bwd.restype = i
    lib.gla_status_string.argtypes = [i]
    lib.gla_status_string.restype = ctypes.c_char_p
    lib.gla_last_device_status.argtypes = [vp]
    lib.gla_last_device_status.restype = i
    lib.gla_version.argtypes = []
    lib.gla_version.restype = i
    return lib


def lib() -> ctypes.CDLL:
    """The loaded library (loaded once per process)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(
                    f"{LIB_PATH} is missing: build it with "
                    "`python -m chunkwise_linear_rnn_gb300.build` (needs nvcc for sm_103a)")
            _lib = _bind(ctypes.CDLL(LIB_PATH))
        return _lib


def status_string(status: int) -> str:
    return lib().gla_status_string(int(status)).decode()


def check(status: int, what: str) -> None:
    if status != GLA_OK:
        raise GlaError(status, what)
