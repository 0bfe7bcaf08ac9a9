"""ctypes binding of ``libmamba_ssd.so`` (the C ABI in ``include/ssd.h``).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI.  Torch tensors serve as device buffers and torch's
current stream as the launch stream.  There is no fallback: when the library
is missing or the tensors are not on the GPU, calls raise.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmamba_ssd.so")

SSD_OK = 0
STATUS_NAMES = {0: "SSD_OK", 1: "SSD_ERR_NULL", 2: "SSD_ERR_SHAPE", 3: "SSD_ERR_DTYPE",
                4: "SSD_ERR_UNSUPPORTED", 5: "SSD_ERR_WORKSPACE", 6: "SSD_ERR_ALIGN", 7: "SSD_ERR_HIP",
                8: "SSD_ERR_SCRATCH"}
SSD_F32, SSD_BF16 = 0, 1
SSD_MMA_BF16, SSD_MMA_F32 = 0, 1
MMA = {"bf16": SSD_MMA_BF16, "f32": SSD_MMA_F32}


class SSDShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int64),
                ("headdim", ctypes.c_int64), ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("chunk", ctypes.c_int64)]

    @classmethod
    def make(cls, batch, seqlen, nheads, headdim, dstate, ngroups, chunk) -> "SSDShape":
        return cls(batch, seqlen, nheads, headdim, dstate, ngroups, chunk)

    def as_dict(self):
        return {k: getattr(self, k) for k, _ in self._fields_}


class SSDConvShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("channels", ctypes.c_int64),
                ("width", ctypes.c_int64)]


class SSDScanShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("channels", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64)]


class SSDScanRows(ctypes.Structure):
    _fields_ = [("u", ctypes.c_int64), ("dt", ctypes.c_int64), ("Bm", ctypes.c_int64), ("Cm", ctypes.c_int64),
                ("z", ctypes.c_int64)]


class SSDDeltaShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int64),
                ("headdim", ctypes.c_int64), ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64)]


class SSDDeltaRows(ctypes.Structure):
    _fields_ = [("q", ctypes.c_int64), ("k", ctypes.c_int64), ("v", ctypes.c_int64), ("dt", ctypes.c_int64),
                ("beta", ctypes.c_int64)]


SSD_DELTA_SOFTPLUS, SSD_DELTA_SIGMOID, SSD_DELTA_QK_NORM, SSD_DELTA_MMA_F32 = 1, 2, 4, 32
SSD_GROUP_RMS, SSD_GROUP_GATE_FIRST, SSD_GROUP_SILU, SSD_GROUP_SHARED = 1, 2, 4, 8

_P = ctypes.c_void_p
_S = ctypes.POINTER(SSDShape)
_E = ctypes.c_int  # enums
_I, _F, _Z = ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_CS, _SS, _SR = ctypes.POINTER(SSDConvShape), ctypes.POINTER(SSDScanShape), ctypes.POINTER(SSDScanRows)
_SCAN_IN = [_SS, _SR, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int, _E]  # shape .. in
_DS, _DR = ctypes.POINTER(SSDDeltaShape), ctypes.POINTER(SSDDeltaRows)
_DELTA_IN = [_DS, _DR, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int, _F, _E]  # shape .. in

_SIGNATURES = {
    "ssd_chunk_cumsum": (ctypes.c_int, [_S, _P, _P, _P, _P, _P]),
    "ssd_chunk_state": (ctypes.c_int, [_S, _P, _P, _E, _P, _P, _P, _E, _E, _P]),
    "ssd_chunk_cumsum_state": (ctypes.c_int, [_S, _P, _P, _E, _P, _P, _P, _P, _P, _E, _E, _P]),
    "ssd_state_passing": (ctypes.c_int, [_S, _P, _E, _P, _E, _P, _P, _P, _P]),
    "ssd_chunk_scan": (ctypes.c_int, [_S, _P, _P, _P, _E, _P, _P, _P, _E, _P, _P, _E, _E, _P]),
    "ssd_chunk_state_passing": (ctypes.c_int, [_S, _P, _P, _E, _P, _P, _P, _P, _E, _P, _E, _P]),
    "ssd_decode_step": (ctypes.c_int, [_S, _P, _P, _P, _P, _P, _P, _E, _P, _P, _E, _P]),
    "ssd_workspace_bytes": (ctypes.c_size_t, [_S]),
    "ssd_workspace_bytes_varlen": (ctypes.c_size_t, [_S]),
    "ssd_forward_varlen": (ctypes.c_int, [_S, _P, _P, _P, _P, _P, _P, _E, _P, _P, _P, _E, _P, ctypes.c_int64, _P, _P,
                                          _P, ctypes.c_size_t, _E, _P]),
    "ssd_forward": (ctypes.c_int, [_S, _P, _P, _P, _P, _P, _P, _E, _P, _P, _E, _P, _P, ctypes.c_size_t, _E, _P]),
    "ssd_forward_noalloc": (ctypes.c_int, [_S, _P, _P, _P, _P, _P, _P, _E, _P, _P, _E, _P, _E, _P]),
    "ssd_backward": (ctypes.c_int, [_S, _P, _P, _P, _P, _P, _P, _E, _P, _P, _E, _P, _P, _P, _P, _P, _P, _P, _P,
                                    _P, ctypes.c_size_t, _E, _P]),
    "ssd_backward_workspace_bytes": (ctypes.c_size_t, [_S]),
    "ssd_causal_conv": (ctypes.c_int, [_CS, _P, _I, _P, _P, _E, ctypes.c_int, _P, _P, _P, _P, _I, _P, _P, _P]),
    "ssd_causal_conv_step": (ctypes.c_int, [_CS, _P, _I, _P, _P, _P, _E, ctypes.c_int, _P, _P, _P]),
    "ssd_causal_conv_backward": (ctypes.c_int, [_CS, _P, _I, _P, _P, _E, ctypes.c_int, _P, _P, _P, _P, _P, _I, _P, _P,
                                                _P, _P, _Z, _P]),
    "ssd_causal_conv_backward_workspace_bytes": (_Z, [_CS]),
    "ssd_selective_scan": (ctypes.c_int, _SCAN_IN + [_P, _P, _P, _P, _I, _P, _P, _P, _Z, _P]),
    "ssd_selective_scan_workspace_bytes": (_Z, [_SS]),
    "ssd_selective_step": (ctypes.c_int, _SCAN_IN + [_P, _P, _P, _P]),
    "ssd_selective_scan_backward": (ctypes.c_int, _SCAN_IN + [_P, _P, _P, _P, _SR] + [_P] * 9 + [_P, _Z, _P]),
    "ssd_selective_scan_backward_workspace_bytes": (_Z, [_SS]),
    "ssd_layer_norm": (ctypes.c_int, [_I, _I, _P, _E, _P, _E, _P, _P, _F, ctypes.c_int, _P, _P, _P, _P, _P]),
    "ssd_layer_norm_backward": (ctypes.c_int, [_I, _I, _P, _E, _P, _E, _P, _P, _P, ctypes.c_int, _P, _P, _P, _P, _P, _P,
                                               _Z, _P]),
    "ssd_layer_norm_backward_workspace_bytes": (_Z, [_I, _I]),
    "ssd_delta_rule": (ctypes.c_int, _DELTA_IN + [_P, _P, _P, _P, _I, _P, _P, _P, _Z, _P]),
    "ssd_delta_rule_workspace_bytes": (_Z, [_DS]),
    "ssd_delta_rule_backward": (ctypes.c_int, _DELTA_IN + [_P, _P, _P, _P, _DR] + [_P] * 8 + [_P, _Z, _P]),
    "ssd_delta_rule_backward_workspace_bytes": (_Z, [_DS]),
    "ssd_delta_step": (ctypes.c_int, _DELTA_IN + [_P, _P, _P, _P]),
    "ssd_group_norm": (ctypes.c_int, [_I, _I, _I, _P, _E, _P, _I, _P, _P, _F, ctypes.c_int, _P, _P, _P, _P]),
    "ssd_group_norm_backward": (ctypes.c_int, [_I, _I, _I, _P, _E, _P, _P, _P, _I, _P, _P, _P, _P, _P, ctypes.c_int,
                                               _P, _P, _I, _P, _P, _P, _Z, _P]),
    "ssd_group_norm_backward_workspace_bytes": (_Z, [_I, _I, _I]),
    "ssd_pack8": (ctypes.c_int, [_I, _I, _P, _I, _E, _P, _P, _P]),
    "ssd_unpack8": (ctypes.c_int, [_I, _I, _P, _P, _P, _I, _E, _P]),
    "ssd_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "ssd_abi_version": (ctypes.c_int, []),
}

_LIB: Optional[ctypes.CDLL] = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the HIP library (raises if it has not been built)."""
    global _LIB
    if _LIB is not None and path == LIB_PATH:
        return _LIB
    if not os.path.exists(path):
        raise RuntimeError(f"HIP library not built: {path}; run `python -m mamba_ssd_scan_chunk_amd.build`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path == LIB_PATH:
        _LIB = lib
    return lib


class SSDError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(msg)
        self.code = code


def check(code: int) -> None:
    if code != SSD_OK:
        lib = load_library()
        raise SSDError(code, lib.ssd_status_string(code).decode())
