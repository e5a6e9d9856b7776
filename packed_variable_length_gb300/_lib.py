"""ctypes loader for libpvl.so: argument and return types of every C entry point.

The library is built in-tree (packed_variable_length_gb300/libpvl.so).  There
is no fallback: if the library is missing or fails to load, every call raises.
"""

from __future__ import annotations

import ctypes
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libpvl.so")

_c_int = ctypes.c_int
_c_size = ctypes.c_size_t
_c_float = ctypes.c_float
_p = ctypes.c_void_p

_i32 = ctypes.c_int32


class Rotary(ctypes.Structure):
    """pvl_rotary"""
    _fields_ = [("B", _i32), ("L", _i32), ("H", _i32), ("Hk", _i32), ("D", _i32), ("R", _i32), ("layout", _i32),
                ("axes", _i32), ("section_1", _i32), ("section_2", _i32), ("gain", _c_float), ("norm", _i32),
                ("eps", _c_float), ("turns", _p), ("positions", _p), ("q_weight", _p), ("k_weight", _p)]


class Heads(ctypes.Structure):
    """pvl_heads"""
    _fields_ = [("data", _p), ("stride_b", ctypes.c_int64), ("stride_l", ctypes.c_int64),
                ("stride_h", ctypes.c_int64)]


class Residual(ctypes.Structure):
    """pvl_residual"""
    _fields_ = [("B", _i32), ("N", _i32), ("D", _i32), ("S", _i32), ("stream_dtype", _i32), ("norm", _i32),
                ("post_norm", _i32), ("alpha", _c_float), ("eps", _c_float), ("gate", _p), ("shift", _p),
                ("scale", _p), ("weight", _p), ("bias", _p), ("post_weight", _p), ("mod_id", _p)]


class ResidualGrads(ctypes.Structure):
    """pvl_residual_grads"""
    _fields_ = [("dgate", _p), ("dshift", _p), ("dscale", _p), ("dweight", _p), ("dbias", _p),
                ("dpost_weight", _p)]


# name -> (restype, argtypes); mirrors include/pvl.h
SIGNATURES = {
    "pack_build_seq_ids": (_c_int, [_p, _p, _c_int, _c_int, _c_int, _c_int, _p, _p]),
    "tile_map_ws_bytes": (_c_size, [_c_int, _c_int, _c_int, _c_int]),
    "tile_map_layout": (_c_int, [_c_int, _c_int, _c_int, _c_int, _p]),
    "tile_map_build": (_c_int, [_p, _c_int, _c_int, _c_int, _c_int, _p, _c_size, _p]),
    "masked_attn_fwd": (_c_int, [_p, _p, _p, _p, _p, _c_int, _c_int, _c_int, _c_int, _c_float, _p, _p, _p]),
    "masked_attn_bwd_ws_bytes": (_c_size, [_c_int, _c_int, _c_int, _c_int]),
    "masked_attn_bwd": (_c_int, [_p, _p, _p, _p, _p, _p, _p, _p, _c_int, _c_int, _c_int, _c_int, _c_float,
                                 _p, _p, _p, _p, _c_size, _p]),
    "masked_attn_bwd_no_alloc": (_c_int, [_p, _p, _p, _p, _p, _p, _p, _p, _c_int, _c_int, _c_int, _c_int,
                                          _c_float, _p, _p, _p, _p]),
    "tile_map_ws_bytes_cross": (_c_size, [_c_int, _c_int, _c_int, _c_int, _c_int]),
    "tile_map_layout_cross": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int, _p]),
    "tile_map_build_cross": (_c_int, [_p, _p, _c_int, _c_int, _c_int, _c_int, _c_int, _p, _c_size, _p]),
    "masked_attn_fwd_cross": (_c_int, [_p, _p, _p, _p, _p, _p, _c_int, _c_int, _c_int, _c_int, _c_int, _c_float,
                                       _p, _p, _p]),
    "masked_attn_bwd_ws_bytes_cross": (_c_size, [_c_int, _c_int, _c_int, _c_int, _c_int]),
    "masked_attn_bwd_cross": (_c_int, [_p, _p, _p, _p, _p, _p, _p, _p, _p, _c_int, _c_int, _c_int, _c_int, _c_int,
                                       _c_float, _p, _p, _p, _p, _c_size, _p]),
    "adaln_fwd": (_c_int, [_p, _p, _p, _c_int, _c_int, _c_int, _c_float, _p, _p, _p, _p]),
    "adaln_bwd_ws_bytes": (_c_size, [_c_int, _c_int, _c_int]),
    "adaln_bwd": (_c_int, [_p, _p, _p, _c_int, _c_int, _c_int, _c_float, _p, _p, _p, _p, _c_size, _p]),
    "pack_build_positions": (_c_int, [_p, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _p, _p]),
    "pack_rotary_fwd": (_c_int, [_p, _p, _p, _p, _p, _p]),
    "pack_rotary_bwd_ws_bytes": (_c_size, [_p]),
    "pack_rotary_bwd": (_c_int, [_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _c_size, _p]),
    "adaln_residual_fwd": (_c_int, [_p, _p, _p, _p, _p, _p]),
    "adaln_residual_bwd_ws_bytes": (_c_size, [_c_int, _c_int, _c_int, _c_int]),
    "adaln_residual_bwd": (_c_int, [_p, _p, _p, _p, _p, _c_int, _p, _p, _p, _p, _c_size, _p]),
    "masked_mse_ws_bytes": (_c_size, [_c_int, _c_int, _c_int]),
    "masked_mse_loss": (_c_int, [_p, _p, _p, _c_int, _c_int, _c_int, _p, _p, _c_float, _p, _c_size, _p]),
    "masked_mse_loss_bwd": (_c_int, [_p, _p, _p, _c_int, _c_int, _c_int, _p, _p, _p, _c_size, _p]),
    "pvl_selftest_wait_timeout": (_c_int, [ctypes.c_uint64, ctypes.c_uint64, _p, _p]),
    "pvl_set_attn_wait_timeout_ns": (_c_int, [ctypes.c_uint64]),
    "pvl_mark_next_bwd_main": (_c_int, [_p, _p]),
    "pvl_device_error": (_c_int, [_p]),
    "pvl_device_error_detail": (_c_int, [_p, _p]),
    "pvl_last_error_message": (ctypes.c_char_p, []),
    "pvl_version": (_c_int, []),
}

_lib = None


def load() -> ctypes.CDLL:
    """Loads libpvl.so once; raises RuntimeError when it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m packed_variable_length_gb300.build` "
                "(or __graft_entry__.build()); there is no non-CUDA fallback")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib
