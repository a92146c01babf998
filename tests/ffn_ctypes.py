"""The structures of awq_ffn.h for tests that call the C entry points directly."""
import ctypes

from bit_weight_only_w4a16_amd import awq

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_f32 = ctypes.c_float
_sz = ctypes.c_size_t


class RmsNormArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("x", "residual", "weight", "h_out", "y", "q", "scale")]
                + [(n, _i64) for n in ("tokens", "x_stride", "residual_stride", "h_stride", "y_stride", "q_stride")]
                + [("width", _i32), ("dtype", _i32), ("eps", _f32), ("reserved", _i32)])


class QuantI8Args(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("x", "inv_s_c", "q", "scale")]
                + [(n, _i64) for n in ("tokens", "x_stride", "q_stride")] + [("width", _i32), ("dtype", _i32)])


class GemmI8Args(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("q", "scale", "packed", "bias", "mul", "residual", "y", "ws")]
                + [("ws_bytes", _sz)] + [(n, _i64) for n in ("M", "N", "K", "q_stride")]
                + [("dtype", _i32), ("act", _i32)])


class MoeRouteArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("x", "w", "bias", "ids", "weights", "ws")] + [("ws_bytes", _sz)]
                + [(n, _i64) for n in ("tokens", "x_stride")]
                + [(n, _i32) for n in ("hidden", "experts", "k", "dtype", "score", "renormalize")]
                + [("scale", _f32), ("reserved", _i32)])


class MoeArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("x", "ids", "weights", "gate", "up", "down", "inv_in", "inv_down", "residual", "y",
                                    "ws")]
                + [("ws_bytes", _sz)]
                + [(n, _i64) for n in ("tokens", "x_stride", "residual_stride", "y_stride", "inv_in_stride",
                                       "inv_down_stride")]
                + [(n, _i32) for n in ("hidden", "ffn", "experts", "k", "group", "fmt", "act", "reserved")])


STRUCTS = {"awq_rms_norm_args": RmsNormArgs, "awq_quant_i8_args": QuantI8Args, "awq_gemm_i8_args": GemmI8Args,
           "awq_moe_route_args": MoeRouteArgs, "awq_moe_args": MoeArgs}
_SIGNATURES = {
    "awq_rms_norm": (ctypes.c_int, [_vp, _vp]),
    "awq_quant_i8": (ctypes.c_int, [_vp, _vp]),
    "awq_packed_i8_bytes": (_sz, [_i64, _i64]),
    "awq_pack_i8": (ctypes.c_int, [_vp, _vp, _i64, _i64, _i32, _vp, _sz, _vp]),
    "awq_gemm_i8_workspace_bytes": (_sz, [_i64] * 3),
    "awq_gemm_i8": (ctypes.c_int, [_vp, _vp]),
    "awq_moe_route_workspace_bytes": (_sz, [_i64, _i32, _i32]),
    "awq_moe_route": (ctypes.c_int, [_vp, _vp]),
    "awq_moe_workspace_bytes": (_sz, [_i64, _i32, _i32, _i32]),
    "awq_moe": (ctypes.c_int, [_vp, _vp]),
}


def lib() -> ctypes.CDLL:
    handle = awq.lib()
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(handle, name)
        fn.restype = res
        fn.argtypes = args
    return handle
