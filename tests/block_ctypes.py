"""The structures of awq_block.h for tests that call the C entry points directly."""
import ctypes

from bit_weight_only_w4a16_amd import awq

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_f32 = ctypes.c_float


class RopeArgs(ctypes.Structure):
    """awq_rope_args of awq_block.h."""
    _fields_ = ([(n, _vp) for n in ("q", "q_out", "k", "k_out", "v", "k_cache", "v_cache", "positions",
                                    "inv_freq", "slots")]
                + [(n, _i64) for n in ("tokens", "q_token", "q_head", "qo_token", "qo_head", "k_token", "k_head",
                                       "ko_token", "ko_head", "v_token", "v_head", "cache_page", "cache_head",
                                       "cache_slot", "pages")]
                + [(n, _i32) for n in ("page_size", "q_heads", "kv_heads", "head_dim", "rot_dim", "dtype",
                                       "interleaved", "inverse")]
                + [("scale", _f32), ("reserved", _i32)])


class AttnPromptArgs(ctypes.Structure):
    """awq_attn_prompt_args of awq_block.h."""
    _fields_ = ([(n, _vp) for n in ("q", "k", "v", "out", "cu")]
                + [(n, _i64) for n in ("tokens", "seqs", "q_token", "q_head", "k_token", "k_head", "v_token",
                                       "v_head", "o_token", "o_head")]
                + [(n, _i32) for n in ("q_heads", "kv_heads", "head_dim", "dtype")]
                + [("scale", _f32), ("reserved", _i32)])


class AttnTreeArgs(ctypes.Structure):
    """awq_attn_tree_args of awq_block.h."""
    _fields_ = ([(n, _vp) for n in ("q", "k_cache", "v_cache", "out", "block_table", "ctx_lens", "cu_q", "mask",
                                    "ws")]
                + [("ws_bytes", ctypes.c_size_t)]
                + [(n, _i64) for n in ("tokens", "seqs", "table_width", "pages", "q_token", "q_head", "o_token",
                                       "o_head", "cache_page", "cache_head", "cache_slot")]
                + [(n, _i32) for n in ("page_size", "max_q", "q_heads", "kv_heads", "head_dim", "dtype")]
                + [("scale", _f32), ("reserved", _i32)])


class Epilogue(ctypes.Structure):
    """awq_epilogue of awq_block.h."""
    _fields_ = [("bias", _vp), ("mul", _vp), ("residual", _vp), ("act", _i32), ("reserved", _i32)]


_SIGNATURES = {
    "awq_gemm_fused": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _i64, _i32, _i32, _vp, _vp, _vp, ctypes.c_size_t,
                                      _vp]),
    "awq_rope": (ctypes.c_int, [_vp, _vp]),
    "awq_attn_prompt": (ctypes.c_int, [_vp, _vp]),
    "awq_attn_tree_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, _i64, _i32, _i32, _i32, _i32, _i32]),
    "awq_attn_tree": (ctypes.c_int, [_vp, _vp]),
}

def lib() -> ctypes.CDLL:
    handle = awq.lib()
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(handle, name)
        fn.restype = res
        fn.argtypes = args
    return handle
