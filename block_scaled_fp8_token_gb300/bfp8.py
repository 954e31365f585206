"""Python binding of libbfp8: the C ABI of include/bfp8.h, name for name.

Argument marshalling only. Every function takes torch tensors (device memory
and shapes come from them), passes raw pointers, sizes and the current CUDA
stream to the library, and raises Bfp8Error on a non-zero status. Nothing
here computes. If libbfp8.so is missing, importing this module raises.
Nothing falls back to another implementation.
"""

from __future__ import annotations

import ctypes
import os
import struct
from pathlib import Path

import torch

_LIB_PATH = Path(__file__).resolve().parent / "libbfp8.so"

if not _LIB_PATH.exists():
    raise ImportError(
        f"{_LIB_PATH} is missing: build it with "
        "`python -m block_scaled_fp8_token_gb300.build` (needs nvcc). "
        "There is no fallback implementation.")

_lib = ctypes.CDLL(os.fspath(_LIB_PATH))

# ---- enums (include/bfp8.h) ------------------------------------------------
BFP8_OK = 0
BFP8_ERR_CUDA = 14
STATUS_NAMES = {
    0: "OK", 1: "INVALID_ARG", 2: "E5M2", 3: "NO_SCALE", 4: "ROW_SCALE",
    5: "AMBIGUOUS_SCALE", 6: "GRID_TRANSPOSED", 7: "GRID_SHAPE", 8: "SCALE_DTYPE",
    9: "BLOCK_SIZE", 10: "QUANT_METHOD", 11: "GROUP", 12: "NOT_FP8",
    13: "UNSUPPORTED", 14: "CUDA", 15: "TIMEOUT",
}
BFP8_DT_NONE, BFP8_DT_E4M3, BFP8_DT_E5M2, BFP8_DT_BF16, BFP8_DT_F16, BFP8_DT_F32 = range(6)
BFP8_MAX_MEMBERS = 8


class Bfp8Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {bfp8_status_string(status)} ({status})")


class bfp8_weight_desc(ctypes.Structure):
    _fields_ = [
        ("weight_dtype", ctypes.c_int32),
        ("weight_rank", ctypes.c_int32),
        ("weight_shape", ctypes.c_int64 * 2),
        ("scale_dtype", ctypes.c_int32),
        ("scale_rank", ctypes.c_int32),
        ("scale_shape", ctypes.c_int64 * 2),
        ("has_row_scale", ctypes.c_int32),
        ("declared_quant_fp8", ctypes.c_int32),
        ("declared_block", ctypes.c_int32 * 2),
        ("n_members", ctypes.c_int32),
        ("member_rows", ctypes.POINTER(ctypes.c_int64)),
        ("tensor_scale_dtype", ctypes.c_int32),
    ]


class bfp8_members(ctypes.Structure):
    _fields_ = [("n_members", ctypes.c_int32), ("member_rows", ctypes.POINTER(ctypes.c_int64))]


class bfp8_kv_cache(ctypes.Structure):
    _fields_ = [
        ("k_e4m3", ctypes.c_void_p), ("v_e4m3", ctypes.c_void_p),
        ("k_exp", ctypes.c_void_p), ("v_exp", ctypes.c_void_p),
        ("n_pages", ctypes.c_int64),
        ("page_size", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("k_stride_page", ctypes.c_int64), ("k_stride_head", ctypes.c_int64),
        ("k_stride_token", ctypes.c_int64),
        ("v_stride_page", ctypes.c_int64), ("v_stride_head", ctypes.c_int64),
        ("v_stride_token", ctypes.c_int64),
        ("exp_stride_page", ctypes.c_int64), ("exp_stride_head", ctypes.c_int64),
    ]


class bfp8_kv_attention_args(ctypes.Structure):
    _fields_ = [
        ("q_bf16", ctypes.c_void_p), ("q_stride_token", ctypes.c_int64),
        ("q_stride_head", ctypes.c_int64),
        ("out_bf16", ctypes.c_void_p), ("out_stride_token", ctypes.c_int64),
        ("out_stride_head", ctypes.c_int64),
        ("lse", ctypes.c_void_p), ("lse_stride_token", ctypes.c_int64),
        ("block_table", ctypes.c_void_p), ("ld_table", ctypes.c_int64),
        ("max_blocks", ctypes.c_int64),
        ("q_offsets", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
        ("batch", ctypes.c_int64), ("tokens", ctypes.c_int64), ("max_q_len", ctypes.c_int64),
        ("n_heads", ctypes.c_int64),
        ("softmax_scale", ctypes.c_float), ("window", ctypes.c_int32),
        ("workspace", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t),
    ]


class bfp8_norm_args(ctypes.Structure):
    _fields_ = [
        ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64),
        ("residual", ctypes.c_void_p), ("ld_residual", ctypes.c_int64),
        ("gate", ctypes.c_void_p), ("ld_gate", ctypes.c_int64),
        ("w_post", ctypes.c_void_p), ("w_pre", ctypes.c_void_p), ("w_dtype", ctypes.c_int32),
        ("weight_offset", ctypes.c_float), ("residual_scale", ctypes.c_float),
        ("eps", ctypes.c_float),
        ("residual_out", ctypes.c_void_p), ("ld_residual_out", ctypes.c_int64),
        ("norm_out", ctypes.c_void_p), ("ld_norm_out", ctypes.c_int64),
        ("q_e4m3", ctypes.c_void_p), ("ldq", ctypes.c_int64),
        ("scales", ctypes.c_void_p), ("s_stride_m", ctypes.c_int64),
        ("s_stride_kb", ctypes.c_int64),
    ]


class bfp8_causal_conv_args(ctypes.Structure):
    _fields_ = [
        ("x_bf16", ctypes.c_void_p), ("x_stride_token", ctypes.c_int64),
        ("out_bf16", ctypes.c_void_p), ("out_stride_token", ctypes.c_int64),
        ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("w_dtype", ctypes.c_int32),
        ("width", ctypes.c_int32), ("silu", ctypes.c_int32), ("state_bf16", ctypes.c_void_p),
        ("state_stride_slot", ctypes.c_int64), ("state_stride_row", ctypes.c_int64),
        ("n_slots", ctypes.c_int64), ("slots_in", ctypes.c_void_p), ("slots_out", ctypes.c_void_p),
        ("q_offsets", ctypes.c_void_p), ("batch", ctypes.c_int64), ("tokens", ctypes.c_int64),
        ("channels", ctypes.c_int64),
    ]


class bfp8_delta_rule_args(ctypes.Structure):
    _fields_ = [
        ("q_bf16", ctypes.c_void_p), ("q_stride_token", ctypes.c_int64),
        ("q_stride_head", ctypes.c_int64), ("k_bf16", ctypes.c_void_p),
        ("k_stride_token", ctypes.c_int64), ("k_stride_head", ctypes.c_int64),
        ("v_bf16", ctypes.c_void_p), ("v_stride_token", ctypes.c_int64),
        ("v_stride_head", ctypes.c_int64), ("a_bf16", ctypes.c_void_p),
        ("a_stride_token", ctypes.c_int64), ("b_bf16", ctypes.c_void_p),
        ("b_stride_token", ctypes.c_int64), ("a_log", ctypes.c_void_p),
        ("dt_bias", ctypes.c_void_p), ("state", ctypes.c_void_p),
        ("state_stride_slot", ctypes.c_int64), ("state_stride_head", ctypes.c_int64),
        ("n_slots", ctypes.c_int64), ("slots_in", ctypes.c_void_p), ("slots_out", ctypes.c_void_p),
        ("q_offsets", ctypes.c_void_p), ("out_bf16", ctypes.c_void_p),
        ("out_stride_token", ctypes.c_int64), ("out_stride_head", ctypes.c_int64),
        ("batch", ctypes.c_int64), ("tokens", ctypes.c_int64), ("max_q_len", ctypes.c_int64),
        ("qk_heads", ctypes.c_int64), ("v_heads", ctypes.c_int64), ("head_dim", ctypes.c_int32),
        ("scale", ctypes.c_float), ("eps", ctypes.c_float), ("workspace", ctypes.c_void_p),
        ("ws_bytes", ctypes.c_size_t),
    ]


class bfp8_gated_norm_args(ctypes.Structure):
    _fields_ = [
        ("x_bf16", ctypes.c_void_p), ("x_stride_token", ctypes.c_int64),
        ("x_stride_head", ctypes.c_int64), ("gate_bf16", ctypes.c_void_p),
        ("gate_stride_token", ctypes.c_int64), ("gate_stride_head", ctypes.c_int64),
        ("weight", ctypes.c_void_p), ("w_dtype", ctypes.c_int32), ("gate_act", ctypes.c_int32),
        ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float), ("out_bf16", ctypes.c_void_p),
        ("out_stride_token", ctypes.c_int64), ("out_stride_head", ctypes.c_int64),
        ("q_e4m3", ctypes.c_void_p), ("ldq", ctypes.c_int64), ("scales", ctypes.c_void_p),
        ("s_stride_m", ctypes.c_int64), ("s_stride_kb", ctypes.c_int64),
        ("tokens", ctypes.c_int64), ("heads", ctypes.c_int64), ("head_dim", ctypes.c_int32),
    ]


class bfp8_rotary_args(ctypes.Structure):
    _fields_ = [
        ("q_bf16", ctypes.c_void_p), ("q_stride_token", ctypes.c_int64),
        ("q_stride_head", ctypes.c_int64), ("q_out_bf16", ctypes.c_void_p),
        ("q_out_stride_token", ctypes.c_int64), ("q_out_stride_head", ctypes.c_int64),
        ("k_bf16", ctypes.c_void_p), ("k_stride_token", ctypes.c_int64),
        ("k_stride_head", ctypes.c_int64), ("k_out_bf16", ctypes.c_void_p),
        ("k_out_stride_token", ctypes.c_int64), ("k_out_stride_head", ctypes.c_int64),
        ("positions", ctypes.c_void_p), ("ld_positions", ctypes.c_int64),
        ("inv_freq", ctypes.c_void_p), ("q_weight", ctypes.c_void_p),
        ("k_weight", ctypes.c_void_p), ("w_dtype", ctypes.c_int32), ("eps", ctypes.c_float),
        ("weight_offset", ctypes.c_float), ("factor", ctypes.c_float), ("tokens", ctypes.c_int64),
        ("q_heads", ctypes.c_int64), ("k_heads", ctypes.c_int64), ("head_dim", ctypes.c_int32),
        ("rotary_dim", ctypes.c_int32), ("axes", ctypes.c_int32), ("sections", ctypes.c_int32 * 4),
        ("interleaved", ctypes.c_int32), ("adjacent", ctypes.c_int32),
    ]


_vp, _i64, _i32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
_SIGS = {
    "bfp8_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "bfp8_validate_grid": (ctypes.c_int, [ctypes.POINTER(bfp8_weight_desc), ctypes.c_char_p, _sz]),
    "bfp8_act_quant_group": (ctypes.c_int, [_vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _vp]),
    "bfp8_silu_mul_act_quant": (ctypes.c_int, [_vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _vp]),
    "bfp8_silu_mul": (ctypes.c_int, [_vp, _i64, _i64, _i64, _vp, _i64, _vp]),
    "bfp8_quantize_weight_block": (ctypes.c_int, [_vp, _i64, _i64, _i64, _vp, _i64, _vp, _i32, _vp]),
    "bfp8_linear_w8a8": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _vp, _i32, _i64, _i64, _i64,
                                        _vp, _i64, ctypes.POINTER(bfp8_members), _vp, _sz, _vp]),
    "bfp8_linear_w8a8_workspace": (_sz, [_i64, _i64, _i64, ctypes.POINTER(bfp8_members)]),
    "bfp8_linear_w8a16": (ctypes.c_int, [_vp, _i64, _vp, _vp, _i32, _i64, _i64, _i64, _vp, _i64,
                                         ctypes.POINTER(bfp8_members), _vp]),
    "bfp8_gemv_decode": (ctypes.c_int, [_vp, _i64, _vp, _vp, _i32, _i64, _i64, _i64, _vp, _i64,
                                        ctypes.POINTER(bfp8_members), _vp, _sz, _vp]),
    "bfp8_gemv_decode_workspace": (_sz, [_i64, _i64, _i64]),
    "bfp8_gemv_decode_w8a8": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _vp, _i32, _i64, _i64,
                                             _i64, _vp, _i64, ctypes.POINTER(bfp8_members), _vp,
                                             _sz, _vp]),
    "bfp8_gemv_decode_noalloc": (ctypes.c_int, [_vp, _i64, _vp, _vp, _i32, _i64, _i64, _i64, _vp,
                                                _i64, ctypes.POINTER(bfp8_members), _vp]),
    "bfp8_grouped_linear": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _vp, _i32, _vp, _i32, _i64,
                                           _i64, _i64, _vp, _i64, _vp, _sz, _vp]),
    "bfp8_grouped_linear_workspace": (_sz, [_i64, _i32, _i64, _i64]),
    "bfp8_linear_w8a8_silu_quant": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _vp, _i32, _i64,
                                                   _i64, _i64, _vp, _i64, _vp, _i64, _i64, _vp,
                                                   _sz, _vp]),
    "bfp8_linear_w8a8_silu_quant_workspace": (_sz, [_i64, _i64, _i64]),
    "bfp8_grouped_linear_silu_quant": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _vp, _i32, _vp,
                                                      _i32, _i64, _i64, _i64, _vp, _i64, _vp, _i64,
                                                      _i64, _vp, _sz, _vp]),
    "bfp8_grouped_linear_silu_quant_workspace": (_sz, [_i64, _i32, _i64, _i64]),
    "bfp8_decode_ffn": (ctypes.c_int, [_i32, _vp, _i64, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i64,
                                       _vp, _i64, _vp, _sz, _vp]),
    "bfp8_decode_ffn_workspace": (_sz, [_i64, _i64, _i64, _i32]),
    "bfp8_moe_gather_act_quant": (ctypes.c_int, [_vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp,
                                                 _i64, _i64, _vp]),
    "bfp8_moe_combine": (ctypes.c_int, [_vp, _i64, _i64, _i64, _vp, _vp, _i64, _i32, _vp, _i64,
                                        _vp]),
    "bfp8_kv_plan": (ctypes.c_int, [_vp, _vp, _i64, _vp, _i64, _vp, _i64, _i64, _i32, _vp, _vp,
                                    _vp, _vp, _i64, _vp, _vp]),
    # (their structs come packed as bytes, or by reference)
    "bfp8_kv_append": (ctypes.c_int, [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _vp]),
    "bfp8_kv_attention": (ctypes.c_int, [_vp, _vp, _vp]),
    "bfp8_kv_attention_workspace": (_sz, [_i64, _i64, _i64, _i64, _i64]),
    "bfp8_residual_norm": (ctypes.c_int, [_vp, _i64, _i64, _vp]),
    "bfp8_causal_conv": (ctypes.c_int, [_vp, _vp]),
    "bfp8_delta_rule": (ctypes.c_int, [_vp, _vp]),
    "bfp8_delta_rule_workspace": (_sz, [_i64, _i64, _i64, _i64, _i64]),
    "bfp8_gated_norm": (ctypes.c_int, [_vp, _vp]),
    "bfp8_rotary": (ctypes.c_int, [_vp, _vp]),
    "bfp8_device_status": (ctypes.c_int, [_vp]),
    "bfp8_selftest_wait_timeout": (ctypes.c_int, [ctypes.c_uint64, _vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def library_path() -> Path:
    return _LIB_PATH


def bfp8_status_string(status: int) -> str:
    return _lib.bfp8_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != BFP8_OK:
        raise Bfp8Error(status, where)


def _ptr(t) -> int | None:
    """A tensor's device address. Every pointer the library takes is memory of
    the current device; a host tensor, or one on another GPU, is refused here,
    before any kernel could read it."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError(f"bfp8: expected a CUDA tensor, got one on {t.device}")
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"bfp8: tensor on {t.device}, but the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


BFP8_SCALE_PER_TENSOR = 0x100


def _scale_dtype(t: torch.Tensor) -> int:
    """The dtype code of a scale tensor. A block grid has rank 2 (rank 3 for
    experts); a scale of rank 0 or 1 (one multiplier, or one per expert) is a
    per-tensor scale and carries BFP8_SCALE_PER_TENSOR."""
    code = {torch.bfloat16: BFP8_DT_BF16, torch.float32: BFP8_DT_F32,
            torch.float16: BFP8_DT_F16}.get(t.dtype, BFP8_DT_NONE)
    return code | BFP8_SCALE_PER_TENSOR if code and t.dim() <= 1 else code


def _members(member_rows):
    if member_rows is None:
        return None, None
    arr = (ctypes.c_int64 * len(member_rows))(*[int(v) for v in member_rows])
    m = bfp8_members(len(member_rows), arr)
    return ctypes.byref(m), (m, arr)


def bfp8_validate_grid(desc: bfp8_weight_desc, msg_len: int = 256) -> tuple[int, str]:
    """Returns (status, message). Host only: needs no GPU."""
    buf = ctypes.create_string_buffer(msg_len)
    rc = _lib.bfp8_validate_grid(ctypes.byref(desc), buf, msg_len)
    return rc, buf.value.decode()


def make_weight_desc(weight_dtype: int, weight_shape, scale_dtype: int = BFP8_DT_NONE,
                     scale_shape=None, has_row_scale: bool = False,
                     declared_quant_fp8: bool = True, declared_block=(128, 128),
                     member_rows=None, tensor_scale_dtype: int = BFP8_DT_NONE):
    """Builds a bfp8_weight_desc; returns (desc, keepalive)."""
    d = bfp8_weight_desc()
    d.weight_dtype = weight_dtype
    d.weight_rank = len(weight_shape)
    for i, v in enumerate(list(weight_shape)[:2]):
        d.weight_shape[i] = int(v)
    d.scale_dtype = scale_dtype
    sshape = list(scale_shape) if scale_shape is not None else []
    d.scale_rank = len(sshape)
    for i, v in enumerate(sshape[:2]):
        d.scale_shape[i] = int(v)
    d.has_row_scale = int(bool(has_row_scale))
    d.declared_quant_fp8 = int(bool(declared_quant_fp8))
    d.declared_block[0], d.declared_block[1] = int(declared_block[0]), int(declared_block[1])
    d.tensor_scale_dtype = tensor_scale_dtype
    keep = None
    if member_rows is not None:
        keep = (ctypes.c_int64 * len(member_rows))(*[int(v) for v in member_rows])
        d.n_members = len(member_rows)
        d.member_rows = keep
    return d, keep


def bfp8_act_quant_group(x, q, scales, s_stride_m=None, s_stride_kb=None, stream=None) -> None:
    M, K = x.shape
    ssm = scales.stride(0) if s_stride_m is None else s_stride_m
    sskb = scales.stride(1) if s_stride_kb is None else s_stride_kb
    _dtypes(x=(x, "bf16"), q=(q, "e4m3"), scales=(scales, "f32"))
    _rows(x, "x")
    _span(x, "x", M, K, x.stride(0), 1, 2)
    _out(q, "q", M, K, 1)
    _scales_out(scales, "scales", M, -(-K // 128), ssm, sskb,
                s_stride_m is not None or s_stride_kb is not None)
    _check(_lib.bfp8_act_quant_group(_ptr(x), M, K, x.stride(0), _ptr(q), q.stride(0),
                                     _ptr(scales), ssm, sskb, _stream(stream)),
           "bfp8_act_quant_group")


def bfp8_silu_mul_act_quant(gu, q, scales, s_stride_m=None, s_stride_kb=None, stream=None) -> None:
    M, two_i = gu.shape
    ssm = scales.stride(0) if s_stride_m is None else s_stride_m
    sskb = scales.stride(1) if s_stride_kb is None else s_stride_kb
    _dtypes(gu=(gu, "bf16"), q=(q, "e4m3"), scales=(scales, "f32"))
    _rows(gu, "gu")
    _span(gu, "gu", M, two_i, gu.stride(0), 1, 2)
    _out(q, "q", M, two_i // 2, 1)
    _scales_out(scales, "scales", M, -(-(two_i // 2) // 128), ssm, sskb,
                s_stride_m is not None or s_stride_kb is not None)
    _check(_lib.bfp8_silu_mul_act_quant(_ptr(gu), M, two_i // 2, gu.stride(0), _ptr(q),
                                        q.stride(0), _ptr(scales), ssm, sskb, _stream(stream)),
           "bfp8_silu_mul_act_quant")


def bfp8_silu_mul(gu, h, stream=None) -> None:
    """h = bf16(silu(gate) * up) for gu = [gate | up] ([M, 2I] BF16); h [M, I] BF16."""
    M, two_i = gu.shape
    _dtypes(gu=(gu, "bf16"), h=(h, "bf16"))
    _rows(gu, "gu")
    _span(gu, "gu", M, two_i, gu.stride(0), 1, 2)
    _out(h, "h", M, two_i // 2, 2)
    _check(_lib.bfp8_silu_mul(_ptr(gu), M, two_i // 2, gu.stride(0), _ptr(h), h.stride(0),
                              _stream(stream)),
           "bfp8_silu_mul")


def bfp8_quantize_weight_block(w, q, scale, stream=None) -> None:
    N, K = w.shape
    _dtypes(w=(w, "f32"), q=(q, "e4m3"))
    _rows(w, "w")
    _span(w, "w", N, K, w.stride(0), 1, 4)  # float32, as the library reads it
    _out(q, "q", N, K, 1)
    _grid_span(scale, "scale", -(-N // 128), -(-K // 128))
    _check(_lib.bfp8_quantize_weight_block(_ptr(w), N, K, w.stride(0), _ptr(q), q.stride(0),
                                           _ptr(scale), _scale_dtype(scale), _stream(stream)),
           "bfp8_quantize_weight_block")


def _span(t, name: str, rows: int, cols: int, rs: int, cs: int, elem_bytes: int) -> None:
    """Refuse a call that would make the library touch memory past the end of
    t's storage: rows x cols elements of elem_bytes bytes at element strides
    (rs, cs) from t's first element, as the library addresses them."""
    if t is None or isinstance(t, int) or rows <= 0 or cols <= 0:
        return
    if rs < 0 or cs < 0:
        raise ValueError(f"bfp8: {name}: negative stride ({rs}, {cs})")
    need = ((rows - 1) * rs + (cols - 1) * cs + 1) * elem_bytes
    if need <= t.numel() * t.element_size() and t.is_contiguous():
        return  # within the tensor's own elements
    st = t.untyped_storage()
    if t.data_ptr() + need > st.data_ptr() + st.nbytes():
        raise ValueError(f"bfp8: {name} is too small for the call: {rows} x {cols} elements "
                         f"at strides ({rs}, {cs}) reach past its storage")


def _layout(t, name: str, shape, pitch: int | None = None) -> None:
    """t must have exactly `shape` and unit stride along its last dimension
    (row pitch `pitch` when given, dense strides for higher ranks): the
    library reads it as dense row-major data, so a transposed view, a column
    slice or a permuted grid would be misread silently. Strides of size-1
    dimensions do not matter and are not checked."""
    if t is None or isinstance(t, int):
        return
    shape = tuple(int(v) for v in shape)
    if tuple(t.shape) != shape:
        raise ValueError(f"bfp8: {name} has shape {list(t.shape)}, expected {list(shape)}")
    want = [1] * len(shape)
    for d in range(len(shape) - 2, -1, -1):
        want[d] = want[d + 1] * shape[d + 1]
    if pitch is not None and len(shape) >= 2:
        want[-2] = int(pitch)
    for d, (st, w) in enumerate(zip(t.stride(), want)):
        if shape[d] > 1 and st != w:
            raise ValueError(f"bfp8: {name} has strides {list(t.stride())}; the library reads it "
                             f"as row-major with strides {want}")


_KINDS = {"bf16": (torch.bfloat16,), "e4m3": (torch.uint8, torch.float8_e4m3fn),
          "f32": (torch.float32,), "i32": (torch.int32,), "i64": (torch.int64,),
          "u8": (torch.uint8,)}


def _dtypes(**args) -> None:
    """Each tensor must hold the element type the library reads or writes at
    that argument (name=(tensor, kind)): a tensor of another type would be
    reinterpreted byte for byte. E4M3 data may be uint8 or float8_e4m3fn."""
    for name, (t, kind) in args.items():
        if t is None or isinstance(t, int):
            continue
        if t.dtype not in _KINDS[kind]:
            allowed = " or ".join(str(d) for d in _KINDS[kind])
            raise ValueError(f"bfp8: {name} must be {allowed}, got {t.dtype}")


def _rows(t, name: str) -> None:
    """An activation or output matrix passed with its own row pitch: the
    columns must be contiguous (unit stride along the last dimension)."""
    if t is None or isinstance(t, int) or t.dim() != 2:
        return
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"bfp8: {name} must have contiguous columns, got strides "
                         f"{list(t.stride())}")


def _out(t, name: str, rows: int, cols: int, elem_bytes: int) -> None:
    """An output the library writes as rows x cols row-major elements at
    t.stride(0): the view must cover them, not only its storage."""
    if rows <= 0 or cols <= 0:
        return
    if t.dim() != 2 or t.shape[0] < rows or t.shape[1] < cols:
        raise ValueError(f"bfp8: {name} is too small for the call: needs [{rows}, {cols}], "
                         f"got {list(t.shape)}")
    _rows(t, name)
    _span(t, name, rows, cols, t.stride(0), 1, elem_bytes)


def _scales_out(t, name: str, rows: int, cols: int, s_m: int, s_kb: int, explicit: bool) -> None:
    """A float32 scale output [rows, cols]: with the view's own strides the
    view must cover it; with caller strides (for example token-contiguous
    scales) only the storage can be checked."""
    if not explicit and rows > 0 and cols > 0 and (
            t.dim() != 2 or t.shape[0] < rows or t.shape[1] < cols):
        raise ValueError(f"bfp8: {name} is too small for the call: needs [{rows}, {cols}], "
                         f"got {list(t.shape)}")
    _span(t, name, rows, cols, s_m, s_kb, 4)


_SCALE_BYTES = {BFP8_DT_BF16: 2, BFP8_DT_F16: 2, BFP8_DT_F32: 4}


def _grid_span(t, name: str, rows: int, kb: int, experts: int | None = None) -> None:
    """A weight-scale argument: the block grid [rows, kb] (rows = the sum of
    ceil(N_i / 128) over members, kb = ceil(K / 128)), or [experts, rows, kb]
    for expert stacks, dense row-major; or one multiplier (one per expert) as
    a tensor of rank 0 or 1. A transposed or mis-shaped grid is refused here
    (the library would read it as this layout)."""
    eb = _SCALE_BYTES.get(_scale_dtype(t) & 0xFF)
    if eb is None:
        return  # refused by the library (SCALE_DTYPE) before anything is read
    n = 1 if experts is None else experts
    if t.dim() <= 1:
        if t.numel() != n:
            raise ValueError(f"bfp8: {name}: a per-tensor scale needs {n} element(s), "
                             f"got {t.numel()}")
        _span(t, name, n, 1, 1, 1, eb)
        return
    _layout(t, name, (rows, kb) if experts is None else (experts, rows, kb))
    _span(t, name, n * rows, kb, kb, 1, eb)


def _scale_rows(N: int, member_rows) -> int:
    return sum(-(-int(m) // 128) for m in member_rows) if member_rows else -(-N // 128)


def _ws(workspace):
    if workspace is None:
        return None, 0
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def bfp8_linear_w8a8_workspace(M: int, N: int, K: int, member_rows=None) -> int:
    mref, _keep = _members(member_rows)
    return int(_lib.bfp8_linear_w8a8_workspace(M, N, K, mref))


def bfp8_linear_w8a8(q_a, s_a, w, w_scale, y, member_rows=None, s_stride_m=None,
                     s_stride_kb=None, workspace=None, stream=None) -> None:
    M, K = q_a.shape
    N = w.shape[0]
    ssm = s_a.stride(0) if s_stride_m is None else s_stride_m
    sskb = s_a.stride(1) if s_stride_kb is None else s_stride_kb
    Kb = -(-K // 128)
    _dtypes(q_a=(q_a, "e4m3"), s_a=(s_a, "f32"), w=(w, "e4m3"), y=(y, "bf16"))
    _layout(q_a, "q_a", (M, K))
    _span(s_a, "s_a", M, Kb, ssm, sskb, 4)
    _layout(w, "w", (N, K))
    _grid_span(w_scale, "w_scale", _scale_rows(N, member_rows), Kb)
    _out(y, "y", M, N, 2)
    mref, _keep = _members(member_rows)
    wsp, wsb = _ws(workspace)
    _check(_lib.bfp8_linear_w8a8(_ptr(q_a), _ptr(s_a), ssm, sskb, _ptr(w), _ptr(w_scale),
                                 _scale_dtype(w_scale), M, N, K, _ptr(y), y.stride(0), mref,
                                 wsp, wsb, _stream(stream)),
           "bfp8_linear_w8a8")


def bfp8_linear_w8a16(x, w, w_scale, y, member_rows=None, stream=None) -> None:
    M, K = x.shape
    N = w.shape[0]
    _dtypes(x=(x, "bf16"), w=(w, "e4m3"), y=(y, "bf16"))
    _rows(x, "x")
    _span(x, "x", M, K, x.stride(0), 1, 2)
    _layout(w, "w", (N, K))
    _grid_span(w_scale, "w_scale", _scale_rows(N, member_rows), -(-K // 128))
    _out(y, "y", M, N, 2)
    mref, _keep = _members(member_rows)
    _check(_lib.bfp8_linear_w8a16(_ptr(x), x.stride(0), _ptr(w), _ptr(w_scale),
                                  _scale_dtype(w_scale), M, N, K, _ptr(y), y.stride(0), mref,
                                  _stream(stream)),
           "bfp8_linear_w8a16")


def bfp8_gemv_decode_workspace(M: int, N: int, K: int) -> int:
    return int(_lib.bfp8_gemv_decode_workspace(M, N, K))


def bfp8_gemv_decode(x, w, w_scale, y, workspace, member_rows=None, stream=None) -> None:
    M, K = x.shape
    N = w.shape[0]
    _dtypes(x=(x, "bf16"), w=(w, "e4m3"), y=(y, "bf16"))
    _rows(x, "x")
    _span(x, "x", M, K, x.stride(0), 1, 2)
    _layout(w, "w", (N, K))
    _grid_span(w_scale, "w_scale", _scale_rows(N, member_rows), -(-K // 128))
    _out(y, "y", M, N, 2)
    mref, _keep = _members(member_rows)
    _check(_lib.bfp8_gemv_decode(_ptr(x), x.stride(0), _ptr(w), _ptr(w_scale),
                                 _scale_dtype(w_scale), M, N, K, _ptr(y), y.stride(0), mref,
                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(stream)),
           "bfp8_gemv_decode")


def bfp8_gemv_decode_w8a8(q_a, s_a, w, w_scale, y, workspace, member_rows=None, s_stride_m=None,
                          s_stride_kb=None, stream=None) -> None:
    """Decode GEMV (M <= 16) on E4M3 tokens with 1x128 scales (W8A8 arithmetic)."""
    M, K = q_a.shape
    N = w.shape[0]
    ssm = s_a.stride(0) if s_stride_m is None else s_stride_m
    sskb = s_a.stride(1) if s_stride_kb is None else s_stride_kb
    Kb = -(-K // 128)
    _dtypes(q_a=(q_a, "e4m3"), s_a=(s_a, "f32"), w=(w, "e4m3"), y=(y, "bf16"))
    _layout(q_a, "q_a", (M, K))
    _span(s_a, "s_a", M, Kb, ssm, sskb, 4)
    _layout(w, "w", (N, K))
    _grid_span(w_scale, "w_scale", _scale_rows(N, member_rows), Kb)
    _out(y, "y", M, N, 2)
    mref, _keep = _members(member_rows)
    _check(_lib.bfp8_gemv_decode_w8a8(_ptr(q_a), _ptr(s_a), ssm, sskb, _ptr(w), _ptr(w_scale),
                                      _scale_dtype(w_scale), M, N, K, _ptr(y), y.stride(0), mref,
                                      _ptr(workspace),
                                      workspace.numel() * workspace.element_size(),
                                      _stream(stream)),
           "bfp8_gemv_decode_w8a8")


def bfp8_gemv_decode_noalloc(x, w, w_scale, y, member_rows=None, stream=None) -> None:
    """bfp8_gemv_decode without a workspace argument, for callers that cannot
    allocate device memory; its scratch is a fixed array inside the library."""
    M, K = x.shape
    N = w.shape[0]
    _dtypes(x=(x, "bf16"), w=(w, "e4m3"), y=(y, "bf16"))
    _rows(x, "x")
    _span(x, "x", M, K, x.stride(0), 1, 2)
    _layout(w, "w", (N, K))
    _grid_span(w_scale, "w_scale", _scale_rows(N, member_rows), -(-K // 128))
    _out(y, "y", M, N, 2)
    mref, _keep = _members(member_rows)
    _check(_lib.bfp8_gemv_decode_noalloc(_ptr(x), x.stride(0), _ptr(w), _ptr(w_scale),
                                         _scale_dtype(w_scale), M, N, K, _ptr(y), y.stride(0),
                                         mref, _stream(stream)),
           "bfp8_gemv_decode_noalloc")


def bfp8_grouped_linear_workspace(total_M: int, G: int, N: int, K: int) -> int:
    return int(_lib.bfp8_grouped_linear_workspace(total_M, G, N, K))


def bfp8_grouped_linear(q_a, s_a, w, w_scale, offsets, y, s_stride_m=None, s_stride_kb=None,
                        workspace=None, stream=None) -> None:
    T, K = q_a.shape
    G, N = w.shape[0], w.shape[1]
    ssm = s_a.stride(0) if s_stride_m is None else s_stride_m
    sskb = s_a.stride(1) if s_stride_kb is None else s_stride_kb
    Kb = -(-K // 128)
    _dtypes(q_a=(q_a, "e4m3"), s_a=(s_a, "f32"), w=(w, "e4m3"), offsets=(offsets, "i32"),
            y=(y, "bf16"))
    _layout(q_a, "q_a", (T, K))
    _span(s_a, "s_a", T, Kb, ssm, sskb, 4)
    _layout(w, "w", (G, N, K))
    _grid_span(w_scale, "w_scale", -(-N // 128), Kb, G)
    _layout(offsets, "offsets", (G + 1,))
    _out(y, "y", T, N, 2)
    wsp, wsb = _ws(workspace)
    _check(_lib.bfp8_grouped_linear(_ptr(q_a), _ptr(s_a), ssm, sskb, _ptr(w), _ptr(w_scale),
                                    _scale_dtype(w_scale), _ptr(offsets), G, T, N, K, _ptr(y),
                                    y.stride(0), wsp, wsb, _stream(stream)),
           "bfp8_grouped_linear")


def bfp8_linear_w8a8_silu_quant_workspace(M: int, I: int, K: int) -> int:
    return int(_lib.bfp8_linear_w8a8_silu_quant_workspace(M, I, K))


def bfp8_linear_w8a8_silu_quant(q_a, s_a, w, w_scale, q_h, s_h, s_stride_m=None,
                                s_stride_kb=None, sh_stride_m=None, sh_stride_kb=None,
                                workspace=None, stream=None) -> None:
    """Gate/up projection (w = gate rows over up rows, [2I, K]) with SiLU(gate)*up
    and the 1x128 quantization of h fused into its epilogue: q_h [M, I], s_h."""
    M, K = q_a.shape
    I = w.shape[0] // 2
    ssm = s_a.stride(0) if s_stride_m is None else s_stride_m
    sskb = s_a.stride(1) if s_stride_kb is None else s_stride_kb
    hsm = s_h.stride(0) if sh_stride_m is None else sh_stride_m
    hskb = s_h.stride(1) if sh_stride_kb is None else sh_stride_kb
    Kb = -(-K // 128)
    _dtypes(q_a=(q_a, "e4m3"), s_a=(s_a, "f32"), w=(w, "e4m3"), q_h=(q_h, "e4m3"),
            s_h=(s_h, "f32"))
    _layout(q_a, "q_a", (M, K))
    _span(s_a, "s_a", M, Kb, ssm, sskb, 4)
    _layout(w, "w", (2 * I, K))
    _grid_span(w_scale, "w_scale", _scale_rows(2 * I, [I, I]), Kb)
    _out(q_h, "q_h", M, I, 1)
    _scales_out(s_h, "s_h", M, -(-I // 128), hsm, hskb,
                sh_stride_m is not None or sh_stride_kb is not None)
    wsp, wsb = _ws(workspace)
    _check(_lib.bfp8_linear_w8a8_silu_quant(_ptr(q_a), _ptr(s_a), ssm, sskb, _ptr(w),
                                            _ptr(w_scale), _scale_dtype(w_scale), M, I, K,
                                            _ptr(q_h), q_h.stride(0), _ptr(s_h), hsm, hskb, wsp,
                                            wsb, _stream(stream)),
           "bfp8_linear_w8a8_silu_quant")


def bfp8_grouped_linear_silu_quant_workspace(total_M: int, G: int, I: int, K: int) -> int:
    return int(_lib.bfp8_grouped_linear_silu_quant_workspace(total_M, G, I, K))


def bfp8_grouped_linear_silu_quant(q_a, s_a, w, w_scale, offsets, q_h, s_h, s_stride_m=None,
                                   s_stride_kb=None, sh_stride_m=None, sh_stride_kb=None,
                                   workspace=None, stream=None) -> None:
    """Per-expert gate/up projection (w [G, 2I, K]) with the fused SiLU*up +
    1x128 quant epilogue over the token-offset table."""
    T, K = q_a.shape
    G, I = w.shape[0], w.shape[1] // 2
    ssm = s_a.stride(0) if s_stride_m is None else s_stride_m
    sskb = s_a.stride(1) if s_stride_kb is None else s_stride_kb
    hsm = s_h.stride(0) if sh_stride_m is None else sh_stride_m
    hskb = s_h.stride(1) if sh_stride_kb is None else sh_stride_kb
    Kb = -(-K // 128)
    _dtypes(q_a=(q_a, "e4m3"), s_a=(s_a, "f32"), w=(w, "e4m3"), offsets=(offsets, "i32"),
            q_h=(q_h, "e4m3"), s_h=(s_h, "f32"))
    _layout(q_a, "q_a", (T, K))
    _span(s_a, "s_a", T, Kb, ssm, sskb, 4)
    _layout(w, "w", (G, 2 * I, K))
    _grid_span(w_scale, "w_scale", _scale_rows(2 * I, [I, I]), Kb, G)
    _layout(offsets, "offsets", (G + 1,))
    _out(q_h, "q_h", T, I, 1)
    _scales_out(s_h, "s_h", T, -(-I // 128), hsm, hskb,
                sh_stride_m is not None or sh_stride_kb is not None)
    wsp, wsb = _ws(workspace)
    _check(_lib.bfp8_grouped_linear_silu_quant(_ptr(q_a), _ptr(s_a), ssm, sskb, _ptr(w),
                                               _ptr(w_scale), _scale_dtype(w_scale),
                                               _ptr(offsets), G, T, I, K, _ptr(q_h),
                                               q_h.stride(0), _ptr(s_h), hsm, hskb, wsp, wsb,
                                               _stream(stream)),
           "bfp8_grouped_linear_silu_quant")


BFP8_DECODE_W8A16, BFP8_DECODE_W8A8 = 0, 1


def bfp8_decode_ffn_workspace(M: int, H: int, I: int, arith: int = BFP8_DECODE_W8A16) -> int:
    return int(_lib.bfp8_decode_ffn_workspace(M, H, I, arith))


def bfp8_decode_ffn(x, w_gate_up, s_gate_up, w_down, s_down, y, workspace,
                    arith: int = BFP8_DECODE_W8A16, stream=None) -> None:
    """One dense-FFN decode step: gate/up GEMV -> SiLU*up -> down GEMV."""
    M, H = x.shape
    I = w_down.shape[1]
    Hb, Ib = -(-H // 128), -(-I // 128)
    _dtypes(x=(x, "bf16"), w_gate_up=(w_gate_up, "e4m3"), w_down=(w_down, "e4m3"),
            y=(y, "bf16"))
    _rows(x, "x")
    _span(x, "x", M, H, x.stride(0), 1, 2)
    _layout(w_gate_up, "w_gate_up", (2 * I, H))
    _grid_span(s_gate_up, "s_gate_up", 2 * Ib, Hb)
    _layout(w_down, "w_down", (H, I))
    _grid_span(s_down, "s_down", Hb, Ib)
    _out(y, "y", M, H, 2)
    # the library takes one scale dtype code for both grids
    sdt = _scale_dtype(s_gate_up)
    if _scale_dtype(s_down) != sdt:
        raise ValueError("bfp8: s_gate_up and s_down must have the same dtype and kind (both "
                         "block grids or both one multiplier): the call reads both with one "
                         f"scale dtype, got {s_gate_up.dtype} rank {s_gate_up.dim()} and "
                         f"{s_down.dtype} rank {s_down.dim()}")
    _check(_lib.bfp8_decode_ffn(arith, _ptr(x), x.stride(0), _ptr(w_gate_up), _ptr(s_gate_up),
                                _ptr(w_down), _ptr(s_down), sdt, M, H, I,
                                _ptr(y), y.stride(0), *_ws(workspace),
                                _stream(stream)),
           "bfp8_decode_ffn")


def bfp8_moe_gather_act_quant(x, row_token, q, scales, s_stride_m=None, s_stride_kb=None,
                              stream=None) -> None:
    """q[r], scales[r] = 1x128 quantization of x[row_token[r]] (int32 on the device)."""
    T, H = x.shape
    R = row_token.shape[0]
    ssm = scales.stride(0) if s_stride_m is None else s_stride_m
    sskb = scales.stride(1) if s_stride_kb is None else s_stride_kb
    _dtypes(x=(x, "bf16"), row_token=(row_token, "i32"), q=(q, "e4m3"), scales=(scales, "f32"))
    _rows(x, "x")
    _span(x, "x", T, H, x.stride(0), 1, 2)
    _layout(row_token, "row_token", (R,))
    _out(q, "q", R, H, 1)
    _scales_out(scales, "scales", R, -(-H // 128), ssm, sskb,
                s_stride_m is not None or s_stride_kb is not None)
    _check(_lib.bfp8_moe_gather_act_quant(_ptr(x), T, H, x.stride(0), _ptr(row_token), R, _ptr(q),
                                          q.stride(0), _ptr(scales), ssm, sskb, _stream(stream)),
           "bfp8_moe_gather_act_quant")


def bfp8_moe_combine(y, token_rows, token_weights, out, stream=None) -> None:
    """out[t] = bf16(sum_j token_weights[t, j] * y[token_rows[t, j]]), slot order j."""
    R, H = y.shape
    T, topk = token_rows.shape
    _dtypes(y=(y, "bf16"), token_rows=(token_rows, "i32"), token_weights=(token_weights, "f32"),
            out=(out, "bf16"))
    _rows(y, "y")
    _span(y, "y", R, H, y.stride(0), 1, 2)
    _layout(token_rows, "token_rows", (T, topk))
    _layout(token_weights, "token_weights", (T, topk))
    _out(out, "out", T, H, 2)
    _check(_lib.bfp8_moe_combine(_ptr(y), R, H, y.stride(0), _ptr(token_rows),
                                 _ptr(token_weights), T, topk, _ptr(out), out.stride(0),
                                 _stream(stream)),
           "bfp8_moe_combine")


# The calls below run once a layer and step, some of them for a few microseconds
# on the GPU, so their checks are one comparison a property; what one of them
# refuses goes to the helpers above, which say why.
_PLAIN = {"i32": torch.int32, "i64": torch.int64, "f32": torch.float32, "bf16": torch.bfloat16}
_KV_CACHE = struct.Struct("4Pq3i8q")         # bfp8_kv_cache
_KV_ATTENTION = struct.Struct("P2qP2qPqP2q2P4qfiPN")   # bfp8_kv_attention_args
_NORM = struct.Struct("PqPqPqPPifffPqPqPqP2q")         # bfp8_norm_args


_WEIGHT_CODES = {None: BFP8_DT_BF16, torch.bfloat16: BFP8_DT_BF16, torch.float32: BFP8_DT_F32,
                 torch.float16: BFP8_DT_F16}


def _device() -> int:
    return torch.cuda.current_device()


def _raw_stream(stream, dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _vec(t, name: str, kind: str, n: int, dev: int) -> int:
    """The address of a dense vector of n elements on the current device."""
    if t.dtype is _PLAIN[kind] and t.shape == (n,) and t.get_device() == dev and (
            n < 2 or t.stride(0) == 1):
        return t.data_ptr()
    _dtypes(**{name: (t, kind)})
    _layout(t, name, (n,))
    return _ptr(t)


def _matrix(t, name: str, kind: str, shape, dev: int) -> tuple[int, int]:
    """The address and row stride of a matrix with contiguous rows. (A matrix
    of one row has no row stride: its width stands in.)"""
    if t.shape != shape:
        raise ValueError(f"bfp8: {name} has shape {list(t.shape)}, expected {list(shape)}")
    st = t.stride()
    if shape[0] > 1 and st[1] == 1 and t.dtype is _PLAIN[kind] and t.get_device() == dev:
        return t.data_ptr(), st[0]
    if t.dtype not in _KINDS[kind] or t.get_device() != dev or (shape[1] > 1 and t.stride(1) != 1):
        _dtypes(**{name: (t, kind)})
        _ptr(t)
        raise ValueError(f"bfp8: {name} must have contiguous columns, got strides "
                         f"{list(t.stride())}")
    return t.data_ptr(), t.stride(0) if shape[0] > 1 else shape[1]


def _out_matrix(t, name: str, kind: str, rows: int, cols: int, elem_bytes: int,
                dev: int) -> tuple[int, int]:
    """The same for an output, which may be larger than what is written."""
    st = t.stride()
    if (rows > 1 and t.shape == (rows, cols) and st[1] == 1 and t.dtype in _KINDS[kind]
            and t.get_device() == dev):
        return t.data_ptr(), st[0]
    if t.dtype not in _KINDS[kind] or t.get_device() != dev or t.shape != (rows, cols):
        _dtypes(**{name: (t, kind)})
        _out(t, name, rows, cols, elem_bytes)
        _ptr(t)
    elif cols > 1 and t.stride(1) != 1:
        _rows(t, name)
    return t.data_ptr(), t.stride(0) if rows > 1 else cols


def _head_rows(t, name: str, T: int, H: int, D: int, dev: int) -> tuple[int, int, int]:
    """Address, token stride and head stride of [T, H, D] BF16 with contiguous head rows."""
    if t.shape != (T, H, D):
        raise ValueError(f"bfp8: {name} has shape {list(t.shape)}, expected {[T, H, D]}")
    if t.dtype is not torch.bfloat16 or t.get_device() != dev:
        _dtypes(**{name: (t, "bf16")})
        _ptr(t)
    st, sh, sd = t.stride()
    if D > 1 and sd != 1:
        raise ValueError(f"bfp8: {name} must have contiguous head rows, got strides {[st, sh, sd]}")
    return t.data_ptr(), st if T > 1 else H * D, sh if H > 1 else D


def _kv_cache(k_cache, v_cache, k_exp, v_exp, dev: int) -> tuple[bytes, int, int]:
    """The cache [pages, kv heads, page size, 128] as the library takes it (any
    strides of pages, heads and tokens, contiguous codes), its heads and width."""
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("bfp8: k_cache and v_cache must be [pages, heads, page size, head dim], "
                         f"got {list(k_cache.shape)} and {list(v_cache.shape)}")
    P, H, page, D = k_cache.shape
    ks, vs, es = k_cache.stride(), v_cache.stride(), k_exp.stride()
    # what a cache nearly always is; anything else is looked at piece by piece below
    e4m3 = _KINDS["e4m3"]
    if (P > 1 and H > 1 and page > 1 and ks[3] == 1 == vs[3] and k_cache.dtype in e4m3
            and v_cache.dtype in e4m3 and k_exp.dtype is v_exp.dtype is torch.uint8
            and k_exp.shape == v_exp.shape == (P, H) and v_exp.stride() == es
            and k_cache.get_device() == dev == v_cache.get_device()
            and k_exp.get_device() == dev == v_exp.get_device()):
        return _KV_CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), k_exp.data_ptr(),
                              v_exp.data_ptr(), P, page, H, D, *ks[:3], *vs[:3], *es), H, D
    lone = 128 * page * H   # the stride of a dimension of one element, which is never stepped along
    flat = []
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.dtype not in _KINDS["e4m3"] or t.get_device() != dev:
            _dtypes(**{name: (t, "e4m3")})
            _ptr(t)
        sp, sh, st, sd = t.stride()
        if D > 1 and sd != 1:
            raise ValueError(f"bfp8: {name} must have contiguous codes, got strides "
                             f"{list(t.stride())}")
        flat += [sp if P > 1 else lone, sh if H > 1 else lone, st if page > 1 else lone]
    exps = []
    for name, t in (("k_exp", k_exp), ("v_exp", v_exp)):
        if t.shape != (P, H):
            raise ValueError(f"bfp8: {name} has shape {list(t.shape)}, expected {[P, H]}")
        if t.dtype is not torch.uint8 or t.get_device() != dev:
            _dtypes(**{name: (t, "u8")})
            _ptr(t)
        sp, sh = t.stride()
        exps.append((sp if P > 1 else H, sh if H > 1 else 1))
    if exps[0] != exps[1]:
        raise ValueError(f"bfp8: k_exp and v_exp must have the same strides, got "
                         f"{list(k_exp.stride())} and {list(v_exp.stride())}")
    return _KV_CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), k_exp.data_ptr(),
                          v_exp.data_ptr(), P, page, H, D, *flat, *exps[0]), H, D


def bfp8_kv_plan(ctx_len, q_len, free_pages, block_table, page_size: int, q_offsets, kv_len, slots,
                 positions, counts, stream=None) -> None:
    """The block plan of one step: pages for each request's new tokens from the
    front of free_pages, and every new token's slot and position."""
    dev = _device()
    B, width = block_table.shape
    T, n_free = slots.shape[0], free_pages.shape[0]
    table, pitch = _matrix(block_table, "block_table", "i32", (B, width), dev)
    _check(_lib.bfp8_kv_plan(_vec(ctx_len, "ctx_len", "i32", B, dev),
                             _vec(q_len, "q_len", "i32", B, dev), B,
                             _vec(free_pages, "free_pages", "i32", n_free, dev), n_free, table,
                             pitch, width, page_size,
                             _vec(q_offsets, "q_offsets", "i32", B + 1, dev),
                             _vec(kv_len, "kv_len", "i32", B, dev),
                             _vec(slots, "slots", "i64", T, dev),
                             _vec(positions, "positions", "i32", T, dev), T,
                             _vec(counts, "counts", "i32", 3, dev), _raw_stream(stream, dev)),
           "bfp8_kv_plan")


def bfp8_kv_append(k, v, slots, k_cache, v_cache, k_exp, v_exp, stream=None) -> None:
    """Quantize new keys and values [T, kv heads, 128] into their slots of the cache."""
    dev = _device()
    cache, H, D = _kv_cache(k_cache, v_cache, k_exp, v_exp, dev)
    T = slots.shape[0]
    _check(_lib.bfp8_kv_append(*_head_rows(k, "k", T, H, D, dev), *_head_rows(v, "v", T, H, D, dev),
                               _vec(slots, "slots", "i64", T, dev), T, cache,
                               _raw_stream(stream, dev)),
           "bfp8_kv_append")


def bfp8_kv_attention_workspace(batch: int, tokens: int, max_q_len: int, n_heads: int,
                                n_kv_heads: int) -> int:
    return int(_lib.bfp8_kv_attention_workspace(batch, tokens, max_q_len, n_heads, n_kv_heads))


def bfp8_kv_attention(q, k_cache, v_cache, k_exp, v_exp, block_table, q_offsets, kv_len, out,
                      max_q_len: int, softmax_scale=None, window: int = -1, lse=None,
                      workspace=None, stream=None) -> None:
    """Causal attention of q [T, heads, 128] over the paged cache; softmax_scale
    defaults to 1 / sqrt(128)."""
    dev = _device()
    cache, H, D = _kv_cache(k_cache, v_cache, k_exp, v_exp, dev)
    T, heads, _ = q.shape
    B, width = block_table.shape
    args = _KV_ATTENTION.pack(
        *_head_rows(q, "q", T, heads, D, dev), *_head_rows(out, "out", T, heads, D, dev),
        *((0, 0) if lse is None else _matrix(lse, "lse", "f32", (T, heads), dev)),
        *_matrix(block_table, "block_table", "i32", (B, width), dev), width,
        _vec(q_offsets, "q_offsets", "i32", B + 1, dev), _vec(kv_len, "kv_len", "i32", B, dev),
        B, T, max_q_len, heads, D ** -0.5 if softmax_scale is None else softmax_scale, window,
        *((0, 0) if workspace is None else _ws(workspace)))
    _check(_lib.bfp8_kv_attention(args, cache, _raw_stream(stream, dev)), "bfp8_kv_attention")


def bfp8_residual_norm(y, residual, residual_out=None, *, q=None, scales=None, norm_out=None,
                       w_post=None, w_pre=None, gate=None, residual_scale: float = 1.0,
                       eps: float = 1e-6, weight_offset: float = 0.0, s_stride_m=None,
                       s_stride_kb=None, stream=None) -> None:
    """The post-norm of y, its gate, the residual sum, the pre-norm of the next
    block and its 1x128 quantization. gate is [H] (every token) or [T, H]."""
    dev = _device()
    T, H = shape = residual.shape
    none = (0, 0)
    if gate is None:
        gate_at = none
    elif gate.dim() == 1:
        gate_at = (_vec(gate, "gate", "bf16", H, dev), 0)
    else:
        gate_at = _matrix(gate, "gate", "bf16", shape, dev)
    weights, w_dtype = [0, 0], None
    for i, w in enumerate((w_post, w_pre)):
        if w is None:
            continue
        if w.shape != shape[1:] or w.get_device() != dev or (H > 1 and w.stride(0) != 1):
            _layout(w, ("w_post", "w_pre")[i], (H,))
        weights[i] = _ptr(w) if w.get_device() != dev else w.data_ptr()
        if w_dtype not in (None, w.dtype):
            raise ValueError("bfp8: w_post and w_pre must have the same dtype")
        w_dtype = w.dtype
    scales_at = (0, 0, 0)
    if q is not None:
        if scales is None:
            raise ValueError("bfp8: q needs scales")
        plain = s_stride_m is None and s_stride_kb is None
        ssm = scales.stride(0) if s_stride_m is None else s_stride_m
        sskb = scales.stride(1) if s_stride_kb is None else s_stride_kb
        if not plain or scales.dtype is not torch.float32 or scales.get_device() != dev or \
                scales.shape != (T, -(-H // 128)):
            _dtypes(scales=(scales, "f32"))
            _scales_out(scales, "scales", T, -(-H // 128), ssm, sskb, not plain)
            _ptr(scales)
        scales_at = (scales.data_ptr(), ssm, sskb)
    args = _NORM.pack(
        *(none if y is None else _matrix(y, "y", "bf16", shape, dev)),
        *_matrix(residual, "residual", "bf16", shape, dev), *gate_at, *weights,
        _WEIGHT_CODES.get(w_dtype, BFP8_DT_NONE),
        weight_offset, residual_scale, eps,
        *(none if residual_out is None else
          _out_matrix(residual_out, "residual_out", "bf16", T, H, 2, dev)),
        *(none if norm_out is None else _out_matrix(norm_out, "norm_out", "bf16", T, H, 2, dev)),
        *(none if q is None else _out_matrix(q, "q", "e4m3", T, H, 1, dev)), *scales_at)
    _check(_lib.bfp8_residual_norm(args, T, H, _raw_stream(stream, dev)), "bfp8_residual_norm")


# Packed as the library's structs lie in memory (a trailing 0q pads to their size).
_CAUSAL_CONV = struct.Struct("PqPq2P3iP3q3P3q")        # bfp8_causal_conv_args
_DELTA_RULE = struct.Struct("P2qP2qP2qPqPq3P3q3PP2q5qiffPN")   # bfp8_delta_rule_args
_GATED_NORM = struct.Struct("P2qP2qPiiffP2qPqP4qi0q")  # bfp8_gated_norm_args
_ROTARY = struct.Struct("P2qP2qP2qP2qPq3Pifff3q9i0q")  # bfp8_rotary_args
BFP8_ACT_SILU, BFP8_ACT_SIGMOID = 0, 1

# The calls below first try what their arguments nearly always are: one expression looks at
# types, shapes and inner strides, and the library itself refuses memory that is not the current
# device's. Where either says no, the call goes through the helpers, piece by piece, which put
# the strides of lone dimensions right, or say what is wrong. A call that the library refuses
# has done nothing; one that ends in a CUDA error may have launched kernels, which have a state
# on its way, and is not made again.
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _raise_cuda(status: int, name: str) -> None:
    if status == BFP8_ERR_CUDA:
        _check(status, name)


def _slots(state, slots_in, slots_out, B: int, dev: int) -> tuple[int, int, int]:
    """The pool's slots, and the addresses of the two slot arrays."""
    if state is None and not (slots_in is None and slots_out is None):
        raise ValueError("bfp8: slots_in and slots_out need a state")
    return (0 if state is None else state.shape[0],
            0 if slots_in is None else _vec(slots_in, "slots_in", "i32", B, dev),
            0 if slots_out is None else _vec(slots_out, "slots_out", "i32", B, dev))


def _weight(w, name: str, shape, dev: int) -> int:
    """The address of a dense weight on the current device (None: 0)."""
    if w is None:
        return 0
    if w.shape != shape or w.get_device() != dev or not w.is_contiguous():
        _layout(w, name, shape)
    return _ptr(w) if w.get_device() != dev else w.data_ptr()


def _one_dtype(names: str, *weights) -> int:
    """The dtype code that the weights share."""
    kinds = {w.dtype for w in weights if w is not None}
    if len(kinds) > 1:
        raise ValueError(f"bfp8: {names} must have the same dtype")
    return _WEIGHT_CODES.get(kinds.pop(), BFP8_DT_NONE) if kinds else BFP8_DT_BF16


def bfp8_causal_conv(x, weight, out, q_offsets, state=None, slots_in=None, slots_out=None, *,
                     bias=None, silu: bool = True, stream=None) -> None:
    """The short depthwise convolution of x [T, C] with weight [C, width] over each
    request's tokens; state [slots, width - 1, C] holds the inputs ahead of them."""
    dev = _device()
    T, C = shape = x.shape
    B, W = q_offsets.shape[0] - 1, weight.shape[1]
    if (state is not None and slots_in is not None and slots_out is not None
            and weight.shape == (C, W) and out.shape == shape
            and state.shape[1:] == (W - 1, C) and slots_in.shape == slots_out.shape == (B,)
            and x.dtype is out.dtype is state.dtype is _BF16
            and q_offsets.dtype is slots_in.dtype is slots_out.dtype is _I32
            and (bias is None or (bias.shape == (C,) and bias.dtype is weight.dtype
                                  and bias.is_contiguous()))
            and weight.is_contiguous() and q_offsets.is_contiguous()
            and slots_in.is_contiguous() and slots_out.is_contiguous()):
        (xt, xc), (ot, oc), (st, sr, sc) = x.stride(), out.stride(), state.stride()
        if xc == oc == sc == 1:
            status = _lib.bfp8_causal_conv(_CAUSAL_CONV.pack(
                x.data_ptr(), xt, out.data_ptr(), ot, weight.data_ptr(),
                0 if bias is None else bias.data_ptr(),
                _WEIGHT_CODES.get(weight.dtype, BFP8_DT_NONE), W, silu, state.data_ptr(), st, sr,
                state.shape[0], slots_in.data_ptr(), slots_out.data_ptr(), q_offsets.data_ptr(), B,
                T, C), _raw_stream(stream, dev))
            if status == BFP8_OK:
                return
            _raise_cuda(status, "bfp8_causal_conv")
    if state is None:
        at = (0, 0, 0)
    else:
        if state.dim() != 3 or state.shape[1:] != (W - 1, C):
            raise ValueError(f"bfp8: state has shape {list(state.shape)}, expected "
                             f"{['slots', W - 1, C]}")
        if state.dtype is not torch.bfloat16 or state.get_device() != dev:
            _dtypes(state=(state, "bf16"))
            _ptr(state)
        ss, sr, sc = state.stride()
        if C > 1 and sc != 1:
            raise ValueError("bfp8: state must have contiguous rows, got strides "
                             f"{list(state.stride())}")
        sr = sr if W > 2 else C
        at = (state.data_ptr(), ss if state.shape[0] > 1 else sr * (W - 1), sr)
    args = _CAUSAL_CONV.pack(
        *_matrix(x, "x", "bf16", (T, C), dev), *_out_matrix(out, "out", "bf16", T, C, 2, dev),
        _weight(weight, "weight", (C, W), dev), _weight(bias, "bias", (C,), dev),
        _one_dtype("weight and bias", weight, bias), W, silu, *at,
        *_slots(state, slots_in, slots_out, B, dev),
        _vec(q_offsets, "q_offsets", "i32", B + 1, dev), B, T, C)
    _check(_lib.bfp8_causal_conv(args, _raw_stream(stream, dev)), "bfp8_causal_conv")


def bfp8_delta_rule_workspace(batch: int, tokens: int, max_q_len: int, qk_heads: int,
                              v_heads: int) -> int:
    return int(_lib.bfp8_delta_rule_workspace(batch, tokens, max_q_len, qk_heads, v_heads))


def bfp8_delta_rule(q, k, v, a, b, a_log, dt_bias, state, slots_in, slots_out, q_offsets, out,
                    max_q_len: int, *, scale=None, eps: float = 1e-6, workspace=None,
                    stream=None) -> None:
    """The gated delta rule of q, k [T, qk heads, 128] and v [T, v heads, 128] with the
    gates' inputs a, b [T, v heads]; state [slots, v heads, 128, 128] is float32, a row a
    value and a column a key. scale defaults to 1 / sqrt(128)."""
    dev = _device()
    T, hk, D = qk = q.shape
    vo, B = v.shape, q_offsets.shape[0] - 1
    hv = vo[1]
    if scale is None:
        scale = D ** -0.5
    if (state is not None and slots_in is not None and slots_out is not None
            and k.shape == qk and vo == out.shape == (T, hv, D) and a.shape == b.shape == (T, hv)
            and a_log.shape == dt_bias.shape == (hv,) and state.shape[1:] == (hv, D, D)
            and slots_in.shape == slots_out.shape == (B,)
            and q.dtype is k.dtype is v.dtype is out.dtype is a.dtype is b.dtype is _BF16
            and a_log.dtype is dt_bias.dtype is state.dtype is _F32
            and q_offsets.dtype is slots_in.dtype is slots_out.dtype is _I32
            and a_log.is_contiguous() and dt_bias.is_contiguous() and q_offsets.is_contiguous()
            and slots_in.is_contiguous() and slots_out.is_contiguous()):
        (qt, qh, qd), (kt, kh, kd), (vt, vh, vd) = q.stride(), k.stride(), v.stride()
        (ot, oh, od), (ss, sh, sv, sk) = out.stride(), state.stride()
        (at, ah), (bt, bh) = a.stride(), b.stride()
        wsp, wsb = (0, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
        if qd == kd == vd == od == ah == bh == sk == 1 and sv == D:
            status = _lib.bfp8_delta_rule(_DELTA_RULE.pack(
                q.data_ptr(), qt, qh, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, a.data_ptr(),
                at, b.data_ptr(), bt, a_log.data_ptr(), dt_bias.data_ptr(), state.data_ptr(),
                ss, sh, state.shape[0], slots_in.data_ptr(), slots_out.data_ptr(),
                q_offsets.data_ptr(), out.data_ptr(), ot, oh, B, T, max_q_len, hk, hv, D,
                scale, eps, wsp, wsb), _raw_stream(stream, dev))
            if status == BFP8_OK:
                return
            _raise_cuda(status, "bfp8_delta_rule")
    if state is None:
        at = (0, 0, 0)
    else:
        if state.dim() != 4 or state.shape[1:] != (hv, D, D):
            raise ValueError(f"bfp8: state has shape {list(state.shape)}, expected "
                             f"{['slots', hv, D, D]}")
        if state.dtype is not torch.float32 or state.get_device() != dev:
            _dtypes(state=(state, "f32"))
            _ptr(state)
        ss, sh, sv, sk = state.stride()
        if D > 1 and (sv, sk) != (D, 1):
            raise ValueError("bfp8: state must have dense matrices, got strides "
                             f"{list(state.stride())}")
        sh = sh if hv > 1 else D * D
        at = (state.data_ptr(), ss if state.shape[0] > 1 else sh * hv, sh)
    args = _DELTA_RULE.pack(
        *_head_rows(q, "q", T, hk, D, dev), *_head_rows(k, "k", T, hk, D, dev),
        *_head_rows(v, "v", T, hv, D, dev), *_matrix(a, "a", "bf16", (T, hv), dev),
        *_matrix(b, "b", "bf16", (T, hv), dev), _vec(a_log, "a_log", "f32", hv, dev),
        _vec(dt_bias, "dt_bias", "f32", hv, dev), *at,
        *_slots(state, slots_in, slots_out, B, dev),
        _vec(q_offsets, "q_offsets", "i32", B + 1, dev), *_head_rows(out, "out", T, hv, D, dev),
        B, T, max_q_len, hk, hv, D, scale, eps,
        *((0, 0) if workspace is None else _ws(workspace)))
    _check(_lib.bfp8_delta_rule(args, _raw_stream(stream, dev)), "bfp8_delta_rule")


def bfp8_gated_norm(x, gate, weight, out=None, *, q=None, scales=None, eps: float = 1e-6,
                    weight_offset: float = 0.0, sigmoid: bool = False, s_stride_m=None,
                    s_stride_kb=None, stream=None) -> None:
    """The heads x [T, heads, 64, 128 or 256] normed (weight None: not), times SiLU (or the
    sigmoid) of gate, to BF16 (out) and / or 1x128 codes (q [T, heads * width], scales)."""
    dev = _device()
    T, H, D = shape = x.shape
    if (gate.shape == shape and x.dtype is gate.dtype is _BF16
            and (weight is None or (weight.shape == (D,) and weight.is_contiguous()))
            and (out is None or (out.shape == shape and out.dtype is _BF16))
            and (q is None or (q.shape == (T, H * D) and q.dtype in _KINDS["e4m3"]
                               and scales is not None and scales.shape == (T, -(-H * D // 128))
                               and scales.dtype is _F32 and s_stride_m is s_stride_kb is None))):
        (xt, xh, xd), (zt, zh, zd) = x.stride(), gate.stride()
        ot, oh, od = (0, 0, 1) if out is None else out.stride()
        (qt, qc), (sm, sk) = ((0, 1), (0, 0)) if q is None else (q.stride(), scales.stride())
        if xd == zd == od == qc == 1:
            status = _lib.bfp8_gated_norm(_GATED_NORM.pack(
                x.data_ptr(), xt, xh, gate.data_ptr(), zt, zh,
                0 if weight is None else weight.data_ptr(),
                _WEIGHT_CODES.get(None if weight is None else weight.dtype, BFP8_DT_NONE),
                BFP8_ACT_SIGMOID if sigmoid else BFP8_ACT_SILU, eps, weight_offset,
                0 if out is None else out.data_ptr(), ot, oh, 0 if q is None else q.data_ptr(), qt,
                0 if q is None else scales.data_ptr(), sm, sk, T, H, D), _raw_stream(stream, dev))
            if status == BFP8_OK:
                return
            _raise_cuda(status, "bfp8_gated_norm")
    scales_at = (0, 0, 0)
    if q is not None:
        if scales is None:
            raise ValueError("bfp8: q needs scales")
        groups, plain = -(-H * D // 128), s_stride_m is None and s_stride_kb is None
        ssm = scales.stride(0) if s_stride_m is None else s_stride_m
        sskb = scales.stride(1) if s_stride_kb is None else s_stride_kb
        if not plain or scales.dtype is not torch.float32 or scales.get_device() != dev or \
                scales.shape != (T, groups):
            _dtypes(scales=(scales, "f32"))
            _scales_out(scales, "scales", T, groups, ssm, sskb, not plain)
            _ptr(scales)
        scales_at = (scales.data_ptr(), ssm if T > 1 else groups, sskb if groups > 1 else 1)
    args = _GATED_NORM.pack(
        *_head_rows(x, "x", T, H, D, dev), *_head_rows(gate, "gate", T, H, D, dev),
        _weight(weight, "weight", (D,), dev), _one_dtype("weight", weight),
        BFP8_ACT_SIGMOID if sigmoid else BFP8_ACT_SILU, eps, weight_offset,
        *((0, 0, 0) if out is None else _head_rows(out, "out", T, H, D, dev)),
        *((0, 0) if q is None else _out_matrix(q, "q", "e4m3", T, H * D, 1, dev)), *scales_at,
        T, H, D)
    _check(_lib.bfp8_gated_norm(args, _raw_stream(stream, dev)), "bfp8_gated_norm")


def bfp8_rotary(q, k, positions, inv_freq, q_out=None, k_out=None, *, sections=None,
                interleaved: bool = False, adjacent: bool = False, q_weight=None, k_weight=None,
                eps: float = 1e-6, weight_offset: float = 0.0, factor: float = 1.0,
                stream=None) -> None:
    """Rotary positions on q and k [T, heads, 64, 128 or 256] (k may be None), in place
    unless q_out and k_out are given, behind the heads' norms where q_weight and k_weight
    are. positions is [T], or [axes, T] with sections pairs of columns to each axis."""
    dev = _device()
    T, H, D = shape = q.shape
    half = inv_freq.shape[0]
    if k is not None and positions.dim() == (1 if sections is None else 2):
        K = k.shape[1]
        qo, ko = q if q_out is None else q_out, k if k_out is None else k_out
        parts = (half,) if sections is None else tuple(sections)
        axes = len(parts)
        if (k.shape == ko.shape == (T, K, D) and qo.shape == shape and axes <= 4
                and positions.shape == ((T,) if sections is None else (axes, T))
                and q.dtype is k.dtype is qo.dtype is ko.dtype is _BF16
                and positions.dtype is _I32 and inv_freq.dtype is _F32 and inv_freq.is_contiguous()
                and (q_weight is None or (q_weight.shape == (D,) and q_weight.is_contiguous()))
                and (k_weight is None or (k_weight.shape == (D,) and k_weight.is_contiguous()
                                          and (q_weight is None or q_weight.dtype is k_weight.dtype)))):
            (qt, qh, qd), (kt, kh, kd), pt = q.stride(), k.stride(), positions.stride()
            (qot, qoh, qod), (kot, koh, kod) = qo.stride(), ko.stride()
            w = k_weight if q_weight is None else q_weight
            if qd == kd == qod == kod == pt[-1] == 1:
                status = _lib.bfp8_rotary(_ROTARY.pack(
                    q.data_ptr(), qt, qh, qo.data_ptr(), qot, qoh, k.data_ptr(), kt, kh,
                    ko.data_ptr(), kot, koh, positions.data_ptr(), pt[0], inv_freq.data_ptr(),
                    0 if q_weight is None else q_weight.data_ptr(),
                    0 if k_weight is None else k_weight.data_ptr(),
                    _WEIGHT_CODES.get(None if w is None else w.dtype, BFP8_DT_NONE), eps,
                    weight_offset, factor, T, H, K, D, 2 * half, axes, *parts, *(0,) * (4 - axes),
                    interleaved, adjacent), _raw_stream(stream, dev))
                if status == BFP8_OK:
                    return
                _raise_cuda(status, "bfp8_rotary")
    axes, pos = (1, (_vec(positions, "positions", "i32", T, dev), T)) if positions.dim() == 1 else \
        (positions.shape[0], _matrix(positions, "positions", "i32", (positions.shape[0], T), dev))
    parts = [half] if sections is None else list(sections)
    if len(parts) != axes or axes > 4:
        raise ValueError(f"bfp8: {len(parts)} sections for {axes} axes of positions (1 to 4)")
    at = []
    for x, out, name in ((q, q_out, "q"), (k, k_out, "k")):
        if x is None:
            at += [0] * 6
            continue
        H = x.shape[1]
        at += [*_head_rows(x, name, T, H, D, dev),
               *_head_rows(x if out is None else out, name + "_out", T, H, D, dev)]
    args = _ROTARY.pack(
        *at, *pos, _vec(inv_freq, "inv_freq", "f32", half, dev),
        _weight(q_weight, "q_weight", (D,), dev), _weight(k_weight, "k_weight", (D,), dev),
        _one_dtype("q_weight and k_weight", q_weight, k_weight), eps, weight_offset, factor, T,
        q.shape[1], 0 if k is None else k.shape[1], D, 2 * half, axes,
        *parts, *(0,) * (4 - axes), interleaved, adjacent)
    _check(_lib.bfp8_rotary(args, _raw_stream(stream, dev)), "bfp8_rotary")


def bfp8_device_status(stream=None) -> int:
    return int(_lib.bfp8_device_status(_stream(stream)))


def bfp8_selftest_wait_timeout(limit_ns: int, stream=None) -> None:
    """Launch the bounded-wait self-test (a barrier whose second arrival never
    comes); the next bfp8_device_status() reports the timeout."""
    _check(_lib.bfp8_selftest_wait_timeout(int(limit_ns), _stream(stream)),
           "bfp8_selftest_wait_timeout")
