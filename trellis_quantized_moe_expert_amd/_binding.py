"""ctypes binding of the C ABI in include/qtip_moe.h (argument marshalling only).

Every function keeps its C name.  Pointer arguments accept an int address, None (NULL)
or any object with a `data_ptr()` method (a torch tensor); device memory and streams
come from PyTorch, all computation happens in the HIP library.  The binding never
falls back to anything else: if the library is missing, `lib()` raises.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_NAME = "libqtip_moe.so"
LIB_PATH = os.path.join(_HERE, LIB_NAME)

QTIP_OK = 0
QTIP_ERR_INVALID_ARG = 1
QTIP_ERR_INVALID_CONFIG = 2
QTIP_ERR_NOT_SUPPORTED = 3
QTIP_ERR_HIP = 4
QTIP_ERR_CAPTURING = 5

QTIP_ARM_AUTO = 0
QTIP_ARM_GEMV = 1
QTIP_ARM_GROUPED = 2
QTIP_ARM_DEQUANT = 3
QTIP_ACT_AUTO = 0
QTIP_ACT_ROWS = 1
QTIP_ACT_FRAGMENTS = 2
QTIP_OUT_BF16 = 0
QTIP_OUT_F32 = 1
QTIP_OUT_E4M3 = 2
QTIP_DEFAULT_DECODE_FLOOR_BITSHIFT = 7
QTIP_DEFAULT_DECODE_FLOOR_LUT = 4
QTIP_DECODE_REGIME_MAX_TOKENS = 8
QTIP_RUNG_BITSHIFT = 0
QTIP_RUNG_LUT = 1
QTIP_SMALL_BATCH_FUSED = 0
QTIP_SMALL_BATCH_SEPARATE = 1
QTIP_LUT_RUNG_BITS = 9
QTIP_GATE_SOFTMAX = 0
QTIP_GATE_SIGMOID = 1
QTIP_MX_BLOCK = 32
QTIP_MX_SRC_BF16 = 0
QTIP_MX_SRC_F16 = 1
QTIP_MX_SRC_F32 = 2
QTIP_MX_SCALE_FLOOR = 0
QTIP_MX_SCALE_NEAREST = 1
QTIP_MX_PASS_GATE_UP = 0
QTIP_MX_PASS_DOWN = 1
QTIP_F8_BLOCK = 128
QTIP_F8_BF16 = 0
QTIP_F8_F16 = 1
QTIP_F8_F32 = 2
QTIP_F8_SCALE_AMAX = 0
QTIP_F8_SCALE_POW2 = 1
QTIP_F8_PASS_GATE_UP = 0
QTIP_F8_PASS_DOWN = 1


class qtip_moe_desc(ctypes.Structure):
    _fields_ = [("num_experts", ctypes.c_int32), ("top_k", ctypes.c_int32), ("hidden", ctypes.c_int32),
                ("inter", ctypes.c_int32), ("max_tokens", ctypes.c_int32), ("arm_override", ctypes.c_int32),
                ("variant", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("tile_m", ctypes.c_int32),
                ("dispatch_tile_m", ctypes.c_int32), ("dequant_traffic_ratio", ctypes.c_int32),
                ("act_layout", ctypes.c_int32), ("rung", ctypes.c_int32), ("decode_floor", ctypes.c_int32),
                ("small_batch", ctypes.c_int32)]


class qtip_moe_weights(ctypes.Structure):
    _fields_ = [("codes_gate", ctypes.c_void_p), ("codes_up", ctypes.c_void_p), ("codes_down", ctypes.c_void_p),
                ("scale_gate", ctypes.c_void_p), ("scale_up", ctypes.c_void_p), ("scale_down", ctypes.c_void_p),
                ("lut", ctypes.c_void_p)]


QTIP_VARIANT_SLOTS = 12


class qtip_moe_stats_t(ctypes.Structure):
    _fields_ = [("forward_calls", ctypes.c_uint64), ("gemv_launches", ctypes.c_uint64),
                ("grouped_launches", ctypes.c_uint64), ("route_launches", ctypes.c_uint64),
                ("combine_launches", ctypes.c_uint64), ("router_launches", ctypes.c_uint64),
                ("dequant_launches", ctypes.c_uint64),
                ("last_arm", ctypes.c_int32),
                ("last_n_tokens", ctypes.c_int32),
                ("gemv_variant_launches", ctypes.c_uint64 * QTIP_VARIANT_SLOTS),
                ("grouped_variant_launches", ctypes.c_uint64 * QTIP_VARIANT_SLOTS),
                ("routed_in_gate_up", ctypes.c_uint64), ("combined_in_down", ctypes.c_uint64)]


class qtip_moe_kernel_shape(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_int32), ("waves_per_workgroup", ctypes.c_int32),
                ("rows_per_task", ctypes.c_int32), ("pairs_per_decode", ctypes.c_int32)]


class qtip_moe_schedule(ctypes.Structure):
    _fields_ = [("arm", ctypes.c_int32), ("tile_m", ctypes.c_int32), ("gate_up", qtip_moe_kernel_shape),
                ("down", qtip_moe_kernel_shape), ("route_in_gate_up", ctypes.c_int32),
                ("combine_in_down", ctypes.c_int32)]


class qtip_moe_gate(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("num_groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("group_top", ctypes.c_int32), ("renormalise", ctypes.c_int32), ("scale", ctypes.c_float),
                ("bias", ctypes.c_void_p)]


class qtip_mx_weights(ctypes.Structure):
    _fields_ = [("codes_gate", ctypes.c_void_p), ("scales_gate", ctypes.c_void_p), ("codes_up", ctypes.c_void_p),
                ("scales_up", ctypes.c_void_p), ("codes_down", ctypes.c_void_p), ("scales_down", ctypes.c_void_p)]


class qtip_f8_weights(ctypes.Structure):
    _fields_ = qtip_mx_weights._fields_


class QtipError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str):
        self.status = status
        super().__init__(f"{fn} -> {status_name(status)}: {detail}")


_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_SIGS = {
    "qtip_moe_plan": (_I32, [ctypes.POINTER(qtip_moe_desc), ctypes.c_int, ctypes.POINTER(_P)]),
    "qtip_moe_plan_for_arch": (_I32, [ctypes.POINTER(qtip_moe_desc), ctypes.c_char_p, ctypes.POINTER(_P)]),
    "qtip_moe_plan_destroy": (_I32, [_P]),
    "qtip_moe_plan_info": (_I32, [_P, ctypes.POINTER(_I32), ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(_I32)]),
    "qtip_moe_select_arm": (_I32, [_P, _I32]),
    "qtip_moe_select_grouped": (_I32, [_P, _I32]),
    "qtip_moe_plan_schedule": (_I32, [_P, _I32, ctypes.POINTER(qtip_moe_schedule)]),
    "qtip_fill_woken_experts": (ctypes.c_double, [_I32, _I32, _I32]),
    "qtip_fill_pairs_per_woken_expert": (ctypes.c_double, [_I32, _I32, _I32]),
    "qtip_fill_select_grouped": (_I32, [_I32, _I32, _I32, _I32]),
    "qtip_fill_min_tokens": (_I32, [_I32, _I32, _I32]),
    "qtip_moe_forward": (_I32, [_P, ctypes.POINTER(qtip_moe_weights), _P, _P, _I32, _P, _P, ctypes.c_size_t, _P]),
    "qtip_moe_forward_noalloc": (_I32, [_P, ctypes.POINTER(qtip_moe_weights), _P, _P, _I32, _P, _P]),
    "qtip_moe_forward_hidden": (_I32, [_P, ctypes.POINTER(qtip_moe_weights), _P, _P, _I32, _P, _P, ctypes.c_size_t,
                                       _P]),
    "qtip_moe_router_logits": (_I32, [_P, _P, _P, _I32, _P, _P, ctypes.c_size_t, _P]),
    "qtip_moe_router_split": (_I32, [_P, _I32]),
    "qtip_moe_dequant_range": (_I32, [_P, ctypes.POINTER(_I32), ctypes.POINTER(_I32)]),
    "qtip_moe_dequantize": (_I32, [_P, ctypes.POINTER(qtip_moe_weights), _I32, _I32, _P, _P]),
    "qtip_fill_select_arm": (_I32, [_I32, _I32, _I32, _I32, _I32]),
    "qtip_moe_route": (_I32, [_P, _P, _I32, _P, _P, _P, _P, _P, _P, _P, _P]),
    "qtip_expert_matmul": (_I32, [_P, _I32, _P, _P, _P, _I32, _I32, _I32, _P, _I32, _P, _I32, _P, _P]),
    "qtip_moe_stats": (_I32, [_P, ctypes.POINTER(qtip_moe_stats_t)]),
    "qtip_moe_stats_reset": (_I32, [_P]),
    "qtip_moe_engaged_line": (_I32, [_P, _I32, ctypes.c_char_p, ctypes.c_size_t]),
    "qtip_moe_log_engaged": (_I32, [_P, _I32, ctypes.POINTER(_I32)]),
    "qtip_arch_witness": (_I32, [ctypes.c_int, _P]),
    "qtip_moe_profile_enable": (_I32, [_P, _I32]),
    "qtip_moe_profile_read": (_I32, [_P, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_I32)]),
    "qtip_measure_lut_gather": (_I32, [_I32, _P, ctypes.c_size_t, _P, ctypes.POINTER(ctypes.c_double)]),
    "qtip_moe_gate_workspace_bytes": (ctypes.c_size_t, [_P]),
    "qtip_moe_gate_route": (_I32, [_P, ctypes.POINTER(qtip_moe_gate), _P, _I32, _P, _P, _P, _P, _P, _P, _P, _P,
                                   ctypes.c_size_t, _P]),
    "qtip_moe_forward_gated": (_I32, [_P, ctypes.POINTER(qtip_moe_weights), ctypes.POINTER(qtip_moe_gate), _P, _P,
                                      _I32, _P, _P, ctypes.c_size_t, _P]),
    "qtip_mx_quantize": (_I32, [_P, _I32, _I32, _I32, ctypes.c_int64, _I32, _P, _P, _P, _P]),
    "qtip_mx_matmul": (_I32, [_P, _P, _I32, _P, _P, _I32, _I32, _P, _I32, _P]),
    "qtip_mx_expert_matmul": (_I32, [_P, _I32, ctypes.POINTER(qtip_mx_weights), _P, _P, _P, _P, _I32, _P, _I32, _P]),
    "qtip_mx_moe_workspace_bytes": (ctypes.c_size_t, [_P]),
    "qtip_mx_moe_forward": (_I32, [_P, ctypes.POINTER(qtip_mx_weights), ctypes.POINTER(qtip_moe_gate), _P, _P, _I32,
                                   _P, _P, ctypes.c_size_t, _P]),
    "qtip_f8_quantize": (_I32, [_P, _I32, _I32, _I32, ctypes.c_int64, _I32, _I32, _P, _P, _P]),
    "qtip_f8_rms_norm": (_I32, [_P, _I32, _I32, _I32, ctypes.c_int64, _P, ctypes.c_int64, _P, _P, _I32, ctypes.c_float,
                                _I32, _P, _P, _P, _P]),
    "qtip_f8_matmul": (_I32, [_P, _P, _I32, _P, _P, _I32, _I32, _P, _I32, _P]),
    "qtip_f8_expert_matmul": (_I32, [_P, _I32, ctypes.POINTER(qtip_f8_weights), _P, _P, _P, _P, _I32, _P, _I32, _P,
                                     _P]),
    "qtip_f8_moe_workspace_bytes": (ctypes.c_size_t, [_P]),
    "qtip_f8_moe_forward": (_I32, [_P, ctypes.POINTER(qtip_f8_weights), ctypes.POINTER(qtip_moe_gate), _P, _P, _P,
                                   _I32, _P, _P, ctypes.c_size_t, _P]),
    "qtip_status_string": (ctypes.c_char_p, [_I32]),
    "qtip_last_error_detail": (ctypes.c_char_p, []),
}

_lib = None


def lib() -> ctypes.CDLL:
    """Load the HIP library (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it first (python -m "
                              f"trellis_quantized_moe_expert_amd.build or __graft_entry__.build())")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def status_name(status: int) -> str:
    return lib().qtip_status_string(status).decode()


def last_error_detail() -> str:
    return lib().qtip_last_error_detail().decode()


def _ptr(obj):
    if obj is None:
        return None
    if hasattr(obj, "data_ptr"):
        return obj.data_ptr()
    return int(obj)


_torch = None       # torch, once it has been needed; None again where it is not installed
_get_device = None  # torch's current device and its stream's handle as plain calls: 0.4 us a call
_get_stream = None  # against 3.6 through torch.cuda.current_stream()
_types = {}         # by kind of array (_KINDS): the element types it may have, the usual one first
_KINDS = {"f": "float32", "i": "int32", "b": "bfloat16 int16 uint16", "h": "float16 int16 uint16",
          "u": "uint8 int8 float4_e2m1fn_x2 float8_e8m0fnu",  # 16-bit values may come as their bits
          "e": "uint8 int8 float8_e4m3fn"}


def _find_torch() -> bool:
    """Import torch on first use and look its calls up once."""
    global _torch, _get_device, _get_stream
    if _torch is None:
        try:
            import torch
        except ImportError:
            return False
        _get_device = torch.cuda.current_device
        _get_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _types.update((kind, [getattr(torch, name) for name in names.split() if hasattr(torch, name)])
                      for kind, names in _KINDS.items())
        _torch = torch
    return True


def _stream(stream):
    if stream is None:
        if _torch is None and not _find_torch():
            return None
        if _get_stream is not None and _torch.cuda.is_initialized():
            return _get_stream(_get_device())
        if _torch.cuda.is_available():
            return _torch.cuda.current_stream().cuda_stream
        return None
    if hasattr(stream, "cuda_stream"):
        return stream.cuda_stream
    return int(stream)


def _check(fn: str, status: int):
    if status != QTIP_OK:
        raise QtipError(fn, status, last_error_detail())


def make_desc(num_experts, top_k, hidden, inter, max_tokens, arm_override=QTIP_ARM_AUTO, variant=0,
              out_dtype=QTIP_OUT_F32, tile_m=0, dispatch_tile_m=0, dequant_traffic_ratio=0,
              act_layout=QTIP_ACT_AUTO, rung=QTIP_RUNG_BITSHIFT, decode_floor=0,
              small_batch=QTIP_SMALL_BATCH_FUSED) -> qtip_moe_desc:
    return qtip_moe_desc(num_experts, top_k, hidden, inter, max_tokens, arm_override, variant, out_dtype, tile_m,
                         dispatch_tile_m, dequant_traffic_ratio, act_layout, rung, decode_floor, small_batch)


def make_weights(codes_gate, codes_up, codes_down, scale_gate, scale_up, scale_down, lut) -> qtip_moe_weights:
    return qtip_moe_weights(*(_ptr(a) for a in (codes_gate, codes_up, codes_down, scale_gate, scale_up,
                                                scale_down, lut)))


class Plan(int):
    """A plan's handle that knows its layer, for the checks of tensors' sizes: `layer` is (E, k, H, I, out_dtype)."""

    def __new__(cls, handle: int, desc: qtip_moe_desc):
        self = super().__new__(cls, handle)
        self.layer = (desc.num_experts, desc.top_k, desc.hidden, desc.inter, desc.out_dtype)
        return self


# ---- the C entry points, same names --------------------------------------------------------
def qtip_moe_plan(desc: qtip_moe_desc, device: int = 0) -> int:
    out = _P()
    _check("qtip_moe_plan", lib().qtip_moe_plan(ctypes.byref(desc), device, ctypes.byref(out)))
    return Plan(out.value, desc)


def qtip_moe_plan_for_arch(desc: qtip_moe_desc, arch: str) -> int:
    out = _P()
    _check("qtip_moe_plan_for_arch", lib().qtip_moe_plan_for_arch(ctypes.byref(desc), arch.encode(), ctypes.byref(out)))
    return Plan(out.value, desc)


def qtip_moe_plan_destroy(plan: int) -> None:
    _check("qtip_moe_plan_destroy", lib().qtip_moe_plan_destroy(plan))


def qtip_moe_plan_info(plan: int) -> dict:
    tm, mt, ws = _I32(), _I32(), ctypes.c_size_t()
    _check("qtip_moe_plan_info", lib().qtip_moe_plan_info(plan, ctypes.byref(tm), ctypes.byref(ws), ctypes.byref(mt)))
    return {"tile_m": tm.value, "workspace_bytes": ws.value, "min_tokens_grouped": mt.value}


def qtip_moe_plan_schedule(plan: int, n_tokens: int) -> dict:
    out = qtip_moe_schedule()
    _check("qtip_moe_plan_schedule", lib().qtip_moe_plan_schedule(plan, n_tokens, ctypes.byref(out)))
    shape = lambda sh: {name: getattr(sh, name) for name, _ in qtip_moe_kernel_shape._fields_}
    return {"arm": out.arm, "tile_m": out.tile_m, "gate_up": shape(out.gate_up), "down": shape(out.down),
            "route_in_gate_up": out.route_in_gate_up, "combine_in_down": out.combine_in_down}


def qtip_moe_select_arm(plan: int, n_tokens: int) -> int:
    return lib().qtip_moe_select_arm(plan, n_tokens)


def qtip_moe_select_grouped(plan: int, n_tokens: int) -> int:
    return lib().qtip_moe_select_grouped(plan, n_tokens)


def qtip_fill_woken_experts(n, k, E) -> float:
    return lib().qtip_fill_woken_experts(n, k, E)


def qtip_fill_pairs_per_woken_expert(n, k, E) -> float:
    return lib().qtip_fill_pairs_per_woken_expert(n, k, E)


def qtip_fill_select_grouped(n, k, E, tile_m) -> int:
    return lib().qtip_fill_select_grouped(n, k, E, tile_m)


def qtip_fill_min_tokens(k, E, tile_m) -> int:
    return lib().qtip_fill_min_tokens(k, E, tile_m)


def qtip_moe_forward(plan, weights: qtip_moe_weights, x_bf16, logits, n_tokens, out, workspace, workspace_bytes,
                     stream=None) -> None:
    _check("qtip_moe_forward", lib().qtip_moe_forward(plan, ctypes.byref(weights), _ptr(x_bf16), _ptr(logits),
                                                      n_tokens, _ptr(out), _ptr(workspace), workspace_bytes,
                                                      _stream(stream)))


QTIP_NOALLOC_SCRATCH_BYTES = 64 << 20


def qtip_moe_forward_noalloc(plan, weights: qtip_moe_weights, x_bf16, logits, n_tokens, out, stream=None) -> None:
    _check("qtip_moe_forward_noalloc", lib().qtip_moe_forward_noalloc(plan, ctypes.byref(weights), _ptr(x_bf16),
                                                                      _ptr(logits), n_tokens, _ptr(out),
                                                                      _stream(stream)))


def qtip_moe_forward_hidden(plan, weights: qtip_moe_weights, w_router_bf16, x_bf16, n_tokens, out, workspace,
                            workspace_bytes, stream=None) -> None:
    _check("qtip_moe_forward_hidden", lib().qtip_moe_forward_hidden(plan, ctypes.byref(weights), _ptr(w_router_bf16),
                                                                    _ptr(x_bf16), n_tokens, _ptr(out),
                                                                    _ptr(workspace), workspace_bytes,
                                                                    _stream(stream)))


def qtip_moe_router_logits(plan, x_bf16, w_router_bf16, n_tokens, logits, workspace, workspace_bytes,
                           stream=None) -> None:
    _check("qtip_moe_router_logits", lib().qtip_moe_router_logits(plan, _ptr(x_bf16), _ptr(w_router_bf16), n_tokens,
                                                                  _ptr(logits), _ptr(workspace), workspace_bytes,
                                                                  _stream(stream)))


def qtip_moe_dequant_range(plan) -> tuple:
    lo, hi = _I32(), _I32()
    _check("qtip_moe_dequant_range", lib().qtip_moe_dequant_range(plan, ctypes.byref(lo), ctypes.byref(hi)))
    return lo.value, hi.value


def qtip_moe_dequantize(plan, weights: qtip_moe_weights, matrix, expert, dense_out, stream=None) -> None:
    _check("qtip_moe_dequantize", lib().qtip_moe_dequantize(plan, ctypes.byref(weights), matrix, expert,
                                                            _ptr(dense_out), _stream(stream)))


def qtip_fill_select_arm(n, k, E, tile_m, dequant_ratio) -> int:
    return lib().qtip_fill_select_arm(n, k, E, tile_m, dequant_ratio)


def qtip_moe_router_split(plan, n_tokens) -> int:
    return lib().qtip_moe_router_split(plan, n_tokens)


def qtip_moe_route(plan, logits, n_tokens, topk_idx, topk_w, counts, offsets, sorted_pair, tile_map, n_tiles,
                   stream=None) -> None:
    _check("qtip_moe_route", lib().qtip_moe_route(plan, _ptr(logits), n_tokens, _ptr(topk_idx), _ptr(topk_w),
                                                  _ptr(counts), _ptr(offsets), _ptr(sorted_pair), _ptr(tile_map),
                                                  _ptr(n_tiles), _stream(stream)))


def qtip_expert_matmul(plan, arm, codes, scales, lut, num_experts, rows, cols, a_bf16, n_rows_a, unit_map, n_units,
                       y, stream=None) -> None:
    _check("qtip_expert_matmul", lib().qtip_expert_matmul(plan, arm, _ptr(codes), _ptr(scales), _ptr(lut),
                                                          num_experts, rows, cols, _ptr(a_bf16), n_rows_a,
                                                          _ptr(unit_map), n_units, _ptr(y), _stream(stream)))


def qtip_moe_stats(plan) -> dict:
    s = qtip_moe_stats_t()
    _check("qtip_moe_stats", lib().qtip_moe_stats(plan, ctypes.byref(s)))
    out = {}
    for name, _ in qtip_moe_stats_t._fields_:
        v = getattr(s, name)
        out[name] = list(v) if isinstance(v, ctypes.Array) else v
    return out


def qtip_moe_stats_reset(plan) -> None:
    _check("qtip_moe_stats_reset", lib().qtip_moe_stats_reset(plan))


def qtip_moe_engaged_line(plan, n_tokens) -> str:
    buf = ctypes.create_string_buffer(512)
    _check("qtip_moe_engaged_line", lib().qtip_moe_engaged_line(plan, n_tokens, buf, len(buf)))
    return buf.value.decode()


def qtip_moe_log_engaged(plan, n_tokens) -> bool:
    printed = _I32()
    _check("qtip_moe_log_engaged", lib().qtip_moe_log_engaged(plan, n_tokens, ctypes.byref(printed)))
    return bool(printed.value)


def qtip_arch_witness(device: int = 0, stream=None) -> None:
    _check("qtip_arch_witness", lib().qtip_arch_witness(device, _stream(stream)))


PROFILE_STAGES = ("route", "bin", "gate_up", "down", "combine")


def qtip_moe_profile_enable(plan, capacity: int) -> None:
    _check("qtip_moe_profile_enable", lib().qtip_moe_profile_enable(plan, capacity))


def qtip_moe_profile_read(plan) -> dict:
    ms = (ctypes.c_double * 5)()
    n = _I32()
    _check("qtip_moe_profile_read", lib().qtip_moe_profile_read(plan, ms, ctypes.byref(n)))
    return {"n_forwards": n.value, **{name: ms[i] for i, name in enumerate(PROFILE_STAGES)}}


def qtip_measure_lut_gather(rounds: int, sink, sink_elems: int, stream=None) -> float:
    out = ctypes.c_double()
    _check("qtip_measure_lut_gather", lib().qtip_measure_lut_gather(rounds, _ptr(sink), sink_elems, _stream(stream),
                                                                    ctypes.byref(out)))
    return out.value


# ---- the gate and MXFP4 -----------------------------------------------------------------------
def make_gate(score=QTIP_GATE_SOFTMAX, num_groups=1, top_groups=1, group_top=1, renormalise=1, scale=1.0,
              bias=None) -> qtip_moe_gate:
    """A gate; it keeps the bias tensor alive."""
    g = qtip_moe_gate(score, num_groups, top_groups, group_top, renormalise, scale, _ptr(bias))
    g.keep = bias
    g.seen = _seen("f", bias)
    return g


def make_mx_weights(codes_gate=None, scales_gate=None, codes_up=None, scales_up=None, codes_down=None,
                    scales_down=None) -> qtip_mx_weights:
    """MXFP4 expert weights; a pass reads only its own.  The struct keeps the tensors alive."""
    arrays = (codes_gate, scales_gate, codes_up, scales_up, codes_down, scales_down)
    w = qtip_mx_weights(*(_ptr(a) for a in arrays))
    w.keep = arrays
    w.seen = tuple(_seen("u", a) for a in arrays)
    return w


def make_f8_weights(codes_gate=None, scales_gate=None, codes_up=None, scales_up=None, codes_down=None,
                    scales_down=None) -> qtip_f8_weights:
    """e4m3 expert weights; a pass reads only its own.  The struct keeps the tensors alive."""
    arrays = (codes_gate, scales_gate, codes_up, scales_up, codes_down, scales_down)
    w = qtip_f8_weights(*(_ptr(a) for a in arrays))
    w.keep = arrays
    w.seen = tuple(_seen("ef"[i & 1], a) for i, a in enumerate(arrays))
    return w


def _is_tensor(obj) -> bool:
    return obj is not None and obj.__class__ is not int and _find_torch() and isinstance(obj, _torch.Tensor)


def _fault(kind: str, obj) -> str:
    """What is wrong with a tensor that stands for a whole array of a kind (".": any) in GPU memory."""
    if obj.get_device() < 0:
        return "is not in GPU memory"
    if kind != "." and obj.dtype not in _types[kind]:
        return f"has elements of {obj.dtype}, not of {_types[kind][0]}"
    return "" if obj.is_contiguous() else "must be contiguous"


def _refuse(fn: str, name: str, fault: str):
    raise QtipError(fn, QTIP_ERR_INVALID_ARG, f"{name} {fault}")


def _refuse_place(fn: str, name: str, device: int, have: int, size: int) -> None:
    if device != _get_device():
        _refuse(fn, name, f"is not on the current device (cuda:{_get_device()})")
    if have < size:
        _refuse(fn, name, f"is smaller than {size} bytes")


def _seen(kind: str, obj):
    """(fault, device, bytes) of a tensor whose address a struct takes; None of anything else."""
    return (_fault(kind, obj), obj.get_device(), obj.nbytes) if _is_tensor(obj) else None


def _check_seen(fn: str, name: str, facts: tuple, size: int) -> None:
    if facts[0]:
        _refuse(fn, name, facts[0])
    if facts[1] != _get_device() or facts[2] < size:
        _refuse_place(fn, name, facts[1], facts[2], size)


def _pointers(fn: str, kinds: str, names: tuple, objs: tuple, sizes: tuple) -> list:
    """The addresses of a call's arrays.  Tensors have to be whole arrays of their kind (a letter of _KINDS each, "."
    for any) and of at least so many bytes in the current GPU's memory; other objects are taken as they come."""
    if _torch is None and not _find_torch():
        return [_ptr(o) for o in objs]
    usual = _types.get(kinds)
    if usual is None:
        usual = _types[kinds] = [_types["u" if kind == "." else kind][0] for kind in kinds]
    tensor, device, out = _torch.Tensor, None, []
    for obj, dtype, size in zip(objs, usual, sizes):
        if obj.__class__ is tensor:
            where = obj.get_device()
            if device is None and where >= 0:
                device = _get_device()
            if where == device and obj.dtype is dtype and obj.nbytes >= size and obj.is_contiguous():
                out.append(obj.data_ptr())
                continue
        i = len(out)
        if isinstance(obj, tensor):
            fault = _fault(kinds[i], obj)
            if fault:
                _refuse(fn, names[i], fault)
            _refuse_place(fn, names[i], obj.get_device(), obj.nbytes, size)
        out.append(_ptr(obj))
    return out


def _layer(plan) -> tuple:
    """(E, k, H, I, out_dtype) of a plan; None of a handle that was not made here, whose arrays' sizes go unchecked."""
    return getattr(plan, "layer", None)


def _check_weights(fn: str, weights, codes: int, scales: int, first: int, last: int) -> None:
    """Arrays [first, last) of the struct's six: codes and scales in turn, of at least so many bytes."""
    device = None
    for facts in getattr(weights, "seen", ())[first:last]:
        if facts is not None:
            device = _get_device() if device is None and not facts[0] else device
            size = codes if first & 1 == 0 else scales
            if facts[0] or facts[1] != device or facts[2] < size:
                _check_seen(fn, weights._fields_[first][0], facts, size)
        first += 1


def _check_mx_weights(fn: str, weights, layer, first: int, last: int) -> None:
    """A matrix has H I values, two codes a byte, 32 to a scale."""
    codes = layer[0] * layer[2] * layer[3] // 2 if layer else 0
    _check_weights(fn, weights, codes, codes // 16, first, last)


def _check_f8_weights(fn: str, weights, layer, first: int, last: int) -> None:
    """A matrix has H I values, a byte each, 128 x 128 to a scale."""
    codes = layer[0] * layer[2] * layer[3] if layer else 0
    _check_weights(fn, weights, codes, codes // 4096, first, last)


def _check_bias(fn: str, gate, layer) -> None:
    facts = getattr(gate, "seen", None)
    if facts is not None:
        _check_seen(fn, "bias", facts, 4 * layer[0] if layer else 0)


def _out_kind(out_dtype: int) -> tuple:
    return ("f", 4) if out_dtype == QTIP_OUT_F32 else ("b", 2)


_ROUTE_NAMES = ("logits", "topk_idx", "topk_w", "counts", "offsets", "sorted_pair", "workspace", "tile_map", "n_tiles")
_SRC_KINDS = {QTIP_MX_SRC_BF16: ("b", 2), QTIP_MX_SRC_F16: ("h", 2), QTIP_MX_SRC_F32: ("f", 4)}


def qtip_moe_gate_workspace_bytes(plan) -> int:
    return lib().qtip_moe_gate_workspace_bytes(plan)


def qtip_moe_gate_route(plan, gate: qtip_moe_gate, logits, n_tokens, topk_idx, topk_w, counts, offsets, sorted_pair,
                        tile_map, n_tiles, workspace, workspace_bytes, stream=None) -> None:
    fn, layer = "qtip_moe_gate_route", _layer(plan)
    E, k = layer[:2] if layer else (-1, 0)
    pairs = 4 * n_tokens * k
    objs = logits, topk_idx, topk_w, counts, offsets, sorted_pair, workspace
    sizes = 4 * n_tokens * E, pairs, pairs, 4 * E, 4 * E + 4, pairs, workspace_bytes
    if tile_map is None and n_tiles is None:
        p = _pointers(fn, "fifiii.", _ROUTE_NAMES, objs, sizes)
        p += [None, None]
    else:
        p = _pointers(fn, "fifiii.ii", _ROUTE_NAMES, (*objs, tile_map, n_tiles), (*sizes, 3 * pairs, 4))
    _check_bias(fn, gate, layer)
    _check(fn, lib().qtip_moe_gate_route(plan, ctypes.byref(gate), p[0], n_tokens, p[1], p[2], p[3], p[4], p[5], p[7],
                                         p[8], p[6], workspace_bytes, _stream(stream)))


def _layer_pointers(fn: str, layer, x_bf16, logits, n_tokens: int, out, workspace, workspace_bytes: int) -> list:
    E, _, H, _, out_dtype = layer or (0, 0, 0, 0, None)
    kind, size = (".", 0) if out_dtype is None else _out_kind(out_dtype)
    return _pointers(fn, "bf" + kind + ".", ("x_bf16", "logits", "out", "workspace"), (x_bf16, logits, out, workspace),
                     (2 * n_tokens * H, 4 * n_tokens * E, size * n_tokens * H, workspace_bytes))


def qtip_moe_forward_gated(plan, weights: qtip_moe_weights, gate: qtip_moe_gate, x_bf16, logits, n_tokens, out,
                           workspace, workspace_bytes, stream=None) -> None:
    fn, layer = "qtip_moe_forward_gated", _layer(plan)
    p = _layer_pointers(fn, layer, x_bf16, logits, n_tokens, out, workspace, workspace_bytes)
    _check_bias(fn, gate, layer)
    _check(fn, lib().qtip_moe_forward_gated(plan, ctypes.byref(weights), ctypes.byref(gate), p[0], p[1], n_tokens, p[2],
                                            p[3], workspace_bytes, _stream(stream)))


def _check_rows(fn: str, name: str, kind: str, obj, rows: int, cols: int, row_stride: int) -> None:
    """A tensor of a kind with `rows` rows of cols elements, row_stride apart: rows of a wider tensor are welcome."""
    if not ((_torch is not None or _find_torch()) and isinstance(obj, _torch.Tensor)):
        return
    if obj.get_device() < 0 or obj.get_device() != _get_device():
        _refuse(fn, name, "is not on the current device")
    if kind != "." and obj.dtype not in _types[kind]:
        _refuse(fn, name, f"has elements of {obj.dtype}, not of {_types[kind][0]}")
    last = (rows - 1) * row_stride + cols
    if obj.numel() < last or not obj.is_contiguous():
        if obj.numel() == 0 or sum((n - 1) * st for n, st in zip(obj.shape, obj.stride())) < last - 1:
            _refuse(fn, name, "is smaller than its rows")
        if cols > 1 and obj.shape[-1] > 1 and obj.stride(-1) != 1:
            _refuse(fn, name, "must have a row's elements side by side")


def qtip_mx_quantize(src, src_type, rows, cols, row_stride, scale_rule, codes, scales, values=None,
                     stream=None) -> None:
    fn = "qtip_mx_quantize"
    blocks = (cols + QTIP_MX_BLOCK - 1) // QTIP_MX_BLOCK
    kind, size = _SRC_KINDS.get(src_type, (".", 0))
    _check_rows(fn, "src", kind, src, rows, cols, row_stride)
    sizes = 16 * rows * blocks, rows * blocks, rows * cols * size
    if values is None:
        p = _pointers(fn, "uu", ("codes", "scales"), (codes, scales), sizes)
        p.append(None)
    else:
        p = _pointers(fn, "uu" + kind, ("codes", "scales", "values"), (codes, scales, values), sizes)
    _check(fn, lib().qtip_mx_quantize(_ptr(src), src_type, rows, cols, row_stride, scale_rule, p[0], p[1], p[2],
                                      _stream(stream)))


def qtip_mx_matmul(a_codes, a_scales, m, w_codes, w_scales, n, k, out, out_dtype, stream=None) -> None:
    kind, size = _out_kind(out_dtype)
    p = _pointers("qtip_mx_matmul", "uuuu" + kind, ("a_codes", "a_scales", "w_codes", "w_scales", "out"),
                  (a_codes, a_scales, w_codes, w_scales, out),
                  (m * k // 2, m * k // 32, n * k // 2, n * k // 32, m * n * size))
    _check("qtip_mx_matmul", lib().qtip_mx_matmul(p[0], p[1], m, p[2], p[3], n, k, p[4], out_dtype, _stream(stream)))


def qtip_mx_expert_matmul(plan, pass_, weights: qtip_mx_weights, a_codes, a_scales, offsets, sorted_pair, n_tokens,
                          out, out_dtype, stream=None) -> None:
    fn, layer = "qtip_mx_expert_matmul", _layer(plan)
    E, k, H, I, _ = layer or (-1, 0, 0, 0, None)
    pairs = n_tokens * k
    gate_up = pass_ == QTIP_MX_PASS_GATE_UP
    values, width = (n_tokens * H, I) if gate_up else (pairs * I, H)
    kind, size = _out_kind(out_dtype)
    p = _pointers(fn, "uuii" + kind, ("a_codes", "a_scales", "offsets", "sorted_pair", "out"),
                  (a_codes, a_scales, offsets, sorted_pair, out),
                  (values // 2, values // 32, 4 * E + 4, 4 * pairs, pairs * width * size))
    _check_mx_weights(fn, weights, layer, 0 if gate_up else 4, 4 if gate_up else 6)
    _check(fn, lib().qtip_mx_expert_matmul(plan, pass_, ctypes.byref(weights), p[0], p[1], p[2], p[3], n_tokens, p[4],
                                           out_dtype, _stream(stream)))


def qtip_mx_moe_workspace_bytes(plan) -> int:
    return lib().qtip_mx_moe_workspace_bytes(plan)


def qtip_mx_moe_forward(plan, weights: qtip_mx_weights, gate, x_bf16, logits, n_tokens, out, workspace,
                        workspace_bytes, stream=None) -> None:
    fn, layer = "qtip_mx_moe_forward", _layer(plan)
    p = _layer_pointers(fn, layer, x_bf16, logits, n_tokens, out, workspace, workspace_bytes)
    _check_bias(fn, gate, layer)
    _check_mx_weights(fn, weights, layer, 0, 6)
    _check(fn, lib().qtip_mx_moe_forward(plan, ctypes.byref(weights), None if gate is None else ctypes.byref(gate),
                                         p[0], p[1], n_tokens, p[2], p[3], workspace_bytes, _stream(stream)))


def _f8_sizes(rows: int, cols: int, block_rows: int = 1) -> tuple:
    """Bytes of the codes and of the scales of rows of cols values."""
    return rows * ((cols + 15) // 16 * 16), 4 * ((rows + block_rows - 1) // block_rows) * ((cols + 127) // 128)


def qtip_f8_quantize(src, src_type, rows, cols, row_stride, block_rows, scale_rule, codes, scales, stream=None) -> None:
    fn = "qtip_f8_quantize"
    kind, size = _SRC_KINDS.get(src_type, (".", 0))
    sizes = _f8_sizes(rows, cols, max(block_rows, 1))
    if row_stride == cols:
        p = _pointers(fn, kind + "ef", ("src", "codes", "scales"), (src, codes, scales), (rows * cols * size, *sizes))
    else:
        _check_rows(fn, "src", kind, src, rows, cols, row_stride)
        p = [_ptr(src)] + _pointers(fn, "ef", ("codes", "scales"), (codes, scales), sizes)
    _check(fn, lib().qtip_f8_quantize(p[0], src_type, rows, cols, row_stride, block_rows, scale_rule, p[1], p[2],
                                      _stream(stream)))


def qtip_f8_rms_norm(x, type_, rows, cols, x_stride, residual, residual_stride, residual_out, weight, weight_type, eps,
                     scale_rule, codes, scales, values=None, stream=None) -> None:
    fn = "qtip_f8_rms_norm"
    kind, size = _SRC_KINDS.get(type_, (".", 0))
    w_kind, w_size = _SRC_KINDS.get(weight_type, (".", 0))
    whole = size * rows * cols
    summed = residual is not None or residual_out is not None
    names, kinds, objs, sizes = ("weight", "codes", "scales"), w_kind + "ef", (weight, codes, scales), (
        w_size * cols, *_f8_sizes(rows, cols))
    if values is not None:
        names, kinds, objs, sizes = (*names, "values"), kinds + kind, (*objs, values), (*sizes, whole)
    if x_stride == cols and (not summed or residual_stride == cols):  # whole arrays all of them
        if summed:
            names, kinds = ("x", "residual", "residual_out", *names), kind * 3 + kinds
            objs = x, residual, residual_out, *objs
            p = _pointers(fn, kinds, names, objs, (whole, whole, whole, *sizes))
        else:
            p = _pointers(fn, kind + kinds, ("x", *names), (x, *objs), (whole, *sizes))
            p[1:1] = None, None
    else:
        _check_rows(fn, "x", kind, x, rows, cols, x_stride)
        if summed:
            _check_rows(fn, "residual", kind, residual, rows, cols, residual_stride)
            _check_rows(fn, "residual_out", kind, residual_out, rows, cols, residual_stride)
        p = [_ptr(x), _ptr(residual), _ptr(residual_out)] + _pointers(fn, kinds, names, objs, sizes)
    _check(fn, lib().qtip_f8_rms_norm(p[0], type_, rows, cols, x_stride, p[1], residual_stride, p[2], p[3], weight_type,
                                      eps, scale_rule, p[4], p[5], p[6] if values is not None else None, _stream(stream)))


def qtip_f8_matmul(a_codes, a_scales, m, w_codes, w_scales, n, k, out, out_dtype, stream=None) -> None:
    kind, size = _out_kind(out_dtype)
    blocks = (k + 127) // 128 * 4
    p = _pointers("qtip_f8_matmul", "efef" + kind, ("a_codes", "a_scales", "w_codes", "w_scales", "out"),
                  (a_codes, a_scales, w_codes, w_scales, out),
                  (m * k, m * blocks, n * k, (n + 127) // 128 * blocks, m * n * size))
    _check("qtip_f8_matmul", lib().qtip_f8_matmul(p[0], p[1], m, p[2], p[3], n, k, p[4], out_dtype, _stream(stream)))


def qtip_f8_expert_matmul(plan, pass_, weights: qtip_f8_weights, a_codes, a_scales, offsets, sorted_pair, n_tokens,
                          out, out_dtype, out_scales=None, stream=None) -> None:
    fn, layer = "qtip_f8_expert_matmul", _layer(plan)
    E, k, H, I, _ = layer or (-1, 0, 0, 0, None)
    pairs = n_tokens * k
    gate_up = pass_ == QTIP_F8_PASS_GATE_UP
    values, width = (n_tokens * H, I) if gate_up else (pairs * I, H)
    kind, size = ("e", 1) if out_dtype == QTIP_OUT_E4M3 else _out_kind(out_dtype)
    objs = a_codes, a_scales, offsets, sorted_pair, out
    sizes = values, values // 32, 4 * E + 4, 4 * pairs, pairs * width * size
    names = "a_codes", "a_scales", "offsets", "sorted_pair", "out", "out_scales"
    if out_scales is None:
        p = _pointers(fn, "efii" + kind, names, objs, sizes)
        p.append(None)
    else:
        p = _pointers(fn, "efii" + kind + "f", names, (*objs, out_scales), (*sizes, pairs * width // 32))
    _check_f8_weights(fn, weights, layer, 0 if gate_up else 4, 4 if gate_up else 6)
    _check(fn, lib().qtip_f8_expert_matmul(plan, pass_, ctypes.byref(weights), p[0], p[1], p[2], p[3], n_tokens, p[4],
                                           out_dtype, p[5], _stream(stream)))


def qtip_f8_moe_workspace_bytes(plan) -> int:
    return lib().qtip_f8_moe_workspace_bytes(plan)


def qtip_f8_moe_forward(plan, weights: qtip_f8_weights, gate, x_codes, x_scales, logits, n_tokens, out, workspace,
                        workspace_bytes, stream=None) -> None:
    fn, layer = "qtip_f8_moe_forward", _layer(plan)
    E, _, H, _, out_dtype = layer or (0, 0, 0, 0, None)
    kind, size = (".", 0) if out_dtype is None else _out_kind(out_dtype)
    p = _pointers(fn, "eff" + kind + ".", ("x_codes", "x_scales", "logits", "out", "workspace"),
                  (x_codes, x_scales, logits, out, workspace),
                  (n_tokens * H, n_tokens * H // 32, 4 * n_tokens * E, size * n_tokens * H, workspace_bytes))
    _check_bias(fn, gate, layer)
    _check_f8_weights(fn, weights, layer, 0, 6)
    _check(fn, lib().qtip_f8_moe_forward(plan, ctypes.byref(weights), None if gate is None else ctypes.byref(gate),
                                         p[0], p[1], p[2], n_tokens, p[3], p[4], workspace_bytes, _stream(stream)))


def raw_status(fn_name: str, *args) -> int:
    """Call a C entry point with raw arguments and return its status (for error-path tests)."""
    return getattr(lib(), fn_name)(*args)
