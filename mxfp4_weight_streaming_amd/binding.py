"""ctypes binding of libmoe_decode.so (the C ABI in include/moe_decode.h).

Argument marshalling only: every step of the layer runs in the HIP kernels of
the library.  Tensors are passed as device pointers (``tensor.data_ptr()``),
streams as ``hipStream_t`` handles (default: torch's current stream).  Importing
this module fails loudly if the library has not been built; there is no other
implementation to fall back to.
"""
from __future__ import annotations

import ctypes
import os
import re

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_decode.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "moe_decode.h")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built; build it with `python -m mxfp4_weight_streaming_amd.build` "
        "(hipcc, gfx950). The MoE layer has no non-HIP implementation.")

_lib = ctypes.CDLL(LIB_PATH)

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED_SHAPE = -2
MOE_ERR_ALIGNMENT = -3
MOE_ERR_WORKSPACE = -4
MOE_ERR_HIP = -5
MOE_ERR_JIT = -6


class MoeShape(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("topk", ctypes.c_int32)]

    def __repr__(self):
        return f"MoeShape(H={self.hidden}, I={self.inter}, E={self.num_experts}, K={self.topk})"


class MoeRouteTaps(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("n_active", ctypes.c_void_p), ("act_experts", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p), ("pair_token", ctypes.c_void_p), ("pair_src", ctypes.c_void_p),
                ("act_fp8", ctypes.c_void_p), ("act_scale", ctypes.c_void_p)]


class MoeExpertTaps(ctypes.Structure):
    _fields_ = [("h", ctypes.c_void_p), ("inter_fp8", ctypes.c_void_p), ("inter_scale", ctypes.c_void_p)]


class MoeSharedExpert(ctypes.Structure):
    _fields_ = [("w13", ctypes.c_void_p), ("w13_scale", ctypes.c_void_p), ("w2", ctypes.c_void_p),
                ("w2_scale", ctypes.c_void_p)]


class MoeRouterParams(ctypes.Structure):
    _fields_ = [("num_experts", ctypes.c_int32), ("topk", ctypes.c_int32), ("score", ctypes.c_int32),
                ("num_groups", ctypes.c_int32), ("group_topk", ctypes.c_int32), ("group_score", ctypes.c_int32),
                ("renormalise", ctypes.c_int32), ("factor", ctypes.c_float)]


class MoeJitReport(ctypes.Structure):
    _fields_ = [("from_cache", ctypes.c_int32), ("has_chunk_path", ctypes.c_int32), ("has_lm_head", ctypes.c_int32),
                ("num_kernels", ctypes.c_int32), ("seconds", ctypes.c_double), ("cache_file", ctypes.c_char * 1024)]

    def as_dict(self) -> dict:
        return {"from_cache": bool(self.from_cache), "has_chunk_path": bool(self.has_chunk_path),
                "has_lm_head": bool(self.has_lm_head), "num_kernels": self.num_kernels, "seconds": self.seconds,
                "cache_file": self.cache_file.decode()}


_V = ctypes.c_void_p
_S = ctypes.POINTER(MoeShape)
_SH = ctypes.POINTER(MoeSharedExpert)
_i32 = ctypes.c_int32
_sz = ctypes.c_size_t
_RP = ctypes.POINTER(MoeRouterParams)

_SIGNATURES = {
    "moe_workspace_bytes": (_sz, [_S, _i32]),
    "moe_workspace_init": (ctypes.c_int, [_V, _sz, _V]),
    "moe_decode_forward": (ctypes.c_int, [_S, _i32, _V, _V, _V, _V, _V, _V, _V, _V, _sz, _V]),
    "moe_decode_forward_events": (ctypes.c_int, [_S, _i32, _V, _V, _V, _V, _V, _V, _V, _V, _sz, _V,
                                                  ctypes.POINTER(ctypes.c_void_p)]),
    "moe_decode_forward_shared": (ctypes.c_int, [_S, _i32, _V, _V, _V, _V, _V, _V, _SH, _V, _V, _sz, _V,
                                                  ctypes.POINTER(ctypes.c_void_p)]),
    "moe_decode_forward_noalloc": (ctypes.c_int, [_S, _i32, _V, _V, _V, _V, _V, _V, _V, _V]),
    "moe_route": (ctypes.c_int, [_S, _i32, _V, _V, _V, _V, ctypes.POINTER(MoeRouteTaps), _V, _sz, _V]),
    "moe_quant_act": (ctypes.c_int, [_S, _i32, _V, _V, _V, _V]),
    "moe_experts_forward": (ctypes.c_int, [_S, _i32, _V, _V, _V, _V, _V, _V, _V, _V, _V,
                                           ctypes.POINTER(MoeExpertTaps), _V, _sz, _V]),
    "moe_experts_forward_shared": (ctypes.c_int, [_S, _i32, _V, _V, _V, _V, _V, _V, _V, _V, _SH, _V,
                                                  ctypes.POINTER(MoeExpertTaps), _V, _sz, _V]),
    "moe_gate_up": (ctypes.c_int, [_S, _i32, _V, _V, _V, _V, _V, _V, _V, _V, _V, _sz, _V]),
    "moe_down_combine": (ctypes.c_int, [_S, _i32, _V, _V, _V, _V, _V, _V, _V, _V, _sz, _V]),
    "moe_fp8_encode_range": (ctypes.c_int, [ctypes.c_uint32, ctypes.c_int64, _V, _V]),
    "moe_lm_head_quantize": (ctypes.c_int, [_V, _i32, _i32, _V, _V, _V]),
    "moe_lm_head_forward": (ctypes.c_int, [_V, _i32, _V, _V, _i32, _i32, _V, _V]),
    "moe_add_rmsnorm": (ctypes.c_int, [_i32, _i32, _V, _i32, _V, _i32, _V, _i32, ctypes.c_double, _V, _V, _V, _i32,
                                       _V, _V]),
    "moe_route_scores": (ctypes.c_int, [_RP, _i32, _V, _V, _V, _V, _V]),
    "moe_router_logits": (ctypes.c_int, [_S, _i32, _V, _V, _V, _V]),
    "moe_decode_forward_scored": (ctypes.c_int, [_S, _RP, _i32, _V, _V, _V, _V, _V, _V, _V, _SH, _V, _V, _sz, _V]),
    "moe_int8_quantize": (ctypes.c_int, [_V, _i32, _i32, _V, _V, _V]),
    "moe_int8_linear": (ctypes.c_int, [_V, _V, _V, _V, _i32, _i32, _i32, _V, _i32, _V]),
    "moe_path_info": (ctypes.c_int, [_S, _i32, ctypes.c_char_p, _sz]),
    "moe_jit_build": (ctypes.c_int, [_S, ctypes.c_char_p, ctypes.c_char_p, ctypes.POINTER(MoeJitReport)]),
    "moe_jit_load": (ctypes.c_int, [_S, ctypes.c_char_p, _i32, ctypes.POINTER(MoeJitReport)]),
    "moe_jit_unload": (_i32, [_S]),
    "moe_workspace_sync_status": (ctypes.c_int, [_V, _sz, _V, _V]),
    "moe_set_wait_limit_us": (None, [ctypes.c_uint32]),
    "moe_set_decode_path": (ctypes.c_int, [_i32]),
    "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_last_error": (ctypes.c_char_p, []),
}
for _name, (_res, _args) in _SIGNATURES.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def header_functions() -> list[str]:
    """Names of the functions declared in include/moe_decode.h."""
    text = open(HEADER_PATH).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[\w]+\s*\*?\s*(moe_\w+)\s*\(", text, re.M)))


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.moe_last_error().decode()
        super().__init__(f"{where}: {_lib.moe_status_string(status).decode()} ({status}): {msg}")


def _check(status: int, where: str) -> int:
    if status != MOE_OK:
        raise MoeError(status, where)
    return status


def _p(t):
    """Device pointer of a tensor (or an int address, or None)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_current = None     # (current device, current stream's handle on a device), made at the first call


def _torch_current():
    """torch's current device and stream handles.  torch.cuda.current_stream() makes a Stream object, 2.8 us a call,
    as long as a kernel launch; torch's own compiled callers ask for the handle alone, 0.1 us."""
    global _current
    if _current is None:
        import torch
        torch.cuda.init()
        device, stream = getattr(torch._C, "_cuda_getDevice", None), getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if device is None or stream is None:
            device, stream = torch.cuda.current_device, lambda d: torch.cuda.current_stream(d).cuda_stream
        _current = device, stream
    return _current


def _stream(stream):
    if stream is None:
        device, handle = _current or _torch_current()
        return handle(device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def shape(hidden: int, inter: int, num_experts: int, topk: int) -> MoeShape:
    return MoeShape(hidden, inter, num_experts, topk)


def moe_workspace_bytes(shp: MoeShape, max_tokens: int) -> int:
    return _lib.moe_workspace_bytes(ctypes.byref(shp), max_tokens)


def moe_workspace_init(ws, stream=None) -> None:
    _check(_lib.moe_workspace_init(_p(ws), _nbytes(ws), _stream(stream)), "moe_workspace_init")


def workspace(shp: MoeShape, max_tokens: int, device="cuda"):
    """Allocate (through torch) and initialise a workspace for up to max_tokens."""
    import torch
    n = moe_workspace_bytes(shp, max_tokens)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED_SHAPE, "moe_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    moe_workspace_init(ws)
    torch.cuda.current_stream().synchronize()   # usable from any stream afterwards
    return ws


def moe_decode_forward(shp, M, hidden, router_w, w13, w13_scale, w2, w2_scale, out, ws, stream=None):
    _check(_lib.moe_decode_forward(ctypes.byref(shp), M, _p(hidden), _p(router_w), _p(w13), _p(w13_scale),
                                   _p(w2), _p(w2_scale), _p(out), _p(ws), _nbytes(ws), _stream(stream)),
           "moe_decode_forward")


def moe_decode_forward_noalloc(shp, M, hidden, router_w, w13, w13_scale, w2, w2_scale, out, stream=None):
    """moe_decode_forward on the library's static scratch (no workspace)."""
    _check(_lib.moe_decode_forward_noalloc(ctypes.byref(shp), M, _p(hidden), _p(router_w), _p(w13), _p(w13_scale),
                                           _p(w2), _p(w2_scale), _p(out), _stream(stream)),
           "moe_decode_forward_noalloc")


def moe_decode_forward_events(shp, M, hidden, router_w, w13, w13_scale, w2, w2_scale, out, ws, events,
                              stream=None):
    """events: 6 torch.cuda.Event (timing enabled, each recorded once so that it
    exists), start/stop pairs stamped by the router, gate/up and down launches."""
    if len(events) != 6:
        raise ValueError("moe_decode_forward_events takes 6 events (start/stop of 3 kernels)")
    arr = (ctypes.c_void_p * 6)(*[None if e is None else e.cuda_event for e in events])
    _check(_lib.moe_decode_forward_events(ctypes.byref(shp), M, _p(hidden), _p(router_w), _p(w13), _p(w13_scale),
                                          _p(w2), _p(w2_scale), _p(out), _p(ws), _nbytes(ws), _stream(stream),
                                          arr),
           "moe_decode_forward_events")


def _shared(shared):
    """A MoeSharedExpert from (w13, w13_scale, w2, w2_scale) tensors, or None."""
    if shared is None:
        return None
    if len(shared) != 4:
        raise ValueError("a shared expert is (w13, w13_scale, w2, w2_scale)")
    return MoeSharedExpert(*[_p(t) for t in shared])


def _events(events):
    if events is None:
        return None
    if len(events) != 6:
        raise ValueError("events: 6 torch.cuda.Event (start/stop of 3 kernels)")
    return (ctypes.c_void_p * 6)(*[None if e is None else e.cuda_event for e in events])


def moe_decode_forward_shared(shp, M, hidden, router_w, w13, w13_scale, w2, w2_scale, shared, out, ws,
                              events=None, stream=None):
    """moe_decode_forward plus the shared expert; shared = (w13, w13_scale, w2,
    w2_scale) of one expert, or None.  events as in moe_decode_forward_events."""
    sh = _shared(shared)
    _check(_lib.moe_decode_forward_shared(ctypes.byref(shp), M, _p(hidden), _p(router_w), _p(w13), _p(w13_scale),
                                          _p(w2), _p(w2_scale), ctypes.byref(sh) if sh is not None else None,
                                          _p(out), _p(ws), _nbytes(ws), _stream(stream), _events(events)),
           "moe_decode_forward_shared")


def moe_route(shp, M, hidden, router_w, topk_ids, topk_w, ws, taps: dict | None = None, stream=None):
    t = None
    if taps is not None:
        t = MoeRouteTaps(*[_p(taps.get(k)) for k, _ in MoeRouteTaps._fields_])
    _check(_lib.moe_route(ctypes.byref(shp), M, _p(hidden), _p(router_w), _p(topk_ids), _p(topk_w),
                          ctypes.byref(t) if t is not None else None, _p(ws), _nbytes(ws), _stream(stream)),
           "moe_route")


def moe_quant_act(shp, M, hidden, act_fp8, act_scale, stream=None):
    _check(_lib.moe_quant_act(ctypes.byref(shp), M, _p(hidden), _p(act_fp8), _p(act_scale), _stream(stream)),
           "moe_quant_act")


def moe_experts_forward(shp, M, act_fp8, act_scale, topk_ids, topk_w, w13, w13_scale, w2, w2_scale, out, ws,
                        taps: dict | None = None, stream=None):
    t = None
    if taps is not None:
        t = MoeExpertTaps(*[_p(taps.get(k)) for k, _ in MoeExpertTaps._fields_])
    _check(_lib.moe_experts_forward(ctypes.byref(shp), M, _p(act_fp8), _p(act_scale), _p(topk_ids), _p(topk_w),
                                    _p(w13), _p(w13_scale), _p(w2), _p(w2_scale), _p(out),
                                    ctypes.byref(t) if t is not None else None, _p(ws), _nbytes(ws),
                                    _stream(stream)),
           "moe_experts_forward")


def moe_experts_forward_shared(shp, M, act_fp8, act_scale, topk_ids, topk_w, w13, w13_scale, w2, w2_scale, shared,
                               out, ws, taps: dict | None = None, stream=None):
    """moe_experts_forward plus the shared expert; taps then hold M*K + M rows."""
    t = None
    if taps is not None:
        t = MoeExpertTaps(*[_p(taps.get(k)) for k, _ in MoeExpertTaps._fields_])
    sh = _shared(shared)
    _check(_lib.moe_experts_forward_shared(ctypes.byref(shp), M, _p(act_fp8), _p(act_scale), _p(topk_ids),
                                           _p(topk_w), _p(w13), _p(w13_scale), _p(w2), _p(w2_scale),
                                           ctypes.byref(sh) if sh is not None else None, _p(out),
                                           ctypes.byref(t) if t is not None else None, _p(ws), _nbytes(ws),
                                           _stream(stream)),
           "moe_experts_forward_shared")


def moe_gate_up(shp, M, act_fp8, act_scale, topk_ids, w13, w13_scale, h, inter_fp8, inter_scale, ws, stream=None):
    _check(_lib.moe_gate_up(ctypes.byref(shp), M, _p(act_fp8), _p(act_scale), _p(topk_ids), _p(w13),
                            _p(w13_scale), _p(h), _p(inter_fp8), _p(inter_scale), _p(ws), _nbytes(ws),
                            _stream(stream)),
           "moe_gate_up")


def moe_down_combine(shp, M, inter_fp8, inter_scale, topk_ids, topk_w, w2, w2_scale, out, ws, stream=None):
    _check(_lib.moe_down_combine(ctypes.byref(shp), M, _p(inter_fp8), _p(inter_scale), _p(topk_ids), _p(topk_w),
                                 _p(w2), _p(w2_scale), _p(out), _p(ws), _nbytes(ws), _stream(stream)),
           "moe_down_combine")


def moe_fp8_encode_range(first_bits: int, n: int, q, stream=None):
    _check(_lib.moe_fp8_encode_range(first_bits & 0xFFFFFFFF, n, _p(q), _stream(stream)), "moe_fp8_encode_range")


def moe_lm_head_quantize(w_bf16, q, scale, stream=None):
    """w_bf16 [V,H] -> q [V,H] E4M3 codes and scale [V] (one fp32 scale per row)."""
    V, H = w_bf16.shape
    _check(_lib.moe_lm_head_quantize(_p(w_bf16), V, H, _p(q), _p(scale), _stream(stream)), "moe_lm_head_quantize")


def moe_lm_head_forward(x_bf16, q, scale, logits, stream=None):
    """logits [M,V] = scale[v] * sum_k E4M3(q[v,k]) * x[t,k]."""
    M, H = x_bf16.shape
    V = q.shape[0]
    _check(_lib.moe_lm_head_forward(_p(x_bf16), M, _p(q), _p(scale), V, H, _p(logits), _stream(stream)),
           "moe_lm_head_forward")


# ---- around the expert layer --------------------------------------------------
# These calls check their tensors: each dense, on the current device, of a type
# the call knows, and of the shape that goes with the others (or, where M and the
# layer's shape are arguments, large enough).  bf16 data may also come as int16 /
# uint16 bits, E4M3 codes as uint8.
TYPE_BF16, TYPE_F32 = 0, 1
QUANT_NONE, QUANT_E4M3, QUANT_INT8 = 0, 1, 2
SCORES = {"softmax": 0, "sigmoid": 1}

_type_tags = None     # made at the first call (torch is imported lazily)


def _types():
    """torch dtypes and their tags: of floats (moe_type), of codes (moe_quant), of bf16 alone, of float32 alone."""
    global _type_tags
    if _type_tags is None:
        import torch
        bf16 = {torch.bfloat16: TYPE_BF16, torch.int16: TYPE_BF16, torch.uint16: TYPE_BF16}
        f32 = {torch.float32: TYPE_F32}
        _type_tags = ({**f32, **bf16},
                      {torch.float8_e4m3fn: QUANT_E4M3, torch.uint8: QUANT_E4M3, torch.int8: QUANT_INT8}, bf16, f32)
    return _type_tags


_int_types = None


def _ints():
    """torch dtypes of int32 data, and of int8 codes."""
    global _int_types
    if _int_types is None:
        import torch
        _int_types = {torch.int32: 0, torch.uint32: 0}, {torch.int8: 0}
    return _int_types


def _refuse(name, t, shape, types, device):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, {tuple(shape)} is needed")
    if not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous")
    if t.dtype not in types:
        raise ValueError(f"{name} has type {t.dtype}, which this call does not take")
    raise ValueError(f"{name} is on {t.device}, another tensor on device {device}")


def _tag(name, t, shape, types, device):
    """The type tag of tensor t, checked: its shape, dense, its dtype one of `types`, its device."""
    tag = types.get(t.dtype)
    if tag is None or t.shape != shape or not t.is_contiguous() or t.get_device() != device:
        _refuse(name, t, shape, types, device)
    return tag


def _vector(name, t, n, types, device):
    """The same for n elements in any shape."""
    if t.dtype not in types or t.numel() != n or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{name} must be a contiguous tensor of {n} elements of {' or '.join(map(str, types))} on the "
                         f"other tensors' device; it has {t.numel()} of {t.dtype} on {t.device}")


def _rows(name, t, M, n, types, device):
    """The same for M rows of n elements: [M, n], or any shape whose elements follow one another in that order (a first
    dimension of M, or all in one dimension).  A transposed tensor is not that."""
    if t.dtype in types and t.shape == (M, n) and t.is_contiguous() and t.get_device() == device:
        return
    if t.dim() > 1 and t.shape[0] != M:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, {(M, n)} is needed")
    _vector(name, t, M * n, types, device)


def _stream_on(device, stream):
    """The stream's handle; the tensors' device must be torch's current one, where kernels are launched, and the
    stream's."""
    current, handle = _current or _torch_current()
    if device != current():
        raise ValueError(f"the tensors are on device {device}, the current device is {current()}")
    if stream is None:
        return handle(device)
    other = device if isinstance(stream, int) else getattr(stream, "device_index", device)
    if other != device:
        raise ValueError(f"the tensors are on device {device}, the stream on device {other}")
    return _stream(stream)


def moe_add_rmsnorm(x, residual, weight, eps, residual_out, y=None, q=None, scale=None, stream=None):
    """residual_out = residual + x; y = its RMS norm times weight in bf16; q, scale = y's 8-bit codes.

    x [M,H] float32 or bf16; residual [M,H] float32 or bf16, or None (then residual_out gives the type, else x's);
    weight [H] float32 or bf16.  residual_out (may be residual), y and (q, scale) may each be None; q's dtype
    chooses the codes: float8_e4m3fn or uint8 for E4M3, int8 for int8."""
    floats, codes, bf16, f32 = _types()
    shape = x.shape
    M, H = shape
    dev = x.get_device()
    r_type = x_type = _tag("x", x, shape, floats, dev)
    r = ro = yp = qp = sp = None
    q_type = QUANT_NONE
    if residual is not None:
        r_type = _tag("residual", residual, shape, floats, dev)
        r = residual.data_ptr()
    if residual_out is not None:
        t = _tag("residual_out", residual_out, shape, floats, dev)
        if r is not None and t != r_type:
            raise ValueError(f"residual_out has type {residual_out.dtype}, residual {residual.dtype}")
        r_type = t
        ro = residual_out.data_ptr()
    w_type = _tag("weight", weight, shape[1:], floats, dev)
    if y is not None:
        _tag("y", y, shape, bf16, dev)
        yp = y.data_ptr()
    if q is not None:
        q_type = _tag("q", q, shape, codes, dev)
        qp = q.data_ptr()
    if scale is not None:
        _vector("scale", scale, M, f32, dev)
        sp = scale.data_ptr()
    st = _stream_on(dev, stream)
    _check(_lib.moe_add_rmsnorm(M, H, x.data_ptr(), x_type, r, r_type, weight.data_ptr(), w_type, eps, ro, yp, qp,
                                q_type, sp, st),
           "moe_add_rmsnorm")


def router(num_experts: int, topk: int, score: str = "sigmoid", groups: int = 1, group_topk: int = 1,
           group_score: int = 2, renormalise: bool = True, factor: float = 1.0) -> MoeRouterParams:
    """A router that chooses by scores, for moe_route_scores and moe_decode_forward_scored."""
    if score not in SCORES:
        raise ValueError(f"score {score!r} is none of {sorted(SCORES)}")
    return MoeRouterParams(num_experts, topk, SCORES[score], groups, group_topk, group_score, int(renormalise), factor)


def moe_route_scores(rp: MoeRouterParams, logits, bias, topk_ids, topk_w, stream=None):
    """topk_ids [M,K] int32 and topk_w [M,K] float32 of logits [M,E] float32; bias [E] float32 or None."""
    f32 = _types()[3]
    M = logits.shape[0]
    dev = logits.get_device()
    _vector("logits", logits, M * rp.num_experts, f32, dev)
    if bias is not None:
        _vector("bias", bias, rp.num_experts, f32, dev)
        bias = bias.data_ptr()
    _rows("topk_ids", topk_ids, M, rp.topk, _ints()[0], dev)
    _rows("topk_w", topk_w, M, rp.topk, f32, dev)
    st = _stream_on(dev, stream)
    _check(_lib.moe_route_scores(ctypes.byref(rp), M, logits.data_ptr(), bias, topk_ids.data_ptr(), topk_w.data_ptr(),
                                 st),
           "moe_route_scores")


def _held(name, t, n, types, device):
    """The address of a dense tensor of at least n elements of one of `types` on a device (any, where it is None).  Its
    shape is the caller's: M and the layer's sizes are arguments, and a buffer may hold more tokens than M.  An int
    address is taken as it is, and None is left to the call."""
    if t is None or t.__class__ is int:
        return t
    if t.dtype in types and t.numel() >= n and t.is_contiguous() and (device is None or t.get_device() == device):
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous tensor of at least {n} elements of {' or '.join(map(str, types))} on "
                     f"the other tensors' device; it has {t.numel()} of {t.dtype} on {t.device}")


def _codes(name, t, n, device):
    """The same for n bytes of codes or block scales, of any type of one byte."""
    if t is None or t.__class__ is int:
        return t
    if t.nbytes == t.numel() >= n and t.is_contiguous() and (device is None or t.get_device() == device):
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous tensor of at least {n} one-byte elements on the other tensors' device; "
                     f"it has {t.numel()} of {t.dtype} on {t.device}")


def moe_router_logits(shp, M, hidden, router_w, logits, stream=None):
    """logits [M,E] float32 of hidden [M,H] and router_w [E,H], both bf16: the router's part of the layer alone."""
    _, _, bf16, f32 = _types()
    H, E = shp.hidden, shp.num_experts
    dev = next((t.get_device() for t in (logits, hidden, router_w) if t is not None and t.__class__ is not int), None)
    x = _held("hidden", hidden, M * H, bf16, dev)
    wr = _held("router_w", router_w, E * H, bf16, dev)
    lg = _held("logits", logits, M * E, f32, dev)
    st = _stream(stream) if dev is None else _stream_on(dev, stream)
    _check(_lib.moe_router_logits(ctypes.byref(shp), M, x, wr, lg, st), "moe_router_logits")


def moe_decode_forward_scored(shp, rp, M, hidden, router_w, bias, w13, w13_scale, w2, w2_scale, out, ws, shared=None,
                              stream=None):
    """The layer with routing by scores (rp from router()); bias [E] float32 or None; shared as in
    moe_decode_forward_shared."""
    _, _, bf16, f32 = _types()
    H, I, E = shp.hidden, shp.inter, shp.num_experts
    dev = ws.get_device()                                # the device of a workspace, always a tensor
    if not ws.is_contiguous():
        raise ValueError("ws is not contiguous")
    x = _held("hidden", hidden, M * H, bf16, dev)
    wr = _held("router_w", router_w, E * H, bf16, dev)
    if bias is not None and bias.__class__ is not int:
        _vector("bias", bias, E, f32, dev)
        bias = bias.data_ptr()
    n13, ns13, n2, ns2 = I * H, 2 * I * (H // 32), H * I // 2, H * (I // 32)
    c13, s13 = _codes("w13", w13, E * n13, dev), _codes("w13_scale", w13_scale, E * ns13, dev)
    c2, s2 = _codes("w2", w2, E * n2, dev), _codes("w2_scale", w2_scale, E * ns2, dev)
    sh = None
    if shared is not None:
        sizes = (("w13", n13), ("w13_scale", ns13), ("w2", n2), ("w2_scale", ns2))
        if len(shared) == 4:
            shared = [_codes("shared " + name, t, n, dev) for t, (name, n) in zip(shared, sizes)]
        sh = ctypes.byref(_shared(shared))
    o = _held("out", out, M * H, f32, dev)
    _check(_lib.moe_decode_forward_scored(ctypes.byref(shp), ctypes.byref(rp), M, x, wr, bias, c13, s13, c2, s2, sh, o,
                                          ws.data_ptr(), ws.nbytes, _stream_on(dev, stream)),
           "moe_decode_forward_scored")


def moe_int8_quantize(x_bf16, q, scale, stream=None):
    """x_bf16 [rows, cols] -> int8 codes q [rows, cols] and scale [rows]."""
    _, _, bf16, f32 = _types()
    shape = x_bf16.shape
    rows, cols = shape
    dev = x_bf16.get_device()
    _tag("x_bf16", x_bf16, shape, bf16, dev)
    _tag("q", q, shape, _ints()[1], dev)
    _vector("scale", scale, rows, f32, dev)
    st = _stream_on(dev, stream)
    _check(_lib.moe_int8_quantize(x_bf16.data_ptr(), rows, cols, q.data_ptr(), scale.data_ptr(), st),
           "moe_int8_quantize")


def moe_int8_linear(a, a_scale, w, w_scale, out, stream=None):
    """out [M,N] (float32 or bf16) = (a [M,K] int8 times w [N,K] int8 transposed) * a_scale [M] * w_scale [N]."""
    floats, _, _, f32 = _types()
    int8 = _ints()[1]
    M, K = a.shape
    N = w.shape[0]
    dev = a.get_device()
    _vector("a", a, M * K, int8, dev)
    _tag("w", w, (N, K), int8, dev)
    out_type = _tag("out", out, (M, N), floats, dev)
    _vector("a_scale", a_scale, M, f32, dev)
    _vector("w_scale", w_scale, N, f32, dev)
    st = _stream_on(dev, stream)
    _check(_lib.moe_int8_linear(a.data_ptr(), a_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(), M, N, K,
                                out.data_ptr(), out_type, st),
           "moe_int8_linear")


def _path_arg(p):
    return None if p is None else os.fsencode(p)


def moe_jit_build(shp: MoeShape, arch: str = "gfx950", cache_dir=None) -> dict:
    """Compile the kernels of (H, I) for `arch` into the cache (no GPU needed)."""
    r = MoeJitReport()
    _check(_lib.moe_jit_build(ctypes.byref(shp), arch.encode(), _path_arg(cache_dir), ctypes.byref(r)),
           "moe_jit_build")
    return r.as_dict()


def moe_jit_load(shp: MoeShape, cache_dir=None, prefer: bool = False) -> dict:
    """Compile or find (H, I) in the cache and load it on the current device."""
    r = MoeJitReport()
    _check(_lib.moe_jit_load(ctypes.byref(shp), _path_arg(cache_dir), 1 if prefer else 0, ctypes.byref(r)),
           "moe_jit_load")
    return r.as_dict()


def moe_jit_unload(shp: MoeShape) -> int:
    return _lib.moe_jit_unload(ctypes.byref(shp))


def moe_path_info(shp: MoeShape, M: int) -> tuple[int, str]:
    buf = ctypes.create_string_buffer(1024)
    st = _lib.moe_path_info(ctypes.byref(shp), M, buf, len(buf))
    return st, buf.value.decode()


def moe_workspace_sync_status(ws, status, stream=None) -> None:
    """Copy the workspace's sticky wait-error bits into `status` (a device
    int32/uint32 tensor of one element)."""
    _check(_lib.moe_workspace_sync_status(_p(ws), _nbytes(ws), _p(status), _stream(stream)),
           "moe_workspace_sync_status")


def sync_errors(ws) -> int:
    """The workspace's wait-error bits, read back (synchronises the current stream)."""
    import torch
    st = torch.zeros(1, dtype=torch.int32, device=ws.device)
    moe_workspace_sync_status(ws, st)
    return int(st.item())


def moe_set_wait_limit_us(us: int) -> None:
    _lib.moe_set_wait_limit_us(us)


PATH_THREE_KERNELS = 0
PATH_ONE_KERNEL = 1


def moe_set_decode_path(path: int) -> None:
    """Select how M <= 8 runs for later calls: PATH_THREE_KERNELS (default) or
    PATH_ONE_KERNEL (layer_kernel)."""
    _check(_lib.moe_set_decode_path(path), "moe_set_decode_path")


def moe_status_string(status: int) -> str:
    return _lib.moe_status_string(status).decode()


def moe_last_error() -> str:
    return _lib.moe_last_error().decode()


def raw():
    """The underlying ctypes library (for argument-validation tests)."""
    return _lib
