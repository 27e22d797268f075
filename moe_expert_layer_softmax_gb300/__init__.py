"""Python binding of libmoe_gb300.so, the sm_103a MoE expert layer library.

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  Tensors are torch CUDA tensors (used for device memory and streams);
the C entry points have the same names without the `moe_` prefix.  There is no
fallback: if the library is missing or cannot be loaded, every call raises.

Shapes follow include/moe.h: x [T, d] bf16, W_r [E, d] bf16, W_gate/W_up
[E, f, d] bf16, W_down [E, d, f] bf16; dispatched row buffers have
`rows_max(shape)` rows.
"""
from __future__ import annotations

import bisect
import ctypes
import os
import struct
from dataclasses import dataclass

_PKG = os.path.dirname(os.path.abspath(__file__))
# MOE_GB300_CHECKS=1 selects the checks build (device-side bounds checks, see
# moe_checks_read) and guard bands around every buffer allocate() hands out
CHECKS = os.environ.get("MOE_GB300_CHECKS", "") == "1"
LIB_PATH = os.path.join(_PKG, "libmoe_gb300_checks.so" if CHECKS else "libmoe_gb300.so")

BF16, MXFP8 = 0, 1
TILE_M = 128

GEMM_FWD1_SWIGLU = 0
GEMM_FWD2 = 1
GEMM_DGRAD2_SWIGLU = 2
GEMM_DGRAD1 = 3
GEMM_WGRAD2 = 4
GEMM_WGRAD1 = 5
GEMM_WGRAD2_NATURAL = 6   # activation operand as MXFP8 codes + scales, dequantised in the kernel
GEMM_WGRAD1_NATURAL = 7

DEVERR_NONFINITE_LOGIT = 0x1
DEVERR_TIMEOUT = 0x2
DEVERR_BOUNDS = 0x4

_ERRORS = {-1: "MOE_ERR_INVALID", -2: "MOE_ERR_UNSUPPORTED", -3: "MOE_ERR_ALIGN",
           -4: "MOE_ERR_CUDA", -5: "MOE_ERR_NOT_INIT", -6: "MOE_ERR_SCRATCH_LIMIT"}
ERR_NOT_INIT, ERR_SCRATCH_LIMIT = -5, -6

# every symbol the C header declares
EXPORTS = (
    "moe_init", "moe_rows_max", "moe_workspace_size", "moe_clear_error", "moe_read_error",
    "moe_route", "moe_dispatch", "moe_quantize_mxfp8", "moe_grouped_gemm", "moe_combine",
    "moe_combine_bwd", "moe_dispatch_bwd", "moe_router_bwd", "moe_layer_fwd", "moe_layer_bwd",
    "moe_route_noalloc", "moe_dequantize_mxfp8", "moe_build_mx_weights",
    "moe_debug_inject_stall", "moe_profile_start", "moe_profile_stop", "moe_load_balance",
    "moe_checks_read", "moe_few_workspace_size", "moe_few_fwd",
    "moe_add_norm", "moe_add_norm_bwd_workspace_size", "moe_add_norm_bwd", "moe_add_layer_norm",
    "moe_add_layer_norm_bwd_workspace_size", "moe_add_layer_norm_bwd", "moe_dropout", "moe_adamw", "moe_adamw_at",
    "moe_add_norm_at", "moe_add_norm_bwd_at", "moe_add_layer_norm_at", "moe_add_layer_norm_bwd_at", "moe_dropout_at",
    "moe_quantize_w4", "moe_dequantize_w4", "moe_matvec_w4", "moe_experts_w4_workspace_size",
    "moe_experts_w4",
)


class MoEError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} returned {code} ({_ERRORS.get(code, 'unknown')})")
        self.code = code


class Shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d_model", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("d_ff", ctypes.c_int32), ("prec", ctypes.c_int32)]


_vp = ctypes.c_void_p


class GemmArgs(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("tile_offsets", "a0", "a1", "w0", "w1", "aux0", "aux1",
                                   "out0", "out1", "out2", "sfa0", "sfa1", "sfb0", "sfb1",
                                   "out3", "osf0", "osf1")]


MX_WEIGHT_FIELDS = ("gu_q", "gu_s", "down_q", "down_s", "downT_q", "downT_s", "gateT_q",
                    "gateT_s", "upT_q", "upT_s")
MX_BUFFER_FIELDS = ("xd_q", "xd_s", "a_q", "a_s", "dy_q", "dy_s", "dh_q", "dh_s", "du_q",
                    "du_s", "xd_dq", "a_dq")


class MxWeights(ctypes.Structure):
    _fields_ = [(n, _vp) for n in MX_WEIGHT_FIELDS]


class MxBuffers(ctypes.Structure):
    _fields_ = [(n, _vp) for n in MX_BUFFER_FIELDS]


class Saved(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("logits", "topk_idx", "gates", "counts", "offsets",
                                   "tile_offsets", "slot_of_route", "route_of_slot", "xd", "h",
                                   "u", "a", "y", "lb_stats")]


class FwdArgs(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("x", "w_router", "logit_bias", "w_gate", "w_up", "w_down",
                                   "out", "mx_weights", "mx")]


class BwdArgs(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("d_out", "x", "w_router", "w_gate", "w_up", "w_down", "dx",
                                   "dw_router", "dw_gate", "dw_up", "dw_down", "d_gates",
                                   "dlogits", "dy", "dh", "du", "dxd", "mx_weights", "mx")] + \
        [("recompute", ctypes.c_int32), ("lb_coef", ctypes.c_float)]


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the library (once).  Raises if it is missing: there is no fallback."""
    global _lib
    if _lib is not None:
        return _lib
    if CHECKS and path == LIB_PATH:
        from . import _build
        _build.build(checks=True)
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with __graft_entry__.build() "
                           "(the MoE layer has no CPU or eager fallback)")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER
    i32, i64 = ctypes.c_int32, ctypes.c_int64
    sig = {
        "moe_init": [ctypes.c_int],
        "moe_rows_max": [P(Shape), P(ctypes.c_int64)],
        "moe_workspace_size": [P(Shape), P(ctypes.c_size_t)],
        "moe_clear_error": [_vp, _vp],
        "moe_read_error": [_vp, P(i32), _vp],
        "moe_debug_inject_stall": [i32],
        "moe_profile_start": [i32],
        "moe_load_balance": [P(Shape), _vp, _vp, _vp, _vp, _vp],
        "moe_profile_stop": [_vp, _vp],
        "moe_route": [P(Shape)] + [_vp] * 11 + [_vp, _vp],
        "moe_route_noalloc": [P(Shape)] + [_vp] * 11 + [_vp, _vp],
        "moe_dispatch": [P(Shape)] + [_vp] * 7 + [_vp],
        "moe_quantize_mxfp8": [i32, i32, i32, i32, _vp, _vp, _vp, _vp],
        "moe_dequantize_mxfp8": [ctypes.c_int64, i32, _vp, _vp, _vp, _vp],
        "moe_build_mx_weights": [P(Shape), _vp, _vp, _vp, P(MxWeights), _vp],
        "moe_grouped_gemm": [P(Shape), i32, P(GemmArgs), _vp, _vp],
        "moe_combine": [P(Shape)] + [_vp] * 4 + [_vp],
        "moe_combine_bwd": [P(Shape)] + [_vp] * 12 + [_vp],
        "moe_dispatch_bwd": [P(Shape)] + [_vp] * 6 + [_vp],
        "moe_router_bwd": [P(Shape)] + [_vp] * 7 + [_vp],
        "moe_layer_fwd": [P(Shape), P(FwdArgs), P(Saved), _vp, _vp],
        "moe_layer_bwd": [P(Shape), P(BwdArgs), P(Saved), _vp, _vp],
        "moe_checks_read": [P(i32), i32],
        "moe_few_workspace_size": [P(Shape), P(ctypes.c_size_t)],
        "moe_few_fwd": [P(Shape), _vp, _vp, _vp],
        "moe_add_norm": [_vp, _vp],
        "moe_add_norm_bwd_workspace_size": [i64, i32, P(ctypes.c_size_t)],
        "moe_add_norm_bwd": [_vp, _vp, _vp],
        "moe_add_layer_norm": [_vp, _vp],
        "moe_add_layer_norm_bwd_workspace_size": [i64, i32, P(ctypes.c_size_t)],
        "moe_add_layer_norm_bwd": [_vp, _vp, _vp],
        "moe_dropout": [i64, i32, i32, _vp, i64, _vp, i64, ctypes.c_float, ctypes.c_uint64,
                        ctypes.c_uint64, _vp],
        "moe_add_norm_at": [_vp, _vp, _vp],
        "moe_add_norm_bwd_at": [_vp, _vp, _vp, _vp],
        "moe_add_layer_norm_at": [_vp, _vp, _vp],
        "moe_add_layer_norm_bwd_at": [_vp, _vp, _vp, _vp],
        "moe_dropout_at": [i64, i32, i32, _vp, i64, _vp, i64, ctypes.c_float, ctypes.c_uint64,
                           ctypes.c_uint64, _vp, _vp],
        "moe_adamw": [_vp, _vp],
        "moe_adamw_at": [_vp, _vp, _vp],
        "moe_quantize_w4": [i64, i32, i32, i32, _vp, _vp, _vp, _vp],
        "moe_dequantize_w4": [i64, i32, i32, i32, _vp, _vp, _vp, _vp],
        "moe_matvec_w4": [i32] * 5 + [_vp, i64, _vp, _vp, _vp, i64, _vp],
        "moe_experts_w4_workspace_size": [i32] * 5 + [P(ctypes.c_size_t)],
        "moe_experts_w4": [_vp, _vp, _vp],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    _lib = lib
    return lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_raw_stream = None   # (function, device function) giving the current stream's handle


def _stream(stream):
    if stream is None:
        global _raw_stream
        if _raw_stream is None:
            import torch
            c = torch._C
            if hasattr(c, "_cuda_getCurrentRawStream") and hasattr(c, "_cuda_getDevice"):
                # the handle without a Stream object around it (3 us less a call)
                _raw_stream = (c._cuda_getCurrentRawStream, c._cuda_getDevice)
            else:
                _raw_stream = (lambda dev: torch.cuda.current_stream(dev).cuda_stream,
                               torch.cuda.current_device)
        return _raw_stream[0](_raw_stream[1]())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, rc: int):
    if rc != 0:
        raise MoEError(fn, rc)


def shape(T, d, E, k, f, prec=BF16) -> Shape:
    return Shape(int(T), int(d), int(E), int(k), int(f), int(prec))


# ------------------------------------------------------------------ set-up
_inited = set()


def init(device: int | None = None):
    import torch
    dev = torch.cuda.current_device() if device is None else int(device)
    if dev in _inited:
        return
    with torch.cuda.device(dev):
        _check("moe_init", load().moe_init(dev))
    _inited.add(dev)


def rows_max(s: Shape) -> int:
    v = ctypes.c_int64()
    _check("moe_rows_max", load().moe_rows_max(ctypes.byref(s), ctypes.byref(v)))
    return v.value


def workspace_size(s: Shape) -> int:
    v = ctypes.c_size_t()
    _check("moe_workspace_size", load().moe_workspace_size(ctypes.byref(s), ctypes.byref(v)))
    return v.value


def checks_read(reset: bool = True) -> int:
    """moe_checks_read: the OR of the checks build's bounds-check words (0 when
    no index left its buffer); raises MoEError(MOE_ERR_UNSUPPORTED) on the
    normal build."""
    v = ctypes.c_int32()
    _check("moe_checks_read", load().moe_checks_read(ctypes.byref(v), int(bool(reset))))
    return v.value


# ---- guard bands (checks mode): every buffer of allocate() sits between two
# 4 KB bands of a known byte pattern, verified by check_canaries()
GUARD_BYTES = 4096
GUARD_BYTE = 0xA5
_guarded = {}   # id of a handed-out buffer -> its whole allocation (bands included)


def _alloc(shape, dtype, device, zero=False):
    import torch
    if not CHECKS:
        return (torch.zeros if zero else torch.empty)(shape, dtype=dtype, device=device)
    import math
    import weakref
    n = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
    base = torch.full((n + 2 * GUARD_BYTES,), GUARD_BYTE, dtype=torch.uint8, device=device)
    mid = base[GUARD_BYTES:GUARD_BYTES + n]
    if zero:
        mid.zero_()
    out = mid.view(dtype).view(shape)
    key = id(out)
    _guarded[key] = base
    weakref.finalize(out, _guarded.pop, key, None)   # forgotten with the buffer
    return out


def check_canaries() -> list:
    """Checks mode: the guard bands of every live buffer from allocate() still
    hold their pattern.  Returns a description of each band that was written."""
    bad = []
    for base in list(_guarded.values()):
        for name, band in (("front", base[:GUARD_BYTES]), ("back", base[-GUARD_BYTES:])):
            changed = int((band != GUARD_BYTE).sum().item())
            if changed:
                bad.append(f"{changed} byte(s) of the {name} guard of a {base.numel() - 2 * GUARD_BYTES}"
                           f"-byte buffer were written")
    return bad


def clear_error(ws, stream=None):
    _check("moe_clear_error", load().moe_clear_error(_ptr(ws), _stream(stream)))


def debug_inject_stall(mode: int) -> int:
    """Test hook: 1 makes the next grouped-GEMM launches stall on purpose (their
    bounded waits time out and report MOE_DEVERR_TIMEOUT); 0 turns it off."""
    rc = load().moe_debug_inject_stall(int(mode))
    if rc < 0:
        raise MoEError("moe_debug_inject_stall", rc)
    return rc


def load_balance(s: Shape, logits, counts, lb_stats, ws, stream=None):
    """moe_load_balance: lb_stats[0] = LBL, lb_stats[1 + e] = P_e."""
    _check("moe_load_balance", load().moe_load_balance(ctypes.byref(s), _ptr(logits), _ptr(counts),
                                                       _ptr(lb_stats), _ptr(ws), _stream(stream)))


def profile_start(op: int):
    """moe_profile_start: time every following launch of grouped-GEMM `op`."""
    _check("moe_profile_start", load().moe_profile_start(int(op)))


def profile_stop():
    """moe_profile_stop: (summed milliseconds, number of timed launches)."""
    ms = ctypes.c_float(0.0)
    n = ctypes.c_int32(0)
    _check("moe_profile_stop", load().moe_profile_stop(ctypes.byref(ms), ctypes.byref(n)))
    return float(ms.value), int(n.value)


def read_error(ws, stream=None) -> int:
    v = ctypes.c_int32()
    _check("moe_read_error", load().moe_read_error(_ptr(ws), ctypes.byref(v), _stream(stream)))
    return v.value


# ------------------------------------------------------------------ stage calls
def route(s, x, w_router, logit_bias, logits, topk_idx, gates, counts, offsets, tile_offsets,
          slot_of_route, route_of_slot, ws, stream=None):
    _check("moe_route", load().moe_route(
        ctypes.byref(s), _ptr(x), _ptr(w_router), _ptr(logit_bias), _ptr(logits), _ptr(topk_idx),
        _ptr(gates), _ptr(counts), _ptr(offsets), _ptr(tile_offsets), _ptr(slot_of_route),
        _ptr(route_of_slot), _ptr(ws), _stream(stream)))


def route_noalloc(s, x, w_router, logit_bias, logits, topk_idx, gates, counts, offsets,
                  tile_offsets, slot_of_route, route_of_slot, dev_error=None, stream=None):
    """moe_route without a workspace: for callers that cannot allocate device
    memory (see include/moe.h); scratch lives in the library's static array."""
    _check("moe_route_noalloc", load().moe_route_noalloc(
        ctypes.byref(s), _ptr(x), _ptr(w_router), _ptr(logit_bias), _ptr(logits), _ptr(topk_idx),
        _ptr(gates), _ptr(counts), _ptr(offsets), _ptr(tile_offsets), _ptr(slot_of_route),
        _ptr(route_of_slot), _ptr(dev_error), _stream(stream)))


def dispatch(s, x, slot_of_route, counts, tile_offsets, xd, xd_scales=None, stream=None,
             xd_dq=None):
    _check("moe_dispatch", load().moe_dispatch(
        ctypes.byref(s), _ptr(x), _ptr(slot_of_route), _ptr(counts), _ptr(tile_offsets), _ptr(xd),
        _ptr(xd_scales), _ptr(xd_dq), _stream(stream)))


def quantize_mxfp8(batch, rows, cols, block_axis, src, q, scales, stream=None):
    _check("moe_quantize_mxfp8", load().moe_quantize_mxfp8(
        int(batch), int(rows), int(cols), int(block_axis), _ptr(src), _ptr(q), _ptr(scales),
        _stream(stream)))


def dequantize_mxfp8(rows, K, q, scales, out, stream=None):
    _check("moe_dequantize_mxfp8", load().moe_dequantize_mxfp8(
        int(rows), int(K), _ptr(q), _ptr(scales), _ptr(out), _stream(stream)))


def build_mx_weights(s, w_gate, w_up, w_down, cache: dict, stream=None):
    c = MxWeights(**{k: _ptr(cache[k]) for k in MX_WEIGHT_FIELDS})
    _check("moe_build_mx_weights", load().moe_build_mx_weights(
        ctypes.byref(s), _ptr(w_gate), _ptr(w_up), _ptr(w_down), ctypes.byref(c), _stream(stream)))


def grouped_gemm(s, op, ws, stream=None, **kw):
    a = GemmArgs(**{k: _ptr(v) for k, v in kw.items()})
    _check("moe_grouped_gemm", load().moe_grouped_gemm(ctypes.byref(s), int(op), ctypes.byref(a),
                                                       _ptr(ws), _stream(stream)))


def combine(s, y, gates, slot_of_route, out, stream=None):
    _check("moe_combine", load().moe_combine(ctypes.byref(s), _ptr(y), _ptr(gates),
                                             _ptr(slot_of_route), _ptr(out), _stream(stream)))


def combine_bwd(s, d_out, y, gates, topk_idx, slot_of_route, counts, tile_offsets, dy, d_gates,
                dlogits, stream=None, dy_q=None, dy_scales=None):
    _check("moe_combine_bwd", load().moe_combine_bwd(
        ctypes.byref(s), _ptr(d_out), _ptr(y), _ptr(gates), _ptr(topk_idx), _ptr(slot_of_route),
        _ptr(counts), _ptr(tile_offsets), _ptr(dy), _ptr(d_gates), _ptr(dlogits), _ptr(dy_q),
        _ptr(dy_scales), _stream(stream)))


def dispatch_bwd(s, dxd, slot_of_route, topk_idx, dlogits, w_router, dx, stream=None):
    _check("moe_dispatch_bwd", load().moe_dispatch_bwd(
        ctypes.byref(s), _ptr(dxd), _ptr(slot_of_route), _ptr(topk_idx), _ptr(dlogits),
        _ptr(w_router), _ptr(dx), _stream(stream)))


def router_bwd(s, x, dlogits, route_of_slot, counts, tile_offsets, dw_router, ws, stream=None):
    _check("moe_router_bwd", load().moe_router_bwd(
        ctypes.byref(s), _ptr(x), _ptr(dlogits), _ptr(route_of_slot), _ptr(counts),
        _ptr(tile_offsets), _ptr(dw_router), _ptr(ws), _stream(stream)))


def layer_fwd(s, fwd: FwdArgs, saved: Saved, ws, stream=None):
    _check("moe_layer_fwd", load().moe_layer_fwd(ctypes.byref(s), ctypes.byref(fwd),
                                                 ctypes.byref(saved), _ptr(ws), _stream(stream)))


def layer_bwd(s, bwd: BwdArgs, saved: Saved, ws, stream=None):
    _check("moe_layer_bwd", load().moe_layer_bwd(ctypes.byref(s), ctypes.byref(bwd),
                                                 ctypes.byref(saved), _ptr(ws), _stream(stream)))


# ------------------------------------------------------------------ around the layer
# The operators before and after the layer in a block (include/moe.h, "around the
# layer").  These wrappers check what the C entry points cannot see: types, shapes,
# devices and strides of the tensors.  The first call on a device sets it up
# (init()), unless its stream is being captured: then it raises MOE_ERR_NOT_INIT.
DT_BF16, DT_F16, DT_F32 = 0, 1, 2
W4_MAX_ROUTES = 4096
_ADD_NORM = struct.Struct("@qiiii" + "Pq" * 2 + "P" + "Pq" * 2 + "PPPP" + "QQff")
_ADD_NORM_BWD = struct.Struct("@qiiii" + "Pq" * 3 + "PP" + "Pq" * 2 + "P" + "QQf0q")
_ADD_LAYER_NORM = struct.Struct("@qiiii" + "Pq" * 2 + "PP" + "Pq" * 2 + "PPPPP" + "QQff")
_ADD_LAYER_NORM_BWD = struct.Struct("@qiiii" + "Pq" * 3 + "PPP" + "Pq" * 2 + "PP" + "QQf0q")
_ADAMW_TENSOR = struct.Struct("@7Pq")
_ADAMW = struct.Struct("@P4iPPP5dqQQ")
_FEW = struct.Struct("@10P")
_EXPERTS_W4 = struct.Struct("@7i" + "P" * 10)
_torch = None
_dtypes = {}
_several = False   # more than one device: tensors may lie on another than the current one


def _dtype(t, what):
    dt = _dtypes.get(t.dtype)
    if dt is not None:
        return dt
    global _torch, _several
    if _torch is None:
        import torch
        _torch, _several = torch, torch.cuda.device_count() > 1
        _dtypes.update({torch.bfloat16: DT_BF16, torch.float16: DT_F16, torch.float32: DT_F32})
        return _dtype(t, what)
    raise TypeError(f"{what}: {t.dtype} is not bf16, fp16 or fp32")


def _capturing(handle):
    """Whether the current stream or the one of this handle is being captured."""
    import torch
    if torch.cuda.is_current_stream_capturing():
        return True
    if not handle:   # the legacy default stream takes no part in a capture
        return False
    with torch.cuda.stream(torch.cuda.ExternalStream(handle)):
        return torch.cuda.is_current_stream_capturing()


def _failed(fn, rc, *args):
    """What follows a call that returned `rc`, not MOE_OK, for `args` (the stream
    last): on a device that has not been set up, set it up and call again."""
    if rc == ERR_NOT_INIT and not _capturing(args[-1]):
        init()
        rc = getattr(load(), fn)(*args)
    _check(fn, rc)


def _shape(x):
    """(rows, columns) of a tensor whose axes before the last are rows."""
    d = x.size(-1)
    return (x.numel() // d if d else 0), d


def _elsewhere(t):
    """Whether a CUDA tensor lies on another device than the current one, whose stream
    and kernels a call takes."""
    return t.get_device() != _torch.cuda.current_device()


def _matrix(t, what, rows, cols, dtype):
    """(address, row stride) of a matrix on the device, its last axis contiguous;
    axes before the last one are rows (more than one of them: contiguous)."""
    if t is None:
        return 0, 0
    if not t.is_cuda:
        raise ValueError(f"{what}: not a CUDA tensor")
    if _several and _elsewhere(t):
        raise ValueError(f"{what}: on {t.device}, not on the current device")
    if t.dtype is not dtype:
        raise TypeError(f"{what}: {t.dtype}, expected {dtype}")
    if t.numel() != rows * cols or t.size(-1) != cols:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {rows} rows of {cols}")
    if t.is_contiguous():
        return t.data_ptr(), cols
    if t.dim() == 2 and t.stride(1) == 1:
        return t.data_ptr(), t.stride(0)
    raise ValueError(f"{what}: the last axis has to be contiguous (and more than two axes all of it)")


def _flat(t, what, numel, dtype, at_least=False):
    """Address of a contiguous tensor of `numel` elements (or more)."""
    if t is None:
        return 0
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what}: not a contiguous CUDA tensor")
    if _several and _elsewhere(t):
        raise ValueError(f"{what}: on {t.device}, not on the current device")
    if t.dtype is not dtype:
        raise TypeError(f"{what}: {t.dtype}, expected {dtype}")
    if t.numel() != numel and not (at_least and t.numel() > numel):
        raise ValueError(f"{what}: {t.numel()} elements, expected {numel}")
    return t.data_ptr()


def _call_at(fn, offset_dev, *args):
    """The form of a call (its arguments, the stream last) that adds `offset_dev`, an int64
    tensor of one element, to the offset."""
    fn, args = fn + "_at", (*args[:-1], _flat(offset_dev, "offset_dev", 1, _torch.int64), args[-1])
    rc = getattr(load(), fn)(*args)
    if rc:
        _failed(fn, rc, *args)


def add_norm(x, weight, y, residual=None, h=None, rstd=None, eps=1e-5, p=0.0, seed=0, offset=0,
             y_q=None, y_scales=None, y_dq=None, stream=None, offset_dev=None):
    """moe_add_norm: h = residual + dropout(x), y = h * rstd * weight.  y=None with
    y_q, y_scales (and y_dq): the MXFP8 output, buffers of roundup(rows, 128) rows.
    offset_dev, here and below: a CUDA int64 tensor of one element that is added to offset
    when the kernel runs (captured graphs whose replays draw masks of their own)."""
    xt = x.dtype
    dt = _dtype(x, "x")
    rows, d = _shape(x)
    px, ld_x = _matrix(x, "x", rows, d, xt)
    like = residual if residual is not None else h   # the stream's type
    st = xt if like is None else like.dtype
    pr, ld_r = _matrix(residual, "residual", rows, d, st)
    ph, ld_h = _matrix(h, "h", rows, d, st)
    py, ld_y = _matrix(y, "y", rows, d, xt)
    pq = ps = pd = 0
    if y_q is not None or y_scales is not None or y_dq is not None:
        pad = (rows + 127) // 128 * 128
        pq = _flat(y_q, "y_q", pad * d, _torch.uint8, True)
        ps = _flat(y_scales, "y_scales", pad * d // 32, _torch.uint8, True)
        pd = _flat(y_dq, "y_dq", pad * d, _torch.bfloat16, True)
    args = _ADD_NORM.pack(
        rows, d, dt, dt if like is None else _dtype(like, "residual"), _dtype(weight, "weight"),
        px, ld_x, pr, ld_r, _flat(weight, "weight", d, weight.dtype), ph, ld_h, py, ld_y,
        _flat(rstd, "rstd", rows, _torch.float32), pq, ps, pd, seed, offset, eps, p)
    st = _stream(stream)
    if offset_dev is not None:
        return _call_at("moe_add_norm", offset_dev, args, st)
    rc = load().moe_add_norm(args, st)
    if rc:
        _failed("moe_add_norm", rc, args, st)


def add_norm_bwd_workspace(rows, d) -> int:
    """Bytes of workspace that add_norm_bwd needs for dw."""
    v = ctypes.c_size_t()
    _check("moe_add_norm_bwd_workspace_size",
           load().moe_add_norm_bwd_workspace_size(int(rows), int(d), ctypes.byref(v)))
    return v.value


def add_norm_bwd(dy, h, rstd, weight, dres=None, dh=None, dx=None, dw=None, ws=None, p=0.0, seed=0,
                 offset=0, stream=None, offset_dev=None):
    """moe_add_norm_bwd: dh (gradient of the stream), dx (of the dropped input), dw."""
    xt, ht = dy.dtype, h.dtype
    dt = _dtype(dy, "dy")
    rows, d = _shape(dy)
    pdy, ld_dy = _matrix(dy, "dy", rows, d, xt)
    ph, ld_h = _matrix(h, "h", rows, d, ht)
    pdr, ld_dr = _matrix(dres, "dres", rows, d, ht)
    pdh, ld_dh = _matrix(dh, "dh", rows, d, ht)
    pdx, ld_dx = _matrix(dx, "dx", rows, d, xt)
    pws = None
    if dw is not None:
        pws = _flat(ws, "ws", add_norm_bwd_workspace(rows, d), _torch.uint8, True) or None
    args = _ADD_NORM_BWD.pack(
        rows, d, dt, _dtype(h, "h"), _dtype(weight, "weight"), pdy, ld_dy, ph, ld_h, pdr, ld_dr,
        _flat(rstd, "rstd", rows, _torch.float32), _flat(weight, "weight", d, weight.dtype),
        pdh, ld_dh, pdx, ld_dx, _flat(dw, "dw", d, _torch.float32), seed, offset, p)
    st = _stream(stream)
    if offset_dev is not None:
        return _call_at("moe_add_norm_bwd", offset_dev, args, pws, st)
    rc = load().moe_add_norm_bwd(args, pws, st)
    if rc:
        _failed("moe_add_norm_bwd", rc, args, pws, st)


def add_layer_norm(x, weight, bias, y, residual=None, h=None, mean=None, rstd=None, eps=1e-5, p=0.0, seed=0, offset=0,
                   y_q=None, y_scales=None, y_dq=None, stream=None, offset_dev=None):
    """moe_add_layer_norm: h = residual + dropout(x), y = (h - mean) * rstd * weight + bias
    (bias=None: none).  y=None with y_q, y_scales (and y_dq): the MXFP8 output, buffers
    of roundup(rows, 128) rows."""
    xt = x.dtype
    dt = _dtype(x, "x")
    rows, d = _shape(x)
    px, ld_x = _matrix(x, "x", rows, d, xt)
    like = residual if residual is not None else h   # the stream's type
    st = xt if like is None else like.dtype
    pr, ld_r = _matrix(residual, "residual", rows, d, st)
    ph, ld_h = _matrix(h, "h", rows, d, st)
    py, ld_y = _matrix(y, "y", rows, d, xt)
    pq = ps = pd = 0
    if y_q is not None or y_scales is not None or y_dq is not None:
        pad = (rows + 127) // 128 * 128
        pq = _flat(y_q, "y_q", pad * d, _torch.uint8, True)
        ps = _flat(y_scales, "y_scales", pad * d // 32, _torch.uint8, True)
        pd = _flat(y_dq, "y_dq", pad * d, _torch.bfloat16, True)
    f32 = _torch.float32
    args = _ADD_LAYER_NORM.pack(
        rows, d, dt, dt if like is None else _dtype(like, "residual"), _dtype(weight, "weight"),
        px, ld_x, pr, ld_r, _flat(weight, "weight", d, weight.dtype), _flat(bias, "bias", d, weight.dtype), ph, ld_h,
        py, ld_y, _flat(mean, "mean", rows, f32), _flat(rstd, "rstd", rows, f32), pq, ps, pd, seed, offset, eps, p)
    st = _stream(stream)
    if offset_dev is not None:
        return _call_at("moe_add_layer_norm", offset_dev, args, st)
    rc = load().moe_add_layer_norm(args, st)
    if rc:
        _failed("moe_add_layer_norm", rc, args, st)


def add_layer_norm_bwd_workspace(rows, d) -> int:
    """Bytes of workspace that add_layer_norm_bwd needs for dw and db."""
    v = ctypes.c_size_t()
    _check("moe_add_layer_norm_bwd_workspace_size",
           load().moe_add_layer_norm_bwd_workspace_size(int(rows), int(d), ctypes.byref(v)))
    return v.value


def add_layer_norm_bwd(dy, h, mean, rstd, weight, dres=None, dh=None, dx=None, dw=None, db=None, ws=None, p=0.0, seed=0,
                       offset=0, stream=None, offset_dev=None):
    """moe_add_layer_norm_bwd: dh (gradient of the stream), dx (of the dropped input),
    dw and db."""
    xt, ht = dy.dtype, h.dtype
    dt = _dtype(dy, "dy")
    rows, d = _shape(dy)
    pdy, ld_dy = _matrix(dy, "dy", rows, d, xt)
    ph, ld_h = _matrix(h, "h", rows, d, ht)
    pdr, ld_dr = _matrix(dres, "dres", rows, d, ht)
    pdh, ld_dh = _matrix(dh, "dh", rows, d, ht)
    pdx, ld_dx = _matrix(dx, "dx", rows, d, xt)
    pws = None
    if dw is not None or db is not None:
        pws = _flat(ws, "ws", add_layer_norm_bwd_workspace(rows, d), _torch.uint8, True) or None
    f32 = _torch.float32
    args = _ADD_LAYER_NORM_BWD.pack(
        rows, d, dt, _dtype(h, "h"), _dtype(weight, "weight"), pdy, ld_dy, ph, ld_h, pdr, ld_dr,
        _flat(mean, "mean", rows, f32), _flat(rstd, "rstd", rows, f32), _flat(weight, "weight", d, weight.dtype),
        pdh, ld_dh, pdx, ld_dx, _flat(dw, "dw", d, f32), _flat(db, "db", d, f32), seed, offset, p)
    st = _stream(stream)
    if offset_dev is not None:
        return _call_at("moe_add_layer_norm_bwd", offset_dev, args, pws, st)
    rc = load().moe_add_layer_norm_bwd(args, pws, st)
    if rc:
        _failed("moe_add_layer_norm_bwd", rc, args, pws, st)


def dropout(x, y, p, seed, offset=0, stream=None, offset_dev=None):
    """moe_dropout: y = dropout(x), the mask a function of (seed, offset, row,
    column); the backward is the same call on the gradient."""
    dt = _dtype(x, "x")
    rows, d = _shape(x)
    px, ld_x = _matrix(x, "x", rows, d, x.dtype)
    py, ld_y = _matrix(y, "y", rows, d, x.dtype)
    args = (rows, d, dt, px, ld_x, py, ld_y, p, seed, offset, _stream(stream))
    if offset_dev is not None:
        return _call_at("moe_dropout", offset_dev, *args)
    rc = load().moe_dropout(*args)
    if rc:
        _failed("moe_dropout", rc, *args)


class AdamWList:
    """The tensors of moe_adamw, checked and laid out once (adamw_list).  It holds them,
    and a step works on the memory that they had when the list was made."""

    __slots__ = ("tensors", "n", "types", "device", "held")


ADAMW_BLOCK = 128   # values that share a scale of the 8-bit states


def adamw_list(params, grads, exp_avg, exp_avg_sq, master=None) -> AdamWList:
    """Contiguous CUDA tensors of one device, four (with master five) lists of the same
    length.  An entry of exp_avg and exp_avg_sq is an fp32 tensor or, for states in 8 bits,
    a pair (uint8 codes, fp32 scales of ADAMW_BLOCK values each); all are of one kind, as
    are all params' types and all grads'."""
    params, grads, exp_avg, exp_avg_sq = list(params), list(grads), list(exp_avg), list(exp_avg_sq)
    master = None if master is None else list(master)
    n = len(params)
    if any(len(v) != n for v in (grads, exp_avg, exp_avg_sq)) or (master is not None and len(master) != n):
        raise ValueError("adamw_list: lists of different lengths")
    lst = AdamWList()
    lst.n, lst.device = n, None
    if n == 0:
        lst.tensors, lst.types, lst.held = b"", (DT_F32, DT_F32, 32), ()
        return lst
    pt, gt, small = params[0].dtype, grads[0].dtype, isinstance(exp_avg[0], (tuple, list))
    lst.types = (_dtype(params[0], "params"), _dtype(grads[0], "grads"), 8 if small else 32)
    dev = params[0].get_device()
    packed, written, read, held = [], [], [], []

    def take(t, what, numel, dtype):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{what}: not a contiguous CUDA tensor")
        if t.get_device() != dev:
            raise ValueError(f"{what}: on {t.device}, the first parameter on device {dev}")
        if t.dtype is not dtype:
            raise TypeError(f"{what}: {t.dtype}, expected {dtype}")
        if t.numel() != numel:
            raise ValueError(f"{what}: {t.numel()} elements, expected {numel}")
        held.append(t)
        at = t.data_ptr()
        if numel:
            (read if what == "grads" else written).append((at, at + numel * t.element_size(), what))
        return at

    f32, u8 = _torch.float32, _torch.uint8
    for i in range(n):
        numel = params[i].numel()
        states, scales = [], []
        for s, what in ((exp_avg[i], "exp_avg"), (exp_avg_sq[i], "exp_avg_sq")):
            if isinstance(s, (tuple, list)) != small:
                raise TypeError(f"{what}: states in 8 and in 32 bits in one list")
            if small:
                states.append(take(s[0], what, numel, u8))
                scales.append(take(s[1], what + " scales", (numel + ADAMW_BLOCK - 1) // ADAMW_BLOCK, f32))
            else:
                states.append(take(s, what, numel, f32))
                scales.append(0)
        packed.append(_ADAMW_TENSOR.pack(
            take(params[i], "params", numel, pt), take(grads[i], "grads", numel, gt),
            0 if master is None else take(master[i], "master", numel, f32), *states, *scales, numel))
    written.sort()
    for (_, end, a), (start, _, b) in zip(written, written[1:]):
        if start < end:
            raise ValueError(f"adamw_list: memory of {a} and {b} overlaps")
    starts = [start for start, _, _ in written]
    for start, end, _ in read:   # the last range that begins before its end
        at = bisect.bisect_left(starts, end) - 1
        if at >= 0 and written[at][1] > start:
            raise ValueError(f"adamw_list: memory of grads and {written[at][2]} overlaps")
    lst.tensors, lst.device, lst.held = b"".join(packed), dev, tuple(held)
    return lst


def adamw(tensors: AdamWList, lr, step, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, grad_scale=None, seed=0,
          offset=0, stream=None, offset_dev=None):
    """moe_adamw: one step on every tensor of the list.  lr (fp32) and step (int64, from 1)
    are numbers or CUDA tensors of one element, read when the kernel runs; grad_scale: a
    CUDA fp32 tensor of one element that the gradients are multiplied with.  seed and
    offset choose the numbers of drawn roundings: another offset for each step.  A captured
    step gets it from offset_dev, a CUDA int64 tensor of one element (the step's own will
    do) that is added to offset when the kernel runs."""
    lst = tensors
    if lst.n == 0:
        return
    if _several and lst.device != _torch.cuda.current_device():
        raise ValueError(f"adamw: tensors on device {lst.device}, not on the current device")
    plr = pstep = 0
    if not isinstance(lr, (int, float)):
        plr, lr = _flat(lr, "lr", 1, _torch.float32), 0.0
    if not isinstance(step, int):
        pstep, step = _flat(step, "step", 1, _torch.int64), 1
    host = ctypes.c_char_p(lst.tensors)
    args = _ADAMW.pack(ctypes.cast(host, _vp).value, lst.n, *lst.types, _flat(grad_scale, "grad_scale", 1, _torch.float32),
                       plr, pstep, lr, beta1, beta2, eps, weight_decay, step, seed, offset)
    st = _stream(stream)
    if offset_dev is not None:
        return _call_at("moe_adamw", offset_dev, args, st)
    rc = load().moe_adamw(args, st)
    if rc:
        _failed("moe_adamw", rc, args, st)


def _w4(q, scales, what):
    """(rows, K, group) of 4-bit weights, from the shapes of codes and scales."""
    _dtype(scales, what)
    if q.dtype is not _torch.uint8:
        raise TypeError(f"{what}: codes are {q.dtype}, expected uint8")
    half, ng = q.size(-1), scales.size(-1)
    K, rows = 2 * half, (q.numel() // half if half else 0)
    if ng == 0 or K % ng or q.shape[:-1] != scales.shape[:-1]:
        raise ValueError(f"{what}: codes {tuple(q.shape)} and scales {tuple(scales.shape)} do not belong together")
    if not (q.is_cuda and scales.is_cuda and q.is_contiguous() and scales.is_contiguous()):
        raise ValueError(f"{what}: not contiguous CUDA tensors")
    if _several and (_elsewhere(q) or _elsewhere(scales)):
        raise ValueError(f"{what}: codes on {q.device}, scales on {scales.device}, not on the current device")
    return rows, K, K // ng


def quantize_w4(src, q, scales, stream=None):
    """moe_quantize_w4: bf16 or fp16 weights [..., K] to codes [..., K/2] and scales
    [..., K/G] of the same type."""
    rows, K, g = _w4(q, scales, "quantize_w4")
    ps = _flat(src, "src", rows * K, scales.dtype)
    args = (rows, K, g, _dtype(src, "src"), ps, q.data_ptr(), scales.data_ptr(), _stream(stream))
    rc = load().moe_quantize_w4(*args)
    if rc:
        _failed("moe_quantize_w4", rc, *args)


def dequantize_w4(q, scales, out, stream=None):
    """moe_dequantize_w4: the weights that codes and scales stand for, fp32."""
    rows, K, g = _w4(q, scales, "dequantize_w4")
    po = _flat(out, "out", rows * K, _torch.float32)
    args = (rows, K, g, _dtype(scales, "scales"), q.data_ptr(), scales.data_ptr(), po, _stream(stream))
    rc = load().moe_dequantize_w4(*args)
    if rc:
        _failed("moe_dequantize_w4", rc, *args)


def matvec_w4(x, q, scales, y, stream=None):
    """moe_matvec_w4: y [M, N] = x [M, K] times the 4-bit weights [N, K] transposed."""
    N, K, g = _w4(q, scales, "matvec_w4")
    dt = scales.dtype
    M = x.numel() // K if K else 0
    px, ld_x = _matrix(x, "x", M, K, dt)
    py, ld_y = _matrix(y, "y", M, N, dt)
    args = (M, N, K, g, _dtypes[dt], px, ld_x, q.data_ptr(), scales.data_ptr(), py, ld_y, _stream(stream))
    rc = load().moe_matvec_w4(*args)
    if rc:
        _failed("moe_matvec_w4", rc, *args)


def experts_w4_workspace(T, d, E, k, f) -> int:
    """Bytes of workspace that experts_w4 needs (its first word is the error word)."""
    v = ctypes.c_size_t()
    _check("moe_experts_w4_workspace_size", load().moe_experts_w4_workspace_size(
        int(T), int(d), int(E), int(k), int(f), ctypes.byref(v)))
    return v.value


def experts_w4(x, topk_idx, gates, w: dict, out, ws, stream=None):
    """moe_experts_w4: the SwiGLU experts on 4-bit weights for a few tokens.  `w`
    holds gate_q, gate_s, up_q, up_s [E, f, ...] and down_q, down_s [E, d, ...];
    an index of -1 in topk_idx stands for no expert."""
    T, k = topk_idx.shape
    gq, uq, dq = w["gate_q"], w["up_q"], w["down_q"]
    gs, us, ds = w["gate_s"], w["up_s"], w["down_s"]
    E, f = gq.size(0), gq.size(1)
    d = x.size(-1)
    shapes = (_w4(gq, gs, "gate"), _w4(uq, us, "up"), _w4(dq, ds, "down"))
    g = shapes[0][2]
    if shapes != ((E * f, d, g), (E * f, d, g), (E * d, f, g)):
        raise ValueError(f"experts_w4: weights {shapes} do not fit E={E}, d={d}, f={f}")
    dt = x.dtype
    if gs.dtype is not dt or us.dtype is not dt or ds.dtype is not dt:
        raise TypeError("experts_w4: scales of another type than x")
    args = _EXPERTS_W4.pack(
        T, d, E, k, f, g, _dtype(x, "x"), _flat(x, "x", T * d, dt),
        _flat(topk_idx, "topk_idx", T * k, _torch.int32), _flat(gates, "gates", T * k, _torch.float32),
        gq.data_ptr(), gs.data_ptr(), uq.data_ptr(), us.data_ptr(), dq.data_ptr(), ds.data_ptr(),
        _flat(out, "out", T * d, dt))
    pws = _flat(ws, "ws", experts_w4_workspace(T, d, E, k, f), _torch.uint8, True)
    st = _stream(stream)
    rc = load().moe_experts_w4(args, pws, st)
    if rc:
        _failed("moe_experts_w4", rc, args, pws, st)


# ------------------------------------------------------------------ a few tokens
FEW_MAX_TOKENS = 64


def few_workspace(s: Shape) -> int:
    """Bytes of workspace that forward_few needs (its first word is the error word)."""
    v = ctypes.c_size_t()
    _check("moe_few_workspace_size", load().moe_few_workspace_size(ctypes.byref(s), ctypes.byref(v)))
    return v.value


def forward_few(s: Shape, x, w_router, logit_bias, w_gate, w_up, w_down, out, ws, topk_idx=None, gates=None, logits=None,
                stream=None):
    """moe_few_fwd: the layer's forward for at most FEW_MAX_TOKENS tokens, in two kernels.
    With w_router topk_idx, gates and logits are outputs (or None); without, topk_idx and
    gates are the routing (-1: no expert)."""
    if _torch is None:
        _dtype(x, "x")
    T, d, E, k, f = s.T, s.d_model, s.n_experts, s.top_k, s.d_ff
    bf, f32 = _torch.bfloat16, _torch.float32
    args = _FEW.pack(
        _flat(x, "x", T * d, bf), _flat(w_router, "w_router", E * d, bf), _flat(logit_bias, "logit_bias", T * E, f32),
        _flat(w_gate, "w_gate", E * f * d, bf), _flat(w_up, "w_up", E * f * d, bf), _flat(w_down, "w_down", E * d * f, bf),
        _flat(logits, "logits", T * E, f32), _flat(topk_idx, "topk_idx", T * k, _torch.int32),
        _flat(gates, "gates", T * k, f32), _flat(out, "out", T * d, bf))
    pws = _flat(ws, "ws", few_workspace(s), _torch.uint8, True)
    st = _stream(stream)
    rc = load().moe_few_fwd(ctypes.byref(s), args, pws, st)
    if rc:
        _failed("moe_few_fwd", rc, ctypes.byref(s), args, pws, st)


# ------------------------------------------------------------------ buffers
@dataclass
class LayerBuffers:
    """Caller-owned device buffers of one layer shape (torch allocates them)."""

    shape: Shape
    rows_max: int
    ws: object
    saved: dict
    grads: dict
    mx_weights: dict | None = None
    mx: dict | None = None

    def saved_struct(self) -> Saved:
        return Saved(**{k: _ptr(v) for k, v in self.saved.items()})

    def mx_structs(self):
        """(MxWeights, MxBuffers) ctypes structs, or (None, None) in BF16 mode.
        The structs are kept on the object so their addresses stay valid."""
        if self.mx is None:
            return None, None
        self._mxw = MxWeights(**{k: _ptr(self.mx_weights[k]) for k in MX_WEIGHT_FIELDS})
        self._mxb = MxBuffers(**{k: _ptr(self.mx.get(k)) for k in MX_BUFFER_FIELDS})
        return ctypes.addressof(self._mxw), ctypes.addressof(self._mxb)


def allocate(s: Shape, device=None, with_grads: bool = True,
             load_balance: bool = False) -> LayerBuffers:
    """Allocate every buffer moe_layer_fwd / moe_layer_bwd need for shape `s`
    (with load_balance, saved["lb_stats"] receives the forward's
    load-balancing statistics)."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device() if device is None else device)
    T, d, E, k, f = s.T, s.d_model, s.n_experts, s.top_k, s.d_ff
    n = rows_max(s)
    bf = dict(dtype=torch.bfloat16, device=dev)
    i32 = dict(dtype=torch.int32, device=dev)
    f32 = dict(dtype=torch.float32, device=dev)
    ws = _alloc((workspace_size(s),), torch.uint8, dev, zero=True)
    u8 = dict(dtype=torch.uint8, device=dev)
    mx = s.prec == MXFP8

    def new(*shape, dtype, device):   # guard bands around it in checks mode
        return _alloc(shape, dtype, device)

    saved = {
        "logits": new(T, E, **f32), "topk_idx": new(T, k, **i32),
        "gates": new(T, k, **f32), "counts": new(E, **i32),
        "offsets": new(E + 1, **i32), "tile_offsets": new(E + 1, **i32),
        "slot_of_route": new(T * k, **i32), "route_of_slot": new(n, **i32),
        "xd": None if mx else new(n, d, **bf), "h": new(n, f, **bf),
        "u": new(n, f, **bf), "a": None if mx else new(n, f, **bf),
        "y": new(n, d, **bf),
        "lb_stats": new(E + 1, **f32) if load_balance else None,
    }
    grads = {}
    if with_grads:
        grads = {
            "dx": new(T, d, **bf), "dw_router": new(E, d, **f32),
            "dw_gate": new(E, f, d, **f32), "dw_up": new(E, f, d, **f32),
            "dw_down": new(E, d, f, **f32), "d_gates": new(T, k, **f32),
            "dlogits": new(T, E, **f32), "dy": new(n, d, **bf),
            "dh": new(n, f, **bf), "du": new(n, f, **bf),
            "dxd": new(n, d, **bf),
        }
    mxw = mxb = None
    if mx:
        mxw = {"gu_q": new(E, 2 * f, d, **u8), "gu_s": new(E * 2 * f * d // 32, **u8),
               "down_q": new(E, d, f, **u8), "down_s": new(E * d * f // 32, **u8),
               "downT_q": new(E, f, d, **u8), "downT_s": new(E * f * d // 32, **u8),
               "gateT_q": new(E, d, f, **u8), "gateT_s": new(E * d * f // 32, **u8),
               "upT_q": new(E, d, f, **u8), "upT_s": new(E * d * f // 32, **u8)}
        mxb = {"xd_q": new(n, d, **u8), "xd_s": new(n * d // 32, **u8),
               "a_q": new(n, f, **u8), "a_s": new(n * f // 32, **u8)}
        if with_grads:
            mxb.update({"dy_q": new(n, d, **u8), "dy_s": new(n * d // 32, **u8),
                        "dh_q": new(n, f, **u8), "dh_s": new(n * f // 32, **u8),
                        "du_q": new(n, f, **u8), "du_s": new(n * f // 32, **u8),
                        "xd_dq": new(n, d, **bf), "a_dq": new(n, f, **bf)})
    return LayerBuffers(s, n, ws, saved, grads, mxw, mxb)


def adamw_states(params, bits=32):
    """(exp_avg, exp_avg_sq) for adamw_list: zeros for each parameter, fp32 or (bits=8)
    pairs of codes and scales."""
    import torch
    if bits not in (8, 32):
        raise ValueError(f"adamw_states: states of {bits} bits")

    def state(p):
        n, dev = p.numel(), p.device
        if bits == 32:
            return _alloc((n,), torch.float32, dev, zero=True)
        return (_alloc((n,), torch.uint8, dev, zero=True),
                _alloc(((n + ADAMW_BLOCK - 1) // ADAMW_BLOCK,), torch.float32, dev, zero=True))
    return [state(p) for p in params], [state(p) for p in params]


def layer_adamw(buf: LayerBuffers, w_router, w_gate, w_up, w_down, bits=32, master=True) -> AdamWList:
    """What adamw() steps after backward(buf, ...): the layer's weights (w_router may be
    None) with the gradients that the backward leaves in buf.grads, new states of `bits`
    bits and, with `master`, fp32 copies of the weights as they are now.  (With MXFP8
    shapes build_mx_weights follows each step.)"""
    g = buf.grads
    pairs = [(w_router, g["dw_router"])] if w_router is not None else []
    pairs += [(w_gate, g["dw_gate"]), (w_up, g["dw_up"]), (w_down, g["dw_down"])]
    params, grads = [p for p, _ in pairs], [v for _, v in pairs]
    copies = None
    if master:
        import torch
        copies = [_alloc((p.numel(),), torch.float32, p.device) for p in params]
        for c, p in zip(copies, params):
            c.copy_(p.view(-1))
    return adamw_list(params, grads, *adamw_states(params, bits), master=copies)


def forward(buf: LayerBuffers, x, w_router, logit_bias, w_gate, w_up, w_down, out, stream=None):
    """moe_layer_fwd.  MXFP8 shapes use buf.mx_weights (fill them with
    build_mx_weights whenever the bf16 weights change)."""
    mw, mb = buf.mx_structs()
    fa = FwdArgs(x=_ptr(x), w_router=_ptr(w_router), logit_bias=_ptr(logit_bias),
                 w_gate=_ptr(w_gate), w_up=_ptr(w_up), w_down=_ptr(w_down), out=_ptr(out),
                 mx_weights=mw, mx=mb)
    layer_fwd(buf.shape, fa, buf.saved_struct(), buf.ws, stream)


def backward(buf: LayerBuffers, d_out, x, w_router, w_gate, w_up, w_down, stream=None,
             recompute: bool = False, lb_coef: float = 0.0):
    """moe_layer_bwd.  recompute=True re-runs dispatch and both expert GEMMs
    from x and the saved routing metadata instead of reading the saved
    activations; lb_coef adds lb_coef * LBL (the load-balancing scalar) to the
    loss."""
    g = buf.grads
    mw, mb = buf.mx_structs()
    ba = BwdArgs(d_out=_ptr(d_out), x=_ptr(x), w_router=_ptr(w_router), w_gate=_ptr(w_gate),
                 w_up=_ptr(w_up), w_down=_ptr(w_down), mx_weights=mw, mx=mb,
                 recompute=1 if recompute else 0, lb_coef=float(lb_coef),
                 **{k: _ptr(v) for k, v in g.items()})
    layer_bwd(buf.shape, ba, buf.saved_struct(), buf.ws, stream)
