"""Python binding of the Strata MoE layer library (libstrata_moe.so).

Argument marshalling only: every function forwards to the C entry point of
the same name declared in include/strata_moe.h, and every step of the layer
runs in the library's CUDA kernels.  PyTorch is used only for device memory
and streams in the torch-tensor functions and the `Layer` convenience wrapper.
There is no fallback: if the shared library has not been built, importing this
package raises.

Streams.  The functions named like C entry points take a raw pointer (None: the
legacy default stream).  The torch-tensor functions and `Layer` take a torch
stream; without one they run on torch's current stream of their tensors' device,
so that they follow what made their inputs and become part of a graph that is
being captured.  With one, the caller orders it with the streams that make the
inputs and use the outputs.  A layer has one workspace and serves one call at a
time: calls of a layer on two streams have to be ordered by the caller.
"""
from __future__ import annotations

import ctypes as C
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
# STRATA_MOE_CHECKED=1 loads the checked build instead (every device-side
# gather/scatter index tested; a bad one reports STRATA_ERR_BOUNDS)
LIB_PATH = os.path.join(_HERE, "libstrata_moe_checked.so" if os.environ.get("STRATA_MOE_CHECKED") == "1"
                        else "libstrata_moe.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: the CUDA library must be built first "
        "(python quantized_expert_ffn_04_b200/build.py, or __graft_entry__.build())")

_lib = C.CDLL(LIB_PATH)

STRATA_OK, STRATA_ERR_INVALID_ARG, STRATA_ERR_UNSUPPORTED, STRATA_ERR_OOM, STRATA_ERR_CUDA, \
    STRATA_ERR_TIMEOUT, STRATA_ERR_BOUNDS = range(7)
STRATA_OPT_PATH, STRATA_OPT_WAIT_BUDGET, STRATA_OPT_DECODE_MAX_T = 1, 2, 3
STRATA_SCORE_SOFTMAX, STRATA_SCORE_SIGMOID = 0, 1
STRATA_GROUP_BEST, STRATA_GROUP_SUM2 = 0, 1
STRATA_BF16, STRATA_F32 = 0, 1
STRATA_Q8_E4M3, STRATA_Q8_INT8 = 0, 1

# every symbol the header declares
SYMBOLS = ("strata_moe_create", "strata_moe_destroy", "strata_moe_route", "strata_moe_forward",
           "strata_moe_forward_host", "strata_moe_rmsnorm", "strata_moe_stack_forward",
           "strata_moe_sync_status", "strata_moe_last_error", "strata_moe_debug_dequant",
           "strata_moe_set_option", "strata_moe_selftest_wait", "strata_moe_version",
           "strata_moe_set_probe", "strata_moe_launch_count", "strata_moe_route_noalloc",
           "strata_moe_debug_fail_alloc", "strata_moe_debug_live_allocs",
           "strata_ep_expert_range", "strata_ep_plan", "strata_ep_gather_rows",
           "strata_moe_expert_rows", "strata_moe_combine_rows", "strata_moe_debug_screen",
           "strata_moe_route_logits", "strata_moe_set_routing", "strata_moe_add_rmsnorm",
           "strata_moe_dequant_rows")


class strata_moe_config(C.Structure):
    _fields_ = [("hidden", C.c_int32), ("n_experts", C.c_int32), ("top_k", C.c_int32),
                ("inter", C.c_int32), ("quant_bits", C.c_int32), ("block", C.c_int32),
                ("max_tokens", C.c_int32), ("has_router_bias", C.c_int32)]


class strata_moe_weights(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("router_w", C.c_void_p),
                ("router_b", C.c_void_p), ("shared_codes", C.c_void_p),
                ("shared_scales", C.c_void_p)]


class strata_moe_routing(C.Structure):
    _fields_ = [("score", C.c_int32), ("n_groups", C.c_int32), ("top_groups", C.c_int32),
                ("group_score", C.c_int32), ("renorm", C.c_int32), ("scale", C.c_float)]


class StrataError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"strata status {status}: {message}")
        self.status = status


_P, _I, _I64 = C.c_void_p, C.c_int, C.c_int64
_sig = {
    "strata_moe_create": [C.POINTER(strata_moe_config), C.POINTER(strata_moe_weights), _I,
                          C.POINTER(C.c_void_p)],
    "strata_moe_route": [_P, _P, _I, _P, _P, _P, _P, _P],
    "strata_moe_forward": [_P, _P, _I, _P, _P],
    "strata_moe_forward_host": [_P, _P, _I, _P, _P],
    "strata_moe_rmsnorm": [_P, _P, _I, _I, _P],
    "strata_moe_stack_forward": [C.POINTER(C.c_void_p), _I, _P, _I, _P, _P],
    "strata_moe_sync_status": [_P, _P],
    "strata_moe_debug_dequant": [_P, _I, _I, _I, _I, _I, _P],
    "strata_moe_set_option": [_P, _I, _I64],
    "strata_moe_selftest_wait": [_I, _I64],
    "strata_moe_set_probe": [_P, _I, _P, _P],
    "strata_moe_launch_count": [_P, _I],
    "strata_moe_route_noalloc": [_P, _I, _I, _P, _P, _I, _I, _P, _P, _P, _P, _P],
    "strata_moe_debug_fail_alloc": [_I64],
    "strata_moe_debug_screen": [_P, _P, _I, _P, _P],
    "strata_ep_expert_range": [_I, _I, _I, _P, _P],
    "strata_ep_plan": [_P, _I, _I, _I, _I, _P, _P, _P],
    "strata_ep_gather_rows": [_P, _P, _I, _I, _I, _P, _P],
    "strata_moe_expert_rows": [_P, _P, _P, _I, _I, _I, _P, _P, _P],
    "strata_moe_combine_rows": [_P, _P, _I, _P, _P, _P, _P, _I, _P, _P],
    "strata_moe_route_logits": [C.POINTER(strata_moe_routing), _P, _I, _I64, _P, _I, _I, _I, _P,
                                _P, _P],
    "strata_moe_set_routing": [_P, C.POINTER(strata_moe_routing), _P],
    "strata_moe_add_rmsnorm": [_P, _P, _P, _I, C.c_float, _I, _I, _P, _P, _I, _I, _P, _I64, _P,
                               _I64, _P],
    "strata_moe_dequant_rows": [_P, _I, _I64, _P, _I64, _I, _P, _I, _I, _I, _P, _P],
}
for _name, _args in _sig.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = C.c_int
_lib.strata_moe_destroy.argtypes = [_P]
_lib.strata_moe_destroy.restype = None
_lib.strata_moe_last_error.restype = C.c_char_p
_lib.strata_moe_version.restype = C.c_char_p
_lib.strata_moe_debug_live_allocs.argtypes = []
_lib.strata_moe_debug_live_allocs.restype = C.c_int64


def _check(status: int):
    if status != STRATA_OK:
        raise StrataError(status, strata_moe_last_error())


def strata_moe_last_error() -> str:
    return _lib.strata_moe_last_error().decode()


def strata_moe_version() -> str:
    return _lib.strata_moe_version().decode()


def strata_moe_create(cfg: strata_moe_config, weights: strata_moe_weights, device: int = 0):
    h = C.c_void_p()
    _check(_lib.strata_moe_create(C.byref(cfg), C.byref(weights), device, C.byref(h)))
    return h


def strata_moe_destroy(h) -> None:
    _lib.strata_moe_destroy(h)


def strata_moe_route(h, x, T, idx, w, offsets=None, lst=None, stream=None) -> None:
    _check(_lib.strata_moe_route(h, x, T, idx, w, offsets, lst, stream))


def strata_moe_forward(h, x, T, y, stream=None) -> None:
    _check(_lib.strata_moe_forward(h, x, T, y, stream))


def strata_moe_forward_host(h, x_host, T, y_host, stream=None) -> None:
    _check(_lib.strata_moe_forward_host(h, x_host, T, y_host, stream))


def strata_moe_rmsnorm(h_dev, xn_dev, T, H, stream=None) -> None:
    _check(_lib.strata_moe_rmsnorm(h_dev, xn_dev, T, H, stream))


def strata_moe_stack_forward(layers, h_dev, T, h_trace=None, stream=None) -> None:
    arr = (C.c_void_p * len(layers))(*[l.value if isinstance(l, C.c_void_p) else l
                                       for l in layers])
    _check(_lib.strata_moe_stack_forward(arr, len(layers), h_dev, T, h_trace, stream))


def strata_moe_sync_status(h, stream=None) -> None:
    _check(_lib.strata_moe_sync_status(h, stream))


def strata_moe_debug_dequant(h, expert, mat, row0, nrows, kind, out_host) -> None:
    _check(_lib.strata_moe_debug_dequant(h, expert, mat, row0, nrows, kind, out_host))


def strata_moe_set_option(h, option, value) -> None:
    _check(_lib.strata_moe_set_option(h, option, int(value)))


def strata_ep_expert_range(rank, n_ranks, n_experts) -> tuple[int, int]:
    b, e = C.c_int32(), C.c_int32()
    _check(_lib.strata_ep_expert_range(rank, n_ranks, n_experts, C.byref(b), C.byref(e)))
    return b.value, e.value


def strata_ep_plan(idx, n_experts, n_ranks):
    """idx: int32 numpy [T][k] (host).  Returns (send_counts [n_ranks],
    send_pick [T*k], slot [T*k]) as int32 numpy arrays."""
    import numpy as np
    idx = np.ascontiguousarray(idx, dtype=np.int32)
    T, k = idx.shape
    counts = np.zeros(n_ranks, dtype=np.int32)
    pick = np.zeros(T * k, dtype=np.int32)
    slot = np.zeros(T * k, dtype=np.int32)
    _check(_lib.strata_ep_plan(idx.ctypes.data, T, k, n_experts, n_ranks, counts.ctypes.data,
                               pick.ctypes.data, slot.ctypes.data))
    return counts, pick, slot


def strata_ep_gather_rows(src, rows, n, n_src, row_bytes, dst, stream=None) -> None:
    _check(_lib.strata_ep_gather_rows(src, rows, n, n_src, row_bytes, dst, stream))


def strata_moe_expert_rows(h, x, ids, n, n_shared, prefill, y, yshared, stream=None) -> None:
    _check(_lib.strata_moe_expert_rows(h, x, ids, n, n_shared, int(prefill), y, yshared, stream))


def strata_moe_combine_rows(h, x, T, idx, w, slot, y, prefill, out, stream=None) -> None:
    _check(_lib.strata_moe_combine_rows(h, x, T, idx, w, slot, y, int(prefill), out, stream))


def strata_moe_debug_screen(h, x, T, a_host, eps_host) -> None:
    _check(_lib.strata_moe_debug_screen(h, x, T, a_host, eps_host))


def strata_moe_debug_fail_alloc(n) -> None:
    _check(_lib.strata_moe_debug_fail_alloc(int(n)))


def strata_moe_debug_live_allocs() -> int:
    return int(_lib.strata_moe_debug_live_allocs())


def strata_moe_selftest_wait(device, budget_cycles) -> None:
    _check(_lib.strata_moe_selftest_wait(device, int(budget_cycles)))


def strata_moe_set_probe(h, stage, ev_begin, ev_end) -> None:
    _check(_lib.strata_moe_set_probe(h, stage, ev_begin, ev_end))


def strata_moe_launch_count(h, T) -> int:
    return _lib.strata_moe_launch_count(h, T)


def strata_moe_route_noalloc(x, T, H, router_w, router_b, E, k, idx, w, offsets=None, lst=None,
                             stream=None) -> None:
    _check(_lib.strata_moe_route_noalloc(x, T, H, router_w, router_b, E, k, idx, w, offsets, lst,
                                         stream))


def strata_moe_route_logits(rule, logits, logits_type, ld, select_bias, T, E, k, idx, w,
                            stream=None) -> None:
    _check(_lib.strata_moe_route_logits(rule, logits, logits_type, ld, select_bias, T, E, k, idx,
                                        w, stream))


def strata_moe_set_routing(h, rule, select_bias=None) -> None:
    """rule: strata_moe_routing or None; select_bias: float numpy [E] (host) or None."""
    import numpy as np
    keep = None if select_bias is None else np.ascontiguousarray(select_bias, dtype=np.float32)
    _check(_lib.strata_moe_set_routing(h, rule, None if keep is None else keep.ctypes.data))


def strata_moe_add_rmsnorm(x, delta, weight, weight_type, eps, T, H, h_out, xn, q8=0, group=0,
                           q=None, q_stride=0, scale=None, scale_stride=0, stream=None) -> None:
    _check(_lib.strata_moe_add_rmsnorm(x, delta, weight, weight_type, eps, T, H, h_out, xn, q8,
                                       group, q, q_stride, scale, scale_stride, stream))


def strata_moe_dequant_rows(q, q8, q_stride, scale, scale_stride, group, rows, n, n_src, H, out,
                            stream=None) -> None:
    _check(_lib.strata_moe_dequant_rows(q, q8, q_stride, scale, scale_stride, group, rows, n,
                                        n_src, H, out, stream))


# ----------------------------------------------------------------- convenience
def make_routing(score="softmax", n_groups=1, top_groups=None, group_score="best", renorm=True,
                 scale=1.0) -> strata_moe_routing:
    """A routing rule: score "softmax" or "sigmoid"; n_groups runs of experts of
    which top_groups (default: all) stay, by their "best" value or the sum of
    their best two ("sum2"); renorm divides the weights by their sum over the
    picks; scale multiplies them."""
    scores = {"softmax": STRATA_SCORE_SOFTMAX, "sigmoid": STRATA_SCORE_SIGMOID}
    groups = {"best": STRATA_GROUP_BEST, "sum2": STRATA_GROUP_SUM2}
    if score not in scores or group_score not in groups:
        raise ValueError(f"unknown score {score!r} or group_score {group_score!r}")
    return strata_moe_routing(scores[score], n_groups, n_groups if top_groups is None else top_groups,
                              groups[group_score], 1 if renorm else 0, scale)


_Q8 = {"e4m3": STRATA_Q8_E4M3, "int8": STRATA_Q8_INT8}


def _rows(t, name, dtypes, cols=None):
    """A contiguous [rows, cols] CUDA tensor of one of the dtypes, else ValueError."""
    if not t.is_cuda or t.dim() != 2 or not t.is_contiguous() or t.dtype not in dtypes:
        raise ValueError(f"{name} must be a contiguous 2-d CUDA tensor of {' or '.join(map(str, dtypes))}")
    if cols is not None and t.shape[1] != cols:
        raise ValueError(f"{name} must have {cols} columns")
    return t.data_ptr()


def _stream_ptr(stream, device):
    """A torch stream's pointer; without one, the device's current stream's."""
    import torch
    return (torch.cuda.current_stream(device) if stream is None else stream).cuda_stream


def _output(stream, make, *args, **kw):
    """A tensor that a call on `stream` writes: memory of that stream, not used again
    before the current stream is done with it either."""
    import torch
    if stream is None:
        return make(*args, **kw)
    with torch.cuda.stream(stream):
        t = make(*args, **kw)
    current = torch.cuda.current_stream(t.device)
    if current != stream:
        t.record_stream(current)
    return t


def _same_device(first, *others):
    for t in others:
        if t is not None and t.device != first.device:
            raise ValueError("all tensors must be on one device")


def route_logits(logits, rule, k, select_bias=None, stream=None):
    """Picks int32 [T, k] and weights float32 [T, k] of logits [T, E] (float32 or
    bfloat16 CUDA tensor; rows may be strided) by a routing rule (make_routing)."""
    import torch
    if not logits.is_cuda or logits.dim() != 2 or logits.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("logits must be a 2-d float32 or bfloat16 CUDA tensor")
    T, E = logits.shape
    if T and E > 1 and logits.stride(1) != 1 or T > 1 and logits.stride(0) < E:
        raise ValueError("logits' rows must be contiguous and may not overlap")
    bias = None
    if select_bias is not None:
        _same_device(logits, select_bias)
        if select_bias.dtype != torch.float32 or select_bias.shape != (E,) or not select_bias.is_contiguous():
            raise ValueError(f"select_bias must be a contiguous float32 tensor of {E} values")
        bias = select_bias.data_ptr()
    idx = _output(stream, torch.empty, (T, k), dtype=torch.int32, device=logits.device)
    w = _output(stream, torch.empty, (T, k), dtype=torch.float32, device=logits.device)
    strata_moe_route_logits(rule, logits.data_ptr(), STRATA_F32 if logits.dtype == torch.float32 else STRATA_BF16,
                            logits.stride(0) if T > 1 else max(E, 1), bias, T, E, k, idx.data_ptr(), w.data_ptr(),
                            _stream_ptr(stream, logits.device))
    return idx, w


def packed_row_bytes(H, group=128) -> int:
    """Bytes of a packed 8-bit row: H codes, then the scales, up to a multiple of 16."""
    return H + (4 * (H // group if group else 1) + 15) // 16 * 16


def add_rmsnorm(x, delta=None, weight=None, eps=1e-6, quant=None, group=128, want_xn=True, stream=None):
    """A block's pre-norm of bfloat16 [T, H] rows: h = x + delta, xn = RMSNorm(h)
    weight.  Returns (h, xn, packed): h is x itself without a delta, xn None
    unless wanted, packed None or, with quant "e4m3" or "int8", the rows in 8
    bits as uint8 [T, packed_row_bytes(H, group)] (codes, then float32 scales; the
    bytes behind them are not written)."""
    import torch
    T, H = x.shape
    xp = _rows(x, "x", (torch.bfloat16,))
    _same_device(x, delta, weight)
    dp = None if delta is None else _rows(delta, "delta", (torch.bfloat16,), H)
    if delta is not None and delta.shape[0] != T:
        raise ValueError(f"delta must have {T} rows")
    if weight is not None and (weight.dtype not in (torch.float32, torch.bfloat16) or weight.shape != (H,)
                               or not weight.is_contiguous()):
        raise ValueError(f"weight must be a contiguous float32 or bfloat16 tensor of {H} values")
    if quant is not None and quant not in _Q8:
        raise ValueError(f"unknown 8-bit type {quant!r}")
    h = x if delta is None else _output(stream, torch.empty_like, x)
    xn = _output(stream, torch.empty_like, x) if want_xn else None
    packed = scale = None
    rb = 0
    if quant is not None:
        rb = packed_row_bytes(H, group)
        packed = _output(stream, torch.empty, (T, rb), dtype=torch.uint8, device=x.device)
        scale = packed.data_ptr() + H
    if T:
        strata_moe_add_rmsnorm(xp, dp, None if weight is None else weight.data_ptr(),
                               STRATA_BF16 if weight is not None and weight.dtype == torch.bfloat16 else STRATA_F32,
                               eps, T, H, None if delta is None else h.data_ptr(), None if xn is None else xn.data_ptr(),
                               _Q8[quant] if quant else 0, group, None if packed is None else packed.data_ptr(), rb,
                               scale, rb // 4, _stream_ptr(stream, x.device))
    return h, xn, packed


def dequant_rows(packed, H, quant="e4m3", group=128, rows=None, out=None, stream=None):
    """Packed 8-bit rows (add_rmsnorm) back in bfloat16 [n, H]: row rows[i] (int32
    CUDA tensor; outside the rows: out's row i stays as it is), or every row."""
    import torch
    if quant not in _Q8:
        raise ValueError(f"unknown 8-bit type {quant!r}")
    p = _rows(packed, "packed", (torch.uint8,), packed_row_bytes(H, group))
    n = packed.shape[0]
    if rows is not None:
        if rows.dtype != torch.int32 or rows.dim() != 1 or not rows.is_contiguous():
            raise ValueError("rows must be a contiguous 1-d int32 tensor")
        n = rows.shape[0]
    _same_device(packed, rows, out)
    if out is None:
        out = _output(stream, torch.empty, (n, H), dtype=torch.bfloat16, device=packed.device)
    op = _rows(out, "out", (torch.bfloat16,), H)
    if out.shape[0] != n:
        raise ValueError(f"out must have {n} rows")
    rb = packed.shape[1]
    strata_moe_dequant_rows(p, _Q8[quant], rb, p + H, rb // 4, group, None if rows is None else rows.data_ptr(), n,
                            packed.shape[0], H, op, _stream_ptr(stream, packed.device))
    return out


def make_config(shape, max_tokens: int) -> strata_moe_config:
    """Config from any object with hidden/n_experts/top_k/inter/bits/router_bias."""
    return strata_moe_config(shape.hidden, shape.n_experts, shape.top_k, shape.inter, shape.bits,
                             32, max_tokens, 1 if shape.router_bias else 0)


def make_weights(layer) -> tuple[strata_moe_weights, list]:
    """Weights struct from numpy arrays (any object with codes, scales, router_w,
    router_b, shared_codes, shared_scales).  Returns the struct and the arrays
    it points into (keep them alive until create returns)."""
    import numpy as np
    keep = [np.ascontiguousarray(layer.codes, dtype=np.uint8),
            np.ascontiguousarray(layer.scales, dtype=np.uint16),
            np.ascontiguousarray(layer.router_w, dtype=np.float32),
            None if layer.router_b is None else np.ascontiguousarray(layer.router_b,
                                                                    dtype=np.float32),
            np.ascontiguousarray(layer.shared_codes, dtype=np.uint8),
            np.ascontiguousarray(layer.shared_scales, dtype=np.uint16)]
    ptr = [None if a is None else a.ctypes.data for a in keep]
    return strata_moe_weights(*ptr), keep


class Layer:
    """One MoE layer on a CUDA device; torch tensors in and out."""

    def __init__(self, layer, max_tokens: int, device: int = 0):
        self.shape = layer.shape
        self.device = device
        cfg = make_config(layer.shape, max_tokens)
        w, keep = make_weights(layer)
        self.handle = strata_moe_create(cfg, w, device)
        del keep

    def close(self):
        if self.handle is not None:
            strata_moe_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_option(self, option, value):
        strata_moe_set_option(self.handle, option, value)

    def set_routing(self, rule=None, select_bias=None):
        """Pick and weigh by `rule` (make_routing) from now on; None: the default.
        select_bias: n_experts floats on the host, or None."""
        import numpy as np
        if select_bias is not None:
            select_bias = np.ascontiguousarray(select_bias, dtype=np.float32)
            if select_bias.shape != (self.shape.n_experts,):
                raise ValueError(f"select_bias must have {self.shape.n_experts} values")
        strata_moe_set_routing(self.handle, rule, select_bias)

    def forward(self, x, out=None, stream=None):
        import torch
        T = x.shape[0]
        if out is None:
            out = _output(stream, torch.empty_like, x)
        strata_moe_forward(self.handle, x.data_ptr(), T, out.data_ptr(), _stream_ptr(stream, x.device))
        return out

    def route(self, x, stream=None):
        import torch
        T, k, E = x.shape[0], self.shape.top_k, self.shape.n_experts
        dev = x.device
        idx = _output(stream, torch.empty, (T, k), dtype=torch.int32, device=dev)
        w = _output(stream, torch.empty, (T, k), dtype=torch.float32, device=dev)
        off = _output(stream, torch.empty, E + 1, dtype=torch.int32, device=dev)
        lst = _output(stream, torch.empty, T * k, dtype=torch.int32, device=dev)
        strata_moe_route(self.handle, x.data_ptr(), T, idx.data_ptr(), w.data_ptr(),
                         off.data_ptr(), lst.data_ptr(), _stream_ptr(stream, dev))
        return idx, w, off, lst

    def sync_status(self, stream=None):
        strata_moe_sync_status(self.handle, _stream_ptr(stream, self.device))

    def debug_dequant(self, expert, mat, row0, nrows, kind=0):
        import numpy as np
        cols = self.shape.hidden if mat < 2 else self.shape.inter
        out = np.empty((nrows, cols), dtype=np.float32)
        strata_moe_debug_dequant(self.handle, expert, mat, row0, nrows, kind,
                                 out.ctypes.data)
        return out
