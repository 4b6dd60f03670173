"""Mixture-of-experts operators, and the int8 and 4-bit linear layers.

A thin ctypes binding over ``libfp8w_moe.so`` (declared in
``include/fp8w_moe.h``), in the manner of the package's FP8 linear layer: the
raw entry points keep the C names and take integers; the tensor helpers check
their arguments, allocate outputs and workspaces with torch and run on torch's
current stream of the tensors' device. The helpers of the timed path go through
a small compiled module (``csrc/moe/helpers.cpp``), which does the same for calls
that are right (and returns the status of a launch that failed); the Python below
it says what is wrong with the others and takes a caller's workspace. There is no
CPU or PyTorch fallback.

    r = route(logits, top_k)                       # who goes where
    h = linear_experts(x, q, scale, r.offsets, x_rows=r.tokens)     # up: gathers tokens, rows by expert
    y = linear_experts(act(h), q2, scale2, r.offsets, y_rows=r.slots)  # down: rows by slot
    out = combine(y, r.weights)                    # each token's weighted sum

    q, scale = quantize_int8(w)                    # build time
    y = linear_int8(x, q, scale, bias)             # x quantized per token in the call

    q, scale = quantize_fp4(w)                     # build time; w [n, k], or [e, n, k] for experts
    y = linear_fp4(x, q, scale, bias)
    h = linear_experts_fp4(x, qe, se, r.offsets, x_rows=r.tokens)

    out = moe_layer(x, logits, top_k, (q, scale), (q2, scale2))    # all of a layer for up to 64 tokens
"""
import contextlib
import ctypes
import math
import os
from typing import NamedTuple

import torch

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_I = ctypes.c_int

# name -> (restype, argtypes), mirroring include/fp8w_moe.h
MOE_EXPORTS = {
    "fp8w_route": (_I, [_P, _I, _I64, _I64, _I64, _I, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "fp8w_route_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "fp8w_linear_experts": (_I, [_P, _I, _I64, _I64, _P, _P, _P, _I64, _I64, _P, _I64, _P, _P, _P, _P, _SZ, _P]),
    "fp8w_linear_experts_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I64, _P, _P]),
    "fp8w_linear_experts_kernel": (ctypes.c_char_p, [_I64, _I64, _I64, _I64, _P, _P]),
    "fp8w_combine": (_I, [_P, _I, _P, _I64, _I64, _I64, _P, _P]),
    "fp8w_quantize_int8": (_I, [_P, _I, _I64, _I64, _P, _P, _P]),
    "fp8w_quantize_activations_int8": (_I, [_P, _I, _I64, _I64, _P, _P, _P]),
    "fp8w_gemm_int8": (_I, [_P, _P, _I64, _I64, _P, _P, _P, _I64, _P, _I, _P]),
    "fp8w_linear_int8": (_I, [_P, _I, _I64, _I64, _P, _P, _P, _I64, _P, _P, _SZ, _P]),
    "fp8w_linear_int8_workspace_bytes": (_SZ, [_I64, _I64, _I64, _P, _P]),
    "fp8w_linear_int8_kernel": (ctypes.c_char_p, [_I64, _I64, _I64, _P, _P]),
    "fp8w_quantize_fp4": (_I, [_P, _I, _I64, _I64, _P, _P, _P]),
    "fp8w_dequantize_fp4": (_I, [_P, _P, _I64, _I64, _P, _I, _P]),
    "fp8w_linear_fp4": (_I, [_P, _I, _I64, _I64, _P, _P, _P, _I64, _P, _P, _SZ, _P]),
    "fp8w_linear_fp4_workspace_bytes": (_SZ, [_I64, _I64, _I64, _P, _P, _P]),
    "fp8w_linear_fp4_kernel": (ctypes.c_char_p, [_I64, _I64, _I64, _P, _P, _P]),
    "fp8w_linear_experts_fp4": (_I, [_P, _I, _I64, _I64, _P, _P, _P, _I64, _I64, _P, _I64, _P, _P, _P, _P]),
    "fp8w_linear_experts_fp4_kernel": (ctypes.c_char_p, [_I64, _I64, _I64, _I64, _P, _P, _P]),
    "fp8w_moe_layer": (_I, [_P, _I, _I64, _I64, _P, _I, _I64, _I64, _I, _I, _P, _P, _P, _I64, _P, _P, _P, _P, _P, _SZ,
                            _P]),
    "fp8w_moe_layer_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I64, _I64]),
    "fp8w_moe_last_hip_error": (_I, []),
}

__all__ = [*MOE_EXPORTS, "MOE_EXPORTS", "Fp8wMoeError", "moe_lib_path", "load_moe", "Route", "route",
           "quantize_experts", "linear_experts", "experts_workspace_bytes", "combine", "quantize_int8",
           "quantize_activations_int8", "gemm_int8", "linear_int8", "int8_workspace_bytes", "quantize_fp4",
           "dequantize_fp4", "linear_fp4", "fp4_workspace_bytes", "linear_experts_fp4", "moe_layer",
           "moe_layer_workspace_bytes", "MOE_LAYER_TOKENS", "WEIGHT_E4M3", "WEIGHT_FP4"]

_LIB = None
_FAST = None


def moe_lib_path() -> str:
    return os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfp8w_moe.so")


def load_moe():
    """Load libfp8w_moe.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        p = moe_lib_path()
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()'); "
                               "there is no non-HIP implementation")
        lib = ctypes.CDLL(p)
        for name, (res, args) in MOE_EXPORTS.items():
            f = getattr(lib, name)
            f.restype = res
            f.argtypes = args
        _LIB = lib
    return _LIB


def _fast():
    """The compiled helpers (raises if they have not been built)."""
    global _FAST
    if _FAST is None:
        load_moe()
        try:
            from . import _moe_helpers
        except ImportError as e:
            raise RuntimeError("_moe_helpers.so is missing or does not load: build it first "
                               "(python -c 'import __graft_entry__ as g; g.build()')") from e
        _FAST = _moe_helpers
    return _FAST


# ------------------------------------------------------------------ raw C entry points
def fp8w_route(logits, dtype, t, e, top_k, renormalize, weights, experts, offsets, slots, tokens, workspace,
               workspace_bytes, stream) -> int:
    return load_moe().fp8w_route(logits, dtype, t, e, top_k, renormalize, weights, experts, offsets, slots, tokens,
                                 workspace, workspace_bytes, stream)


def fp8w_route_workspace_bytes(t, e, top_k) -> int:
    return load_moe().fp8w_route_workspace_bytes(t, e, top_k)


def fp8w_linear_experts(x, act_dtype, x_count, k, q, scale, bias, e, n, offsets, m, x_rows, y_rows, y, workspace,
                        workspace_bytes, stream) -> int:
    return load_moe().fp8w_linear_experts(x, act_dtype, x_count, k, q, scale, bias, e, n, offsets, m, x_rows, y_rows,
                                          y, workspace, workspace_bytes, stream)


def fp8w_linear_experts_workspace_bytes(m, e, n, k, x, q) -> int:
    return load_moe().fp8w_linear_experts_workspace_bytes(m, e, n, k, x, q)


def fp8w_linear_experts_kernel(m, e, n, k, x, q):
    r = load_moe().fp8w_linear_experts_kernel(m, e, n, k, x, q)
    return r.decode() if r is not None else None


def fp8w_combine(y, act_dtype, weights, t, top_k, n, out, stream) -> int:
    return load_moe().fp8w_combine(y, act_dtype, weights, t, top_k, n, out, stream)


def fp8w_quantize_int8(w, w_dtype, n, k, q, scale, stream) -> int:
    return load_moe().fp8w_quantize_int8(w, w_dtype, n, k, q, scale, stream)


def fp8w_quantize_activations_int8(x, act_dtype, m, k, qx, sx, stream) -> int:
    return load_moe().fp8w_quantize_activations_int8(x, act_dtype, m, k, qx, sx, stream)


def fp8w_gemm_int8(qx, sx, m, k, q, scale, bias, n, y, out_dtype, stream) -> int:
    return load_moe().fp8w_gemm_int8(qx, sx, m, k, q, scale, bias, n, y, out_dtype, stream)


def fp8w_linear_int8(x, act_dtype, m, k, q, scale, bias, n, y, workspace, workspace_bytes, stream) -> int:
    return load_moe().fp8w_linear_int8(x, act_dtype, m, k, q, scale, bias, n, y, workspace, workspace_bytes, stream)


def fp8w_linear_int8_workspace_bytes(m, n, k, x, q) -> int:
    return load_moe().fp8w_linear_int8_workspace_bytes(m, n, k, x, q)


def fp8w_linear_int8_kernel(m, n, k, x, q):
    r = load_moe().fp8w_linear_int8_kernel(m, n, k, x, q)
    return r.decode() if r is not None else None


def fp8w_quantize_fp4(w, w_dtype, n, k, q, scale, stream) -> int:
    return load_moe().fp8w_quantize_fp4(w, w_dtype, n, k, q, scale, stream)


def fp8w_dequantize_fp4(q, scale, n, k, out, out_dtype, stream) -> int:
    return load_moe().fp8w_dequantize_fp4(q, scale, n, k, out, out_dtype, stream)


def fp8w_linear_fp4(x, act_dtype, m, k, q, scale, bias, n, y, workspace, workspace_bytes, stream) -> int:
    return load_moe().fp8w_linear_fp4(x, act_dtype, m, k, q, scale, bias, n, y, workspace, workspace_bytes, stream)


def fp8w_linear_fp4_workspace_bytes(m, n, k, x, q, scale) -> int:
    return load_moe().fp8w_linear_fp4_workspace_bytes(m, n, k, x, q, scale)


def fp8w_linear_fp4_kernel(m, n, k, x, q, scale):
    r = load_moe().fp8w_linear_fp4_kernel(m, n, k, x, q, scale)
    return r.decode() if r is not None else None


def fp8w_linear_experts_fp4(x, act_dtype, x_count, k, q, scale, bias, e, n, offsets, m, x_rows, y_rows, y,
                            stream) -> int:
    return load_moe().fp8w_linear_experts_fp4(x, act_dtype, x_count, k, q, scale, bias, e, n, offsets, m, x_rows,
                                              y_rows, y, stream)


def fp8w_linear_experts_fp4_kernel(m, e, n, k, x, q, scale):
    r = load_moe().fp8w_linear_experts_fp4_kernel(m, e, n, k, x, q, scale)
    return r.decode() if r is not None else None


def fp8w_moe_layer(x, act_dtype, t, hidden, logits, logits_dtype, e, top_k, renormalize, format, q_gate_up, scale_gate_up,
                   bias_gate_up, inner, q_down, scale_down, bias_down, out, workspace, workspace_bytes, stream) -> int:
    return load_moe().fp8w_moe_layer(x, act_dtype, t, hidden, logits, logits_dtype, e, top_k, renormalize, format,
                                     q_gate_up, scale_gate_up, bias_gate_up, inner, q_down, scale_down, bias_down, out,
                                     workspace, workspace_bytes, stream)


def fp8w_moe_layer_workspace_bytes(t, e, top_k, hidden, inner) -> int:
    return load_moe().fp8w_moe_layer_workspace_bytes(t, e, top_k, hidden, inner)


def fp8w_moe_last_hip_error() -> int:
    return load_moe().fp8w_moe_last_hip_error()


# ------------------------------------------------------------------ tensor helpers
# The handle of a device's current stream, without the stream object that torch.cuda.current_stream makes.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_DT = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_STATUS = ("success", "invalid value (size, dtype, NULL pointer or overlapping buffers)", "misaligned pointer",
           "non-finite weight (NaN or infinity)", "workspace missing or too small", "HIP runtime error")
_ERR_HIP = 5
MOE_LAYER_TOKENS = 64            # the most tokens that moe_layer takes
WEIGHT_E4M3, WEIGHT_FP4 = 0, 1   # fp8w_weight_format_t


class Fp8wMoeError(RuntimeError):
    """A call of libfp8w_moe.so failed; ``status`` is its fp8w_status_t."""

    def __init__(self, status: int, where: str):
        self.status = status
        msg = _STATUS[status] if 0 <= status < len(_STATUS) else "unknown status"
        if status == _ERR_HIP:
            msg += f" (hipError {fp8w_moe_last_hip_error()})"
        super().__init__(f"{where}: {msg}")


def _check(st: int, where: str) -> None:
    if st != 0:
        raise Fp8wMoeError(st, where)


def _act_code(t: torch.dtype, name: str) -> int:
    if t not in (torch.bfloat16, torch.float16):
        raise TypeError(f"{name} must be bf16 or fp16, not {t}")
    return _DT[t]


def _want(t, name: str, shape, dtype, device) -> int:
    """The device address of a tensor that must look like this (0 for None and empty ones)."""
    if t is None:
        return 0
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        if t.shape != shape or t.dtype is not dtype:
            raise ValueError(f"{name} must be {list(shape)} of {dtype}, not {list(t.shape)} of {t.dtype}")
        if t.device != device:
            raise ValueError(f"{name} must be on the GPU of the first argument")
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr() if t.numel() else 0


def _gpu(t: torch.Tensor, name: str, dims: int) -> torch.device:
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    return t.device


def _workspace(ws, need: int, device):
    """(address, bytes) of the caller's workspace, or of a new one of ``need`` bytes; the tensor keeps it alive."""
    if ws is None:
        ws = torch.empty((need,), dtype=torch.uint8, device=device) if need else None
    elif not ws.is_cuda or ws.device != device or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the GPU of the first argument")
    if ws is None or ws.numel() == 0:
        return ws, 0, 0
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def _stream(device: torch.device) -> int:
    return _raw_stream(device.index)


_SAME_DEVICE = contextlib.nullcontext()


def _on(device: torch.device):
    """The tensors' device made the current one for a call of the library: it launches on the current device, and
    torch's default stream has the same handle (0) on each."""
    if device.type != "cuda" or device.index == _current_device():  # others are refused by the argument checks
        return _SAME_DEVICE
    return torch.cuda.device(device)


class Route(NamedTuple):
    weights: torch.Tensor  # [t, top_k] fp32
    experts: torch.Tensor  # [t, top_k] int32, -1: none
    offsets: torch.Tensor  # [e + 1] int32: expert i has positions offsets[i] .. offsets[i + 1] - 1
    slots: torch.Tensor    # [t * top_k] int32: token * top_k + j, ordered by expert
    tokens: torch.Tensor   # [t * top_k] int32: slots // top_k


def route(logits: torch.Tensor, top_k: int, renormalize: bool = True, out: Route = None,
          workspace: torch.Tensor = None) -> Route:
    """The top_k experts of each token and the row lists of the experts' products.

    logits: [t, e] bf16 / fp16 / fp32, e up to 1024. The weights are the
    softmax's values at the chosen experts, divided by their sum when
    ``renormalize``. Equal logits go to the lower index; an expert with logit
    -inf is never taken (its place holds -1 and weight 0), so a row of -inf is a
    padding token. ``out`` takes the results of an earlier call's shape."""
    if out is None and workspace is None:
        r = (_FAST or _fast()).route(logits, top_k, renormalize)
        if r is not None:
            return Route._make(r) if type(r) is not int else _check(r, "fp8w_route")
    dev = _gpu(logits, "logits", 2)
    t, e = logits.shape
    if logits.dtype not in _DT:
        raise TypeError(f"logits must be bf16, fp16 or fp32, not {logits.dtype}")
    if not 1 <= top_k <= min(e, 64) or e > 1024:
        raise ValueError("expected 1 <= top_k <= min(e, 64) and e <= 1024")
    lp = _want(logits, "logits", (t, e), logits.dtype, dev)
    if out is None:
        out = Route(logits.new_empty((t, top_k), dtype=torch.float32),
                    logits.new_empty((t, top_k), dtype=torch.int32), logits.new_empty((e + 1,), dtype=torch.int32),
                    logits.new_empty((t * top_k,), dtype=torch.int32),
                    logits.new_empty((t * top_k,), dtype=torch.int32))
    ptr = [_want(out.weights, "weights", (t, top_k), torch.float32, dev),
           _want(out.experts, "experts", (t, top_k), torch.int32, dev),
           _want(out.offsets, "offsets", (e + 1,), torch.int32, dev),
           _want(out.slots, "slots", (t * top_k,), torch.int32, dev),
           _want(out.tokens, "tokens", (t * top_k,), torch.int32, dev)]
    workspace, wp, wb = _workspace(workspace, fp8w_route_workspace_bytes(t, e, top_k), dev)
    with _on(dev):
        st = fp8w_route(lp, _DT[logits.dtype], t, e, top_k, int(renormalize), *ptr, wp, wb, _stream(dev))
    _check(st, "fp8w_route")
    return out


def quantize_experts(w: torch.Tensor):
    """e4m3 codes and scales of a stack of expert weights [e, n, k] (fp32, bf16
    or fp16): (q uint8 [e, n, k], scale fp32 [e, n]), each as ``quantize`` gives."""
    from . import quantize
    if w.dim() != 3:
        raise ValueError("w must be [e, n, k]")
    e, n, k = w.shape
    q, scale = quantize(w.reshape(e * n, k))
    return q.view(e, n, k), scale.view(e, n)


def experts_workspace_bytes(m: int, x: torch.Tensor, q: torch.Tensor) -> int:
    e, n, k = q.shape
    return fp8w_linear_experts_workspace_bytes(m, e, n, k, x.data_ptr(), q.data_ptr())


def linear_experts(x: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, offsets: torch.Tensor,
                   bias: torch.Tensor = None, x_rows: torch.Tensor = None, y_rows: torch.Tensor = None,
                   out: torch.Tensor = None, workspace: torch.Tensor = None) -> torch.Tensor:
    """Each expert's product on its own rows: for offsets[i] <= p < offsets[i+1],
    y[y_rows[p]] = scale[i] * (q[i] @ x[x_rows[p]]) + bias[i], rounded once to x.dtype.

    x: [rows, k] bf16 / fp16; q: [e, n, k] uint8 codes; scale: [e, n] fp32;
    bias: [e, n] of x.dtype; offsets: [e + 1] int32; x_rows / y_rows: [m] int32
    (without them position p reads row p / writes row p). Rows of positions from
    offsets[e] on are zeros. With ``x_rows`` m is its length, else x's. No
    workspace is needed (experts_workspace_bytes is 0); one that is given is not
    used."""
    r = (_FAST or _fast()).linear_experts(x, q, scale, offsets, bias, x_rows, y_rows, out)
    if r is not None:
        return r if type(r) is not int else _check(r, "fp8w_linear_experts")
    dev = _gpu(x, "x", 2)
    if q.dim() != 3:
        raise ValueError("q must have 3 dimensions")
    rows, k = x.shape
    e, n = q.shape[:2]
    m = rows if x_rows is None else x_rows.numel()
    act = _act_code(x.dtype, "x")
    xp = _want(x, "x", (rows, k), x.dtype, dev)
    qp = _want(q, "q", (e, n, k), torch.uint8, dev)
    sp = _want(scale, "scale", (e, n), torch.float32, dev)
    bp = _want(bias, "bias", (e, n), x.dtype, dev)
    op = _want(offsets, "offsets", (e + 1,), torch.int32, dev)
    ip = _want(x_rows, "x_rows", (m,), torch.int32, dev)
    jp = _want(y_rows, "y_rows", (m,), torch.int32, dev)
    if out is None:
        out = x.new_empty((m, n))
    yp = _want(out, "out", (m, n), x.dtype, dev)
    with _on(dev):
        st = fp8w_linear_experts(xp, act, rows, k, qp, sp, bp, e, n, op, m, ip, jp, yp, 0, 0, _stream(dev))
    _check(st, "fp8w_linear_experts")
    return out


def combine(y: torch.Tensor, weights: torch.Tensor, out: torch.Tensor = None) -> torch.Tensor:
    """out[t] = sum_j weights[t, j] * y[t * top_k + j], fp32 sums, rounded once:
    y [t * top_k, n] bf16 / fp16 (rows by slot), weights [t, top_k] fp32."""
    r = (_FAST or _fast()).combine(y, weights, out)
    if r is not None:
        return r if type(r) is not int else _check(r, "fp8w_combine")
    dev = _gpu(y, "y", 2)
    if weights.dim() != 2:
        raise ValueError("weights must have 2 dimensions")
    t, top = weights.shape
    n = y.shape[1]
    act = _act_code(y.dtype, "y")
    yp = _want(y, "y", (t * top, n), y.dtype, dev)
    wp = _want(weights, "weights", (t, top), torch.float32, dev)
    if out is None:
        out = y.new_empty((t, n))
    op = _want(out, "out", (t, n), y.dtype, dev)
    with _on(dev):
        st = fp8w_combine(yp, act, wp, t, top, n, op, _stream(dev))
    _check(st, "fp8w_combine")
    return out


def quantize_int8(w: torch.Tensor):
    """Per-output-channel int8 quantization of a [n, k] weight (fp32, bf16 or
    fp16): (q int8 [n, k], scale fp32 [n] = amax / 127). Synchronizes; raises
    Fp8wMoeError on NaN / inf weights."""
    dev = _gpu(w, "w", 2)
    n, k = w.shape
    if w.dtype not in _DT:
        raise TypeError(f"unsupported dtype {w.dtype}")
    q = torch.empty((n, k), dtype=torch.int8, device=dev)
    scale = torch.empty((n,), dtype=torch.float32, device=dev)
    wp = _want(w, "w", (n, k), w.dtype, dev)
    with _on(dev):
        st = fp8w_quantize_int8(wp, _DT[w.dtype], n, k, q.data_ptr() if q.numel() else 0, scale.data_ptr() if n else 0,
                                _stream(dev))
    _check(st, "fp8w_quantize_int8")
    return q, scale


def quantize_activations_int8(x: torch.Tensor):
    """Per-token int8 codes of activations x [m, k] (bf16 / fp16): (qx int8
    [m, k], sx fp32 [m] = amax / 127). Non-finite rows get NaN scales."""
    dev = _gpu(x, "x", 2)
    m, k = x.shape
    qx = torch.empty((m, k), dtype=torch.int8, device=dev)
    sx = torch.empty((m,), dtype=torch.float32, device=dev)
    xp, act = _want(x, "x", (m, k), x.dtype, dev), _act_code(x.dtype, "x")
    with _on(dev):
        st = fp8w_quantize_activations_int8(xp, act, m, k, qx.data_ptr() if qx.numel() else 0,
                                            sx.data_ptr() if m else 0, _stream(dev))
    _check(st, "fp8w_quantize_activations_int8")
    return qx, sx


def gemm_int8(qx: torch.Tensor, sx: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, bias: torch.Tensor = None,
              out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor = None) -> torch.Tensor:
    """y = (qx @ q.T) * sx[:, None] * scale[None, :] + bias: integer sums, rounded once to out_dtype."""
    dev = _gpu(qx, "qx", 2)
    m, k = qx.shape
    n = q.shape[0]
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=dev)
    act = _act_code(out.dtype, "out")
    xp, tp = _want(qx, "qx", (m, k), torch.int8, dev), _want(sx, "sx", (m,), torch.float32, dev)
    qp, sp = _want(q, "q", (n, k), torch.int8, dev), _want(scale, "scale", (n,), torch.float32, dev)
    bp, yp = _want(bias, "bias", (n,), out.dtype, dev), _want(out, "out", (m, n), out.dtype, dev)
    with _on(dev):
        st = fp8w_gemm_int8(xp, tp, m, k, qp, sp, bp, n, yp, act, _stream(dev))
    _check(st, "fp8w_gemm_int8")
    return out


def int8_workspace_bytes(x: torch.Tensor, q: torch.Tensor) -> int:
    return fp8w_linear_int8_workspace_bytes(x.shape[0], q.shape[0], x.shape[1], x.data_ptr(), q.data_ptr())


def linear_int8(x: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, bias: torch.Tensor = None,
                out: torch.Tensor = None, workspace: torch.Tensor = None) -> torch.Tensor:
    """The int8 layer on bf16 / fp16 activations x [m, k]: per-token quantization
    of x, integer products with q int8 [n, k], y = sums * sx * scale + bias
    rounded once to x.dtype."""
    if workspace is None:
        r = (_FAST or _fast()).linear_int8(x, q, scale, bias, out)
        if r is not None:
            return r if type(r) is not int else _check(r, "fp8w_linear_int8")
    dev = _gpu(x, "x", 2)
    m, k = x.shape
    n = q.shape[0]
    act = _act_code(x.dtype, "x")
    xp = _want(x, "x", (m, k), x.dtype, dev)
    qp = _want(q, "q", (n, k), torch.int8, dev)
    sp = _want(scale, "scale", (n,), torch.float32, dev)
    bp = _want(bias, "bias", (n,), x.dtype, dev)
    if out is None:
        out = x.new_empty((m, n))
    yp = _want(out, "out", (m, n), x.dtype, dev)
    workspace, wp, wb = _workspace(workspace, fp8w_linear_int8_workspace_bytes(m, n, k, xp, qp), dev)
    with _on(dev):
        st = fp8w_linear_int8(xp, act, m, k, qp, sp, bp, n, yp, wp, wb, _stream(dev))
    _check(st, "fp8w_linear_int8")
    return out


def quantize_fp4(w: torch.Tensor):
    """4-bit quantization of a weight [n, k], or of a stack of experts' [e, n, k]
    (fp32, bf16 or fp16): (q uint8 [.., n, (k + 1) // 2], two e2m1 codes to a byte,
    the even k in the low four bits; scale uint8 [.., n, (k + 31) // 32], one
    power of two 2^(s - 127) for 32 weights). Synchronizes; raises Fp8wMoeError on
    NaN / inf weights."""
    if w.dim() not in (2, 3):
        raise ValueError("w must be [n, k] or [e, n, k]")
    dev = _gpu(w, "w", w.dim())
    lead, n, k = w.shape[:-1], math.prod(w.shape[:-1]), w.shape[-1]
    if w.dtype not in _DT:
        raise TypeError(f"unsupported dtype {w.dtype}")
    q = torch.empty((*lead, (k + 1) // 2), dtype=torch.uint8, device=dev)
    scale = torch.empty((*lead, (k + 31) // 32), dtype=torch.uint8, device=dev)
    wp = _want(w, "w", w.shape, w.dtype, dev)
    with _on(dev):
        st = fp8w_quantize_fp4(wp, _DT[w.dtype], n, k, q.data_ptr() if q.numel() else 0,
                               scale.data_ptr() if scale.numel() else 0, _stream(dev))
    _check(st, "fp8w_quantize_fp4")
    return q, scale


def dequantize_fp4(q: torch.Tensor, scale: torch.Tensor, k: int = None,
                   dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """The weights [.., n, k] of ``quantize_fp4``'s codes and scales (k: 2 q.shape[-1]
    unless given) in ``dtype``: exact in fp32 and bf16, rounded once in fp16."""
    if q.dim() not in (2, 3):
        raise ValueError("q must have 2 or 3 dimensions")
    dev = _gpu(q, "q", q.dim())
    k = 2 * q.shape[-1] if k is None else k
    lead, n = q.shape[:-1], math.prod(q.shape[:-1])
    if (k + 1) // 2 != q.shape[-1]:
        raise ValueError("k must be 2 q.shape[-1] or one less")
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype}")
    qp = _want(q, "q", q.shape, torch.uint8, dev)
    sp = _want(scale, "scale", (*lead, (k + 31) // 32), torch.uint8, dev)
    out = torch.empty((*lead, k), dtype=dtype, device=dev)
    with _on(dev):
        st = fp8w_dequantize_fp4(qp, sp, n, k, out.data_ptr() if out.numel() else 0, _DT[dtype], _stream(dev))
    _check(st, "fp8w_dequantize_fp4")
    return out


def fp4_workspace_bytes(x: torch.Tensor, q: torch.Tensor, scale: torch.Tensor) -> int:
    return fp8w_linear_fp4_workspace_bytes(x.shape[0], q.shape[0], x.shape[1], x.data_ptr(), q.data_ptr(),
                                           scale.data_ptr())


def linear_fp4(x: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, bias: torch.Tensor = None,
               out: torch.Tensor = None, workspace: torch.Tensor = None) -> torch.Tensor:
    """y = x @ w.T + bias on 4-bit weights, fp32 sums, rounded once to x.dtype.

    x: [m, k] bf16 / fp16, any m; q: [n, (k + 1) // 2] uint8 and scale: [n, (k + 31)
    // 32] uint8 as ``quantize_fp4`` gives them; bias: [n] of x.dtype. In fp16 a
    weight is its fp16 value (exact for scales 2^-23 .. 2^13)."""
    if workspace is None:
        r = (_FAST or _fast()).linear_fp4(x, q, scale, bias, out)
        if r is not None:
            return r if type(r) is not int else _check(r, "fp8w_linear_fp4")
    dev = _gpu(x, "x", 2)
    if q.dim() != 2:
        raise ValueError("q must have 2 dimensions")
    m, k = x.shape
    n = q.shape[0]
    act = _act_code(x.dtype, "x")
    xp = _want(x, "x", (m, k), x.dtype, dev)
    qp = _want(q, "q", (n, (k + 1) // 2), torch.uint8, dev)
    sp = _want(scale, "scale", (n, (k + 31) // 32), torch.uint8, dev)
    bp = _want(bias, "bias", (n,), x.dtype, dev)
    if out is None:
        out = x.new_empty((m, n))
    yp = _want(out, "out", (m, n), x.dtype, dev)
    workspace, wp, wb = _workspace(workspace, fp8w_linear_fp4_workspace_bytes(m, n, k, xp, qp, sp), dev)
    with _on(dev):
        st = fp8w_linear_fp4(xp, act, m, k, qp, sp, bp, n, yp, wp, wb, _stream(dev))
    _check(st, "fp8w_linear_fp4")
    return out


def linear_experts_fp4(x: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, offsets: torch.Tensor,
                       bias: torch.Tensor = None, x_rows: torch.Tensor = None, y_rows: torch.Tensor = None,
                       out: torch.Tensor = None) -> torch.Tensor:
    """``linear_experts`` on 4-bit weights: q [e, n, (k + 1) // 2] uint8 and scale
    [e, n, (k + 31) // 32] uint8 as ``quantize_fp4`` gives them for [e, n, k]."""
    r = (_FAST or _fast()).linear_experts_fp4(x, q, scale, offsets, bias, x_rows, y_rows, out)
    if r is not None:
        return r if type(r) is not int else _check(r, "fp8w_linear_experts_fp4")
    dev = _gpu(x, "x", 2)
    if q.dim() != 3:
        raise ValueError("q must have 3 dimensions")
    rows, k = x.shape
    e, n = q.shape[:2]
    m = rows if x_rows is None else x_rows.numel()
    act = _act_code(x.dtype, "x")
    xp = _want(x, "x", (rows, k), x.dtype, dev)
    qp = _want(q, "q", (e, n, (k + 1) // 2), torch.uint8, dev)
    sp = _want(scale, "scale", (e, n, (k + 31) // 32), torch.uint8, dev)
    bp = _want(bias, "bias", (e, n), x.dtype, dev)
    op = _want(offsets, "offsets", (e + 1,), torch.int32, dev)
    ip = _want(x_rows, "x_rows", (m,), torch.int32, dev)
    jp = _want(y_rows, "y_rows", (m,), torch.int32, dev)
    if out is None:
        out = x.new_empty((m, n))
    yp = _want(out, "out", (m, n), x.dtype, dev)
    with _on(dev):
        st = fp8w_linear_experts_fp4(xp, act, rows, k, qp, sp, bp, e, n, op, m, ip, jp, yp, _stream(dev))
    _check(st, "fp8w_linear_experts_fp4")
    return out


def moe_layer_workspace_bytes(x: torch.Tensor, logits: torch.Tensor, top_k: int, gate_up) -> int:
    """The workspace of ``moe_layer`` on these, in bytes."""
    t, e = logits.shape
    return fp8w_moe_layer_workspace_bytes(t, e, top_k, x.shape[1], gate_up[0].shape[1] // 2)


def moe_layer(x: torch.Tensor, logits: torch.Tensor, top_k: int, gate_up, down, gate_up_bias: torch.Tensor = None,
              down_bias: torch.Tensor = None, renormalize: bool = True, out: torch.Tensor = None,
              workspace: torch.Tensor = None) -> torch.Tensor:
    """A mixture-of-experts layer for up to 64 tokens, in two launches: ``route`` on the logits [t, e], each expert's
    gate and up products on its tokens, silu(gate) * up, the down products, and the sum over a token's experts.

    x: [t, hidden] bf16 / fp16. gate_up, down: (q, scale) pairs of weights [e, 2 inner, hidden] (gate's rows first)
    and [e, hidden, inner], both from ``quantize_experts`` or both from ``quantize_fp4``. Biases [e, 2 inner] and
    [e, hidden] of x.dtype. Sums in fp32; silu(gate) * up and the result are rounded to x.dtype (in fp16 a silu(gate) * up
    above 65504 makes its token's row infinite or NaN, as it would between separate calls). For more tokens call ``route``, ``linear_experts`` (``linear_experts_fp4``) and ``combine``. ``workspace``: of
    moe_layer_workspace_bytes, allocated when None."""
    if workspace is None:
        r = (_FAST or _fast()).moe_layer(x, logits, top_k, gate_up, down, gate_up_bias, down_bias, renormalize, out)
        if r is not None:
            return r if type(r) is not int else _check(r, "fp8w_moe_layer")
    dev = _gpu(x, "x", 2)
    _gpu(logits, "logits", 2)
    t, hidden = x.shape
    e = logits.shape[1]
    (qu, su), (qd, sd) = gate_up, down
    if qu.dim() != 3 or qd.dim() != 3 or qu.shape[1] % 2:
        raise ValueError("gate_up and down must be (q, scale) of [e, 2 inner, hidden] and [e, hidden, inner] weights")
    inner = qu.shape[1] // 2
    if t > MOE_LAYER_TOKENS:
        raise ValueError(f"moe_layer takes up to {MOE_LAYER_TOKENS} tokens, not {t}: call route, linear_experts "
                         "(linear_experts_fp4) and combine")
    if logits.dtype not in _DT:
        raise TypeError(f"logits must be bf16, fp16 or fp32, not {logits.dtype}")
    if not 1 <= top_k <= min(e, 64) or e > 1024:
        raise ValueError("expected 1 <= top_k <= min(e, 64) and e <= 1024")
    act = _act_code(x.dtype, "x")
    fp4 = su.dtype is torch.uint8
    xp = _want(x, "x", (t, hidden), x.dtype, dev)
    lp = _want(logits, "logits", (t, e), logits.dtype, dev)
    ptr = []
    for name, q, s, n, k in (("gate_up", qu, su, 2 * inner, hidden), ("down", qd, sd, hidden, inner)):
        ptr.append((_want(q, name + "[0]", (e, n, (k + 1) // 2 if fp4 else k), torch.uint8, dev),
                    _want(s, name + "[1]", (e, n, (k + 31) // 32) if fp4 else (e, n),
                          torch.uint8 if fp4 else torch.float32, dev)))
    ub = _want(gate_up_bias, "gate_up_bias", (e, 2 * inner), x.dtype, dev)
    db = _want(down_bias, "down_bias", (e, hidden), x.dtype, dev)
    if out is None:
        out = x.new_empty((t, hidden))
    op = _want(out, "out", (t, hidden), x.dtype, dev)
    workspace, wp, wb = _workspace(workspace, fp8w_moe_layer_workspace_bytes(t, e, top_k, hidden, inner), dev)
    with _on(dev):
        st = fp8w_moe_layer(xp, act, t, hidden, lp, _DT[logits.dtype], e, top_k, int(renormalize),
                            WEIGHT_FP4 if fp4 else WEIGHT_E4M3, *ptr[0], ub, inner, *ptr[1], db, op, wp, wb,
                            _stream(dev))
    _check(st, "fp8w_moe_layer")
    return out
