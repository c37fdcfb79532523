"""GB300 MoE expert layer: thin Python binding of the C ABI in ``include/moe.h``.

Every step of the layer runs in the CUDA kernels of ``libmoe.so``; this module only checks
and marshals arguments.  PyTorch provides device memory and streams.  There is no fallback:
if the library is not built, importing a plan raises.

    plan = MoePlan(E=256, k=8, d_model=2048, d_ff=512, n_shared=1)
    plan.set_weights(w_router, None, w_gate, w_up, w_down)    # device tensors
    plan.set_shared(512, ws_gate, ws_up, ws_down)
    plan.allocate_workspace(T_max=8195)
    out = plan.forward(x, n_prefill=2048)                    # x bf16 [T][d] on the GPU
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from .build import LIB as LIB_PATH

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_NOT_READY = 0, 1, 2, 3
MOE_ERR_WORKSPACE, MOE_ERR_CUDA, MOE_ERR_DEVICE, MOE_ERR_TIMEOUT = 4, 5, 6, 7
MOE_W_BF16, MOE_W_MXFP4, MOE_W_FP8 = 0, 1, 3
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}  # moe_dtype
FP8_BLOCK = 128  # elements (of a row), or rows and columns (of a weight), that share a scale
SCORES = {"softmax": 0, "sigmoid": 1}
PATHS = {"auto": 0, "simt": 1, "tc": 2}
DEVERR_EXPERT_RANGE, DEVERR_NONFINITE, DEVERR_TIMEOUT, DEVERR_SEGMENT, DEVERR_RANGE = 0x1, 0x2, 0x4, 0x8, 0x10

EXPORTED = (
    "moe_plan_create", "moe_plan_destroy", "moe_last_error", "moe_plan_set_weights", "moe_plan_set_shared",
    "moe_plan_workspace_bytes", "moe_plan_set_workspace", "moe_plan_set_path", "moe_layer_forward",
    "moe_route", "moe_route_logits", "moe_permute", "moe_experts", "moe_combine",
    "moe_plan_get_device_error", "moe_plan_enable_timing", "moe_plan_timing_report",
    "moe_plan_last_launch_count", "moe_compose_prefill", "moe_permute_static", "moe_selftest_wait_expiry",
    "moe_plan_resolved_path", "moe_quantize_rows", "moe_quantize_blocks", "moe_linear_create", "moe_linear_destroy",
    "moe_linear_set_weights", "moe_linear_workspace_bytes", "moe_linear_set_workspace", "moe_linear_forward",
    "moe_linear_forward_quantized", "moe_linear_get_device_error", "moe_layer_forward_routed",
    "moe_plan_set_routing", "moe_sort_rows", "moe_sort_rows_backward", "moe_combine_rows", "moe_combine_rows_backward",
    "moe_verify_drafts", "moe_adapters_create", "moe_adapters_destroy", "moe_adapters_set", "moe_adapters_workspace_bytes",
    "moe_adapters_set_workspace", "moe_adapters_forward", "moe_adapters_get_device_error",
)

_lib = None


class PrefillCall(ctypes.Structure):
    """moe_prefill_call: one layer call of a prompt's prefill."""
    _fields_ = [("pos", ctypes.c_int64), ("n", ctypes.c_int32), ("piece", ctypes.c_int32)]


class Routing(ctypes.Structure):
    """moe_routing: how a plan scores and selects experts."""
    _fields_ = [("score", ctypes.c_int), ("bias", ctypes.c_void_p), ("n_groups", ctypes.c_int),
                ("topk_groups", ctypes.c_int), ("group_top", ctypes.c_int), ("renormalize", ctypes.c_int),
                ("scale", ctypes.c_float)]


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"moe status {status}: {msg}")
        self.status = status


def load_library(path: str = LIB_PATH):
    """Load libmoe.so (built by ``decode_batches_gb300.build``).  Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m decode_batches_gb300.build` "
                          "(there is no CPU or eager fallback)")
    lib = ctypes.CDLL(path)
    vp, i32, sz, u32p = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.POINTER(ctypes.c_uint32)
    i64 = ctypes.c_int64
    sig = {
        "moe_plan_create": ([i32, i32, i32, i32, i32, i32], vp),
        "moe_plan_destroy": ([vp], None),
        "moe_last_error": ([], ctypes.c_char_p),
        "moe_plan_set_weights": ([vp] * 9, i32),
        "moe_plan_set_shared": ([vp, i32, vp, vp, vp], i32),
        "moe_plan_workspace_bytes": ([vp, i32], sz),
        "moe_plan_set_workspace": ([vp, vp, sz, i32], i32),
        "moe_plan_set_path": ([vp, i32], i32),
        "moe_layer_forward": ([vp, vp, i32, i32, vp, vp], i32),
        "moe_plan_set_routing": ([vp, ctypes.POINTER(Routing)], i32),
        "moe_layer_forward_routed": ([vp, vp, i32, vp, vp, vp, vp], i32),
        "moe_route": ([vp, vp, i32, vp, vp, vp, vp], i32),
        "moe_route_logits": ([vp, vp, i32, vp, vp, vp], i32),
        "moe_permute": ([vp, vp, i32, vp, vp, vp, vp, vp], i32),
        "moe_experts": ([vp, vp, i32, vp, vp, vp, vp, vp], i32),
        "moe_combine": ([vp, vp, vp, vp, vp, i32, vp, vp], i32),
        "moe_plan_get_device_error": ([vp, u32p], i32),
        "moe_plan_enable_timing": ([vp, i32], i32),
        "moe_plan_timing_report": ([vp, ctypes.c_char_p, sz], sz),
        "moe_plan_last_launch_count": ([vp], i32),
        "moe_plan_resolved_path": ([vp], i32),
        "moe_compose_prefill": ([ctypes.c_int64, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                 ctypes.POINTER(PrefillCall), ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)], i32),
    }
    sig.update({
        "moe_quantize_rows": ([vp, i32, i64, i32, i32, vp, i64, vp, i64, vp], i32),
        "moe_quantize_blocks": ([vp, i32, i32, i32, vp, vp, vp], i32),
        "moe_linear_create": ([i32, i32], vp),
        "moe_linear_destroy": ([vp], None),
        "moe_linear_set_weights": ([vp, vp, vp], i32),
        "moe_linear_workspace_bytes": ([vp, i32], sz),
        "moe_linear_set_workspace": ([vp, vp, sz, i32], i32),
        "moe_linear_forward": ([vp, vp, i32, i64, i32, vp, i32, i64, vp], i32),
        "moe_linear_forward_quantized": ([vp, vp, i64, vp, i64, i32, vp, i32, i64, vp], i32),
        "moe_linear_get_device_error": ([vp, u32p], i32),
        "moe_sort_rows": ([vp, i32, i64, i32, i32, i32, vp, vp, vp, i64, i64, vp], i32),
        "moe_sort_rows_backward": ([vp, i32, i64, i64, i32, i32, i32, vp, vp, vp, i64, vp, i64, vp, vp], i32),
        "moe_combine_rows": ([vp, i32, i64, i64, i32, i32, i32, vp, vp, vp, i32, i64, vp, i32, i64, vp], i32),
        "moe_combine_rows_backward": ([vp, i32, i64, i32, i32, i32, vp, vp, vp, i64, vp, i32, i64, i64, vp, vp], i32),
        "moe_verify_drafts": ([vp, i32, i64, vp, i64, i32, i32, vp, vp, i32, vp, vp, vp, vp, vp], i32),
        "moe_adapters_create": ([i32, i32, i32, i32, i32], vp),
        "moe_adapters_destroy": ([vp], None),
        "moe_adapters_set": ([vp, i32, vp, vp, i32, ctypes.c_float], i32),
        "moe_adapters_workspace_bytes": ([vp, i32], sz),
        "moe_adapters_set_workspace": ([vp, vp, sz, i32], i32),
        "moe_adapters_forward": ([vp, vp, i64, i32, vp, vp, i64, vp, i32, i64, vp], i32),
        "moe_adapters_get_device_error": ([vp, u32p], i32),
    })
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def compose_prefill(start_pos: int, n_tokens: int, quantum: int, generation_active: bool,
                    prefill_cap: int = 4096):
    """The layer calls that prefill ``n_tokens`` prompt tokens from context position
    ``start_pos`` (moe_compose_prefill): a list of (pos, n, piece) tuples, in order."""
    lib = load_library()
    total = ctypes.c_int64(0)
    _check(lib.moe_compose_prefill(start_pos, n_tokens, quantum, int(bool(generation_active)), prefill_cap, None, 0,
                                   ctypes.byref(total)))
    arr = (PrefillCall * max(1, total.value))()
    _check(lib.moe_compose_prefill(start_pos, n_tokens, quantum, int(bool(generation_active)), prefill_cap, arr,
                                   total.value, ctypes.byref(total)))
    return [(c.pos, c.n, c.piece) for c in arr[:total.value]]


def _check(status: int):
    if status != MOE_OK:
        raise MoeError(status, load_library().moe_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()  # an int: the argument types of load_library make it a pointer


def _dev(t: Optional[torch.Tensor], name: str, dtype=None, shape=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return _ptr(t)


# A call that is given a stream runs under it (torch.cuda.stream), so that what it allocates, fills or
# copies lies in memory that this stream uses, in the order of its work: the current stream's pool could
# hand out memory that work queued there still reads.
# The current stream's handle without a Stream object around it (3 us of a small call's host time on
# a Grace core), where this torch has the call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream():
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _rows(t: torch.Tensor, name: str, dtypes, width: int):
    """(pointer, row pitch in elements) of a 2-D CUDA tensor [rows][width] whose rows are dense."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {[str(d) for d in dtypes]}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2 or shape[1] != width:
        raise ValueError(f"{name} must have shape (rows, {width}), got {tuple(shape)}")
    pitch, step = t.stride()
    if step != 1 and shape[0] and width > 1:
        raise ValueError(f"{name} must have dense rows")
    if shape[0] <= 1:  # with one row (or none) the pitch is never used to step; keep it valid
        pitch = max(pitch, width)
    return t.data_ptr(), pitch


def _blocks(n: int) -> int:
    return -(-n // FP8_BLOCK)


def quantize_fp8(x: torch.Tensor, stream=None):
    """Rows x [T][K] (bf16, fp16 or fp32, any row pitch) as e4m3 codes [T][K] and fp32 scales
    [T][ceil(K/128)] of 1 x 128 blocks (moe_quantize_rows).  Both are views of padded rows, as
    ``Fp8Linear.forward_quantized`` takes them."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return quantize_fp8(x)
    lib = load_library()
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D, got {tuple(x.shape)}")
    T, K = x.shape
    if K < 1:
        raise ValueError("x must have at least one column")
    px, ldx = _rows(x, "x", DTYPES, K)
    nb = _blocks(K)
    q = torch.empty((T, nb * FP8_BLOCK), dtype=torch.float8_e4m3fn, device=x.device)
    s = torch.empty((T, (nb + 3) // 4 * 4), dtype=torch.float32, device=x.device)
    _check(lib.moe_quantize_rows(px, DTYPES[x.dtype], ldx, T, K, _ptr(q), q.shape[1], _ptr(s), s.shape[1],
                                 _stream()))
    return q[:, :K], s[:, :nb]


def quantize_fp8_weight(w: torch.Tensor, stream=None):
    """A weight [..., rows, K] as e4m3 codes of the same shape and fp32 scales
    [..., ceil(rows/128), ceil(K/128)] of 128 x 128 blocks (moe_quantize_blocks, a call per matrix)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return quantize_fp8_weight(w)
    lib = load_library()
    if w.dim() < 2 or w.shape[-1] < 1:
        raise ValueError(f"w must be a matrix or a batch of matrices, got {tuple(w.shape)}")
    if not w.is_cuda or w.dtype not in DTYPES:
        raise ValueError("w must be a CUDA tensor of bf16, fp16 or fp32")
    rows, K = w.shape[-2:]
    w = w.contiguous()
    q = torch.empty(w.shape, dtype=torch.float8_e4m3fn, device=w.device)
    s = torch.empty((*w.shape[:-2], _blocks(rows), _blocks(K)), dtype=torch.float32, device=w.device)
    if w.numel() == 0:
        return q, s
    for wm, qm, sm in zip(w.view(-1, rows, K), q.view(-1, rows, K), s.view(-1, s.shape[-2], s.shape[-1])):
        _check(lib.moe_quantize_blocks(_ptr(wm), DTYPES[w.dtype], rows, K, _ptr(qm), _ptr(sm), _stream()))
    return q, s


def _here(*tensors):
    """The current device, which has to be the tensors' (launches go to its current stream)."""
    dev = torch._C._cuda_getDevice()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors must be on the current CUDA device ({dev}), got {t.device}")


def _row_args(t: torch.Tensor, name: str, dtypes, rows: Optional[int], width: int):
    """``_rows`` for a tensor whose device is known, with a number of rows (None: any)."""
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {[str(d) for d in dtypes]}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2 or shape[1] != width or (rows is not None and shape[0] != rows) or shape[0] > 0x7fffffff:
        raise ValueError(f"{name} must have shape ({'rows' if rows is None else rows}, {width}), got {tuple(shape)}")
    pitch, step = t.stride()
    if step != 1 and shape[0] and width > 1:
        raise ValueError(f"{name} must have dense rows")
    if shape[0] <= 1 and pitch < width:  # with one row (or none) the pitch is never used to step; keep it valid
        pitch = width
    return t.data_ptr(), pitch


def _assignments(inv: torch.Tensor, weights: Optional[torch.Tensor]):
    """(T, k, inv's pointer, weights' pointer) of the assignments' rows."""
    shape = inv.shape
    if len(shape) != 2:
        raise ValueError(f"inv must have shape (T, k), got {tuple(shape)}")
    T, k = shape
    if inv.dtype is not torch.int32 or T > 0x7fffffff:
        raise ValueError(f"inv must be torch.int32 with fewer than 2^31 rows, got {inv.dtype} {tuple(shape)}")
    if weights is None:
        return T, k, _ptr(inv), None
    if weights.dtype is not torch.float32 or weights.shape != shape:
        raise ValueError(f"weights must be torch.float32 of shape {tuple(shape)}, got {weights.dtype} {tuple(weights.shape)}")
    return T, k, _ptr(inv), _ptr(weights)


def _vector(t: torch.Tensor, name: str, dtype, n: int):
    """The pointer of a dense vector of n elements whose device is known."""
    if t.dtype is not dtype or t.shape != (n,):
        raise ValueError(f"{name} must be {dtype} of shape ({n},), got {t.dtype} {tuple(t.shape)}")
    return _ptr(t)


def _outside(out: torch.Tensor, *inputs):
    """out must not share memory with an input: their extents are compared, and where both are rows of one pitch (parts of
    one wide buffer) their columns."""
    def extent(t):
        n = 1 + sum((s - 1) * st for s, st in zip(t.shape, t.stride()))
        return t.data_ptr(), t.data_ptr() + n * t.element_size()
    base = out.untyped_storage().data_ptr()
    for t in inputs:
        if t is not None and t.untyped_storage().data_ptr() == base and t.numel() and out.numel():
            (lo, hi), (a, b) = extent(out), extent(t)
            if not (a < hi and lo < b):
                continue
            if t.dim() == out.dim() == 2 and t.stride() == out.stride() and t.element_size() == out.element_size():
                pitch, off = out.stride(0), (a - lo) // out.element_size() % max(1, out.stride(0))
                if out.shape[1] <= off and off + t.shape[1] <= pitch:
                    continue
            raise ValueError("an output overlaps an input")


def _lost_gradient(call: str):
    """A call whose result has no gradient of its own, given tensors that want one: refused rather than detached."""
    if torch.is_grad_enabled():
        raise ValueError(f"{call} does not record its gradient: call it under torch.no_grad(), or in a torch.autograd.Function "
                         f"whose backward calls {call}_backward")


def sort_rows(x: torch.Tensor, inv: torch.Tensor, weights: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None, stream=None):
    """Token rows x [T][d] (bf16, fp16 or fp32, any row pitch) in expert order: out[inv[t, j]] = weights[t, j] x[t]
    (moe_sort_rows).  inv int32 [T][k] is ``MoePlan.permute``'s, viewed as (T, k); -1: dropped.  out [rows][d] of
    x's type (default T * k rows) keeps the rows that no entry names; a new one's are undefined.  Tensors that require
    a gradient are refused while gradients are recorded: ``sort_rows_backward`` computes it."""
    if x.requires_grad or (weights is not None and weights.requires_grad):
        _lost_gradient("sort_rows")
    if stream is not None:
        with torch.cuda.stream(stream):
            return sort_rows(x, inv, weights, out)
    _here(x, inv, weights, out)
    T, k, pi, pw = _assignments(inv, weights)
    d = x.shape[-1]
    px, ldx = _row_args(x, "x", DTYPES, T, d)
    if out is None:
        out = torch.empty((T * k, d), dtype=x.dtype, device=x.device)
        po, ldo = out.data_ptr(), d
    else:
        _outside(out, x, inv, weights)
        po, ldo = _row_args(out, "out", (x.dtype,), None, d)
    _check(load_library().moe_sort_rows(px, DTYPES[x.dtype], ldx, T, k, d, pi, pw, po, ldo, out.shape[0], _stream()))
    return out


def sort_rows_backward(grad: torch.Tensor, inv: torch.Tensor, weights: Optional[torch.Tensor] = None,
                       x: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, stream=None):
    """The gradient of ``sort_rows``: grad [rows][d] in expert order -> dx [T][d] (dx[t] = sum_j weights[t, j]
    grad[inv[t, j]]) and, when x is given, (dx, dweights) with dweights[t, j] = <x[t], grad[inv[t, j]]> in fp32."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return sort_rows_backward(grad, inv, weights, x, out)
    _here(grad, inv, weights, x, out)
    T, k, pi, pw = _assignments(inv, weights)
    d = grad.shape[-1]
    pg, ldg = _row_args(grad, "grad", DTYPES, None, d)
    px = ldx = dw = None
    if x is not None:
        px, ldx = _row_args(x, "x", (grad.dtype,), T, d)
        dw = torch.empty((T, k), dtype=torch.float32, device=grad.device)
    if out is None:
        out = torch.empty((T, d), dtype=grad.dtype, device=grad.device)
        po, ldo = out.data_ptr(), d
    else:
        _outside(out, grad, inv, weights, x)
        po, ldo = _row_args(out, "out", (grad.dtype,), T, d)
    _check(load_library().moe_sort_rows_backward(pg, DTYPES[grad.dtype], ldg, grad.shape[0], T, k, d, pi, pw, px, ldx or 0,
                                                 po, ldo, _ptr(dw), _stream()))
    return out if dw is None else (out, dw)


def combine_rows(y: torch.Tensor, inv: torch.Tensor, weights: Optional[torch.Tensor] = None,
                 shared: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, out_dtype=None, stream=None):
    """Rows y [rows][d] in expert order back to the tokens: out[t] = sum_j weights[t, j] y[inv[t, j]] + shared[t]
    (moe_combine_rows), in out_dtype (default y's).  y, shared and out: bf16, fp16 or fp32 each, any row pitch.  Tensors
    that require a gradient are refused while gradients are recorded: ``combine_rows_backward`` computes it."""
    if y.requires_grad or (weights is not None and weights.requires_grad) or (shared is not None and shared.requires_grad):
        _lost_gradient("combine_rows")
    if stream is not None:
        with torch.cuda.stream(stream):
            return combine_rows(y, inv, weights, shared, out, out_dtype)
    _here(y, inv, weights, shared, out)
    T, k, pi, pw = _assignments(inv, weights)
    d = y.shape[-1]
    py, ldy = _row_args(y, "y", DTYPES, None, d)
    ps, lds, sdt = None, 0, 0
    if shared is not None:
        ps, lds = _row_args(shared, "shared", DTYPES, T, d)
        sdt = DTYPES[shared.dtype]
    if out is None:
        if out_dtype is not None and out_dtype not in DTYPES:
            raise ValueError(f"out must be bf16, fp16 or fp32, got {out_dtype}")
        out = torch.empty((T, d), dtype=out_dtype or y.dtype, device=y.device)
        po, ldo = out.data_ptr(), d
    else:
        _outside(out, y, inv, weights, shared)
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError(f"out must be {out_dtype}, got {out.dtype}")
        po, ldo = _row_args(out, "out", DTYPES, T, d)
    _check(load_library().moe_combine_rows(py, DTYPES[y.dtype], ldy, y.shape[0], T, k, d, pi, pw, ps, sdt, lds, po,
                                           DTYPES[out.dtype], ldo, _stream()))
    return out


def combine_rows_backward(grad: torch.Tensor, inv: torch.Tensor, weights: Optional[torch.Tensor] = None,
                          y: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, stream=None):
    """The gradient of ``combine_rows``: grad [T][d] -> dy [rows][d] in expert order (dy[inv[t, j]] = weights[t, j]
    grad[t]) and, when y is given, (dy, dweights) with dweights[t, j] = <grad[t], y[inv[t, j]]> in fp32.  dy has y's
    type and rows (without y: out's, or T * k rows of grad's type); rows that no entry names keep out's contents, in
    a new dy they are undefined.  The gradient of ``shared`` is grad itself."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return combine_rows_backward(grad, inv, weights, y, out)
    _here(grad, inv, weights, y, out)
    T, k, pi, pw = _assignments(inv, weights)
    d = grad.shape[-1]
    pg, ldg = _row_args(grad, "grad", DTYPES, T, d)
    py = ldy = dw = None
    if y is not None:
        py, ldy = _row_args(y, "y", DTYPES, None, d)
        dw = torch.empty((T, k), dtype=torch.float32, device=grad.device)
    if out is None:
        out = torch.empty((T * k if y is None else y.shape[0], d), dtype=(grad if y is None else y).dtype, device=grad.device)
        po, ldo = out.data_ptr(), d
    else:
        _outside(out, grad, inv, weights, y)
        po, ldo = _row_args(out, "out", DTYPES if y is None else (y.dtype,), None if y is None else y.shape[0], d)
    _check(load_library().moe_combine_rows_backward(pg, DTYPES[grad.dtype], ldg, T, k, d, pi, pw, py, ldy or 0, po,
                                                    DTYPES[out.dtype], ldo, out.shape[0], _ptr(dw), _stream()))
    return out if dw is None else (out, dw)


def verify_drafts(target: torch.Tensor, drafts: torch.Tensor, offsets: torch.Tensor, u: torch.Tensor,
                  u_sample: torch.Tensor, draft_probs: Optional[torch.Tensor] = None,
                  tokens: Optional[torch.Tensor] = None, accepted: Optional[torch.Tensor] = None, stream=None):
    """Drafted tokens against the target's probabilities, from given uniform numbers (moe_verify_drafts).

    target [R][V] (bf16, fp16 or fp32, any row pitch): the probabilities of a step's verify rows; offsets int32
    [B + 1]: request b owns rows offsets[b] .. offsets[b + 1] - 1, one a draft and one behind the last; drafts int32
    [R]; draft_probs like target, or None for drafts that were certain; u fp32 [R] decides the drafts, u_sample fp32
    [B] draws the token behind the accepted ones.  Returns (tokens int32 [R], accepted int32 [B]): in a request's
    rows the accepted drafts, the drawn token, then -1.  Rows of no request keep the contents of tokens; in a
    new tensor they are undefined."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return verify_drafts(target, drafts, offsets, u, u_sample, draft_probs, tokens, accepted)
    _here(target, drafts, offsets, u, u_sample, draft_probs, tokens, accepted)
    if target.dim() != 2 or u_sample.dim() != 1:
        raise ValueError(f"target must be 2-D and u_sample 1-D, got {tuple(target.shape)} and {tuple(u_sample.shape)}")
    (R, V), B = target.shape, u_sample.shape[0]
    pt, ldt = _row_args(target, "target", DTYPES, R, V)
    pd = ldd = None
    if draft_probs is not None:
        pd, ldd = _row_args(draft_probs, "draft_probs", (target.dtype,), R, V)
    i32, f32, dev = torch.int32, torch.float32, target.device
    if tokens is None:
        tokens = torch.empty((R,), dtype=i32, device=dev)
    else:
        _outside(tokens, target, drafts, offsets, u, u_sample, draft_probs)
    if accepted is None:
        accepted = torch.empty((B,), dtype=i32, device=dev)
    else:
        _outside(accepted, target, drafts, offsets, u, u_sample, draft_probs, tokens)
    _check(load_library().moe_verify_drafts(
        pt, DTYPES[target.dtype], ldt, pd, ldd or 0, R, V, _vector(drafts, "drafts", i32, R),
        _vector(offsets, "offsets", i32, B + 1), B, _vector(u, "u", f32, R), _vector(u_sample, "u_sample", f32, B),
        _vector(tokens, "tokens", i32, R), _vector(accepted, "accepted", i32, B), _stream()))
    return tokens, accepted


class Fp8Linear:
    """A projection with e4m3 weights and a scale for each block of 128 x 128 (C ABI ``moe_linear``).

        lin = Fp8Linear(N, K)
        lin.set_weights(*quantize_fp8_weight(w))     # w [N][K]
        lin.allocate_workspace(T_max)
        out = lin.forward(x)                         # x [T][K] -> [T][N]
    """

    def __init__(self, N: int, K: int):
        self.lib = load_library()
        self.N, self.K = N, K
        h = self.lib.moe_linear_create(N, K)
        if not h:
            raise MoeError(MOE_ERR_INVALID_ARG, self.lib.moe_last_error().decode())
        self._h = ctypes.c_void_p(h)
        self._ws = None
        self.T_max = 0

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            self.lib.moe_linear_destroy(h)
            self._h = None

    close = __del__

    def set_weights(self, q: torch.Tensor, s: torch.Tensor):
        _check(self.lib.moe_linear_set_weights(
            self._h, _dev(q, "q", torch.float8_e4m3fn, (self.N, self.K)),
            _dev(s, "s", torch.float32, (_blocks(self.N), _blocks(self.K)))))

    def workspace_bytes(self, T_max: int) -> int:
        return int(self.lib.moe_linear_workspace_bytes(self._h, T_max))

    def set_workspace(self, buf: torch.Tensor, T_max: int):
        _check(self.lib.moe_linear_set_workspace(self._h, _dev(buf, "workspace"), buf.numel() * buf.element_size(), T_max))
        self._ws = buf
        self.T_max = T_max

    def allocate_workspace(self, T_max: int, device=None) -> torch.Tensor:
        buf = torch.empty(self.workspace_bytes(T_max), dtype=torch.uint8, device=device or "cuda")
        self.set_workspace(buf, T_max)
        return buf

    def _out(self, T, out, out_dtype, device):
        if out is None:
            if out_dtype not in (torch.bfloat16, torch.float32):
                raise ValueError(f"out must be bf16 or fp32, got {out_dtype}")
            out = torch.empty((T, self.N), dtype=out_dtype, device=device)
            return out, out.data_ptr(), self.N
        if out.shape[0] != T:
            raise ValueError(f"out must have {T} rows, got {out.shape[0]}")
        return out, *_rows(out, "out", (torch.bfloat16, torch.float32), self.N)

    def forward(self, x: torch.Tensor, out: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16, stream=None,
                adapters: Optional["LowRankAdapters"] = None, adapter_ids: Optional[torch.Tensor] = None):
        """x [T][K] (bf16, fp16 or fp32; rows may have a pitch) -> [T][N] in bf16 or fp32.  With adapters (of the same N
        and K, x in their type) and adapter_ids int32 [T], each row's adapter is added to the rounded projection."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.forward(x, out, out_dtype, None, adapters, adapter_ids)
        if (adapters is None) != (adapter_ids is None):
            raise ValueError("adapters and adapter_ids go together")
        if adapters is not None:
            adapters._beside(self, x, adapter_ids, out)
        px, ldx = _rows(x, "x", DTYPES, self.K)
        T = x.shape[0]
        out, po, ldo = self._out(T, out, out_dtype, x.device)
        _check(self.lib.moe_linear_forward(self._h, px, DTYPES[x.dtype], ldx, T, po, DTYPES[out.dtype], ldo, _stream()))
        if adapters is not None:
            adapters.forward(x, adapter_ids, out, out=out)
        return out

    def forward_quantized(self, q: torch.Tensor, s: torch.Tensor, out: Optional[torch.Tensor] = None,
                          out_dtype=torch.bfloat16, stream=None):
        """The same for rows that ``quantize_fp8`` already quantised (several projections of one x)."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.forward_quantized(q, s, out, out_dtype)
        pq, ldq = _rows(q, "q", (torch.float8_e4m3fn,), self.K)
        ps, lds = _rows(s, "s", (torch.float32,), _blocks(self.K))
        T = q.shape[0]
        if s.shape[0] != T:
            raise ValueError(f"s must have {T} rows, got {s.shape[0]}")
        if T == 1:  # a single row: its pitch may be anything; only its padding to the vector width matters
            ldq, lds = (ldq + 15) // 16 * 16, (lds + 3) // 4 * 4
        out, po, ldo = self._out(T, out, out_dtype, q.device)
        _check(self.lib.moe_linear_forward_quantized(self._h, pq, ldq, ps, lds, T, po, DTYPES[out.dtype], ldo,
                                                     _stream()))
        return out

    def device_error(self) -> int:
        code = ctypes.c_uint32(0)
        st = self.lib.moe_linear_get_device_error(self._h, ctypes.byref(code))
        if st not in (MOE_OK, MOE_ERR_DEVICE):
            _check(st)
        return int(code.value)


class LowRankAdapters:
    """Low-rank adapters of many requests beside a shared projection (C ABI ``moe_adapters``).

        ad = LowRankAdapters(n, N, K, rank)          # n slots for A [r][K], B [N][r], r <= rank
        ad.set(slot, A, B, scale)
        ad.allocate_workspace(T_max)
        out = ad.forward(x, ids, base)               # base[t] + scale_a B_a (A_a x[t]), a = ids[t] (-1: none)
        out = lin.forward(x, adapters=ad, adapter_ids=ids)    # beside an Fp8Linear
    """

    def __init__(self, n: int, N: int, K: int, rank: int, dtype=torch.bfloat16):
        self.lib = load_library()
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"dtype must be bf16 or fp16, got {dtype}")
        self.n, self.N, self.K, self.rank, self.dtype = n, N, K, rank, dtype
        h = self.lib.moe_adapters_create(n, N, K, rank, DTYPES[dtype])
        if not h:
            raise MoeError(MOE_ERR_INVALID_ARG, self.lib.moe_last_error().decode())
        self._h = ctypes.c_void_p(h)
        self._ws = None
        self.T_max = 0

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            self.lib.moe_adapters_destroy(h)
            self._h = None

    close = __del__

    def set(self, slot: int, A: torch.Tensor, B: torch.Tensor, scale: float = 1.0):
        """A [r][K] and B [N][r] of the handle's type into slot `slot` (copied; synchronous)."""
        _here(A, B)
        if A.dim() != 2:
            raise ValueError(f"A must be 2-D, got {tuple(A.shape)}")
        self._slot(slot)
        r = A.shape[0]
        _check(self.lib.moe_adapters_set(self._h, slot, _dev(A, "A", self.dtype, (r, self.K)),
                                         _dev(B, "B", self.dtype, (self.N, r)), r, scale))

    def clear(self, slot: int):
        """Empty slot `slot`: rows that ask for it get the base alone."""
        self._slot(slot)
        _check(self.lib.moe_adapters_set(self._h, slot, None, None, 0, 1.0))

    def _slot(self, slot: int):
        if not 0 <= slot < self.n:
            raise ValueError(f"slot must be in [0, {self.n}), got {slot}")

    def workspace_bytes(self, T_max: int) -> int:
        return int(self.lib.moe_adapters_workspace_bytes(self._h, T_max))

    def set_workspace(self, buf: torch.Tensor, T_max: int):
        _here(buf)
        _check(self.lib.moe_adapters_set_workspace(self._h, _dev(buf, "workspace"), buf.numel() * buf.element_size(), T_max))
        self._ws = buf
        self.T_max = T_max

    def allocate_workspace(self, T_max: int, device=None) -> torch.Tensor:
        buf = torch.empty(self.workspace_bytes(T_max), dtype=torch.uint8, device=device or "cuda")
        self.set_workspace(buf, T_max)
        return buf

    def _beside(self, lin, x, ids, out):
        """The checks of a projection's call with these adapters, before anything of it is queued."""
        if (lin.N, lin.K) != (self.N, self.K):
            raise ValueError(f"adapters of {self.N} x {self.K} beside a projection of {lin.N} x {lin.K}")
        _here(x, ids)
        _row_args(x, "x", (self.dtype,), None, self.K)
        _dev(ids, "adapter_ids", torch.int32, (x.shape[0],))
        if x.shape[0] > self.T_max:
            raise ValueError(f"the adapters' workspace holds {self.T_max} rows, got {x.shape[0]}")
        if out is not None:
            _here(out)
            _outside(out, x, ids)

    def forward(self, x: torch.Tensor, ids: torch.Tensor, base: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, out_dtype=None, stream=None):
        """x [T][K] of the handle's type, ids int32 [T], base [T][N] (None: zero) -> [T][N] in base's type, else in
        out_dtype (default the handle's).  Rows may have a pitch; out may be base."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.forward(x, ids, base, out, out_dtype)
        _here(x, ids, base, out)
        px, ldx = _row_args(x, "x", (self.dtype,), None, self.K)
        T = x.shape[0]
        pb, ldb = None, 0
        if base is not None:
            if out_dtype is not None and out_dtype != base.dtype:
                raise ValueError(f"out has base's type {base.dtype}, got {out_dtype}")
            out_dtype = base.dtype
            pb, ldb = _row_args(base, "base", DTYPES, T, self.N)
        if out is None:
            out = torch.empty((T, self.N), dtype=out_dtype or self.dtype, device=x.device)
            if out.dtype not in DTYPES:
                raise ValueError(f"out must be bf16, fp16 or fp32, got {out.dtype}")
            po, ldo = out.data_ptr(), self.N
        else:
            po, ldo = _row_args(out, "out", DTYPES if out_dtype is None else (out_dtype,), T, self.N)
            _outside(out, x, ids, base if pb != po or ldb != ldo else None)
        _check(self.lib.moe_adapters_forward(self._h, px, ldx, T, _vector(ids, "ids", torch.int32, T), pb, ldb, po,
                                             DTYPES[out.dtype], ldo, _stream()))
        return out

    def device_error(self) -> int:
        code = ctypes.c_uint32(0)
        st = self.lib.moe_adapters_get_device_error(self._h, ctypes.byref(code))
        if st not in (MOE_OK, MOE_ERR_DEVICE):
            _check(st)
        return int(code.value)


class MoePlan:
    """One MoE layer plan (C ABI ``moe_plan``)."""

    def __init__(self, E: int, k: int, d_model: int, d_ff: int, n_shared: int = 0, weight_dtype: str = "bf16"):
        self.lib = load_library()
        wd = {"bf16": MOE_W_BF16, "mxfp4": MOE_W_MXFP4, "fp8": MOE_W_FP8}[weight_dtype]
        self.E, self.k, self.d, self.f, self.n_shared, self.weight_dtype = E, k, d_model, d_ff, n_shared, weight_dtype
        self.f_s = 0
        h = self.lib.moe_plan_create(E, k, d_model, d_ff, n_shared, wd)
        if not h:
            raise MoeError(MOE_ERR_INVALID_ARG, self.lib.moe_last_error().decode())
        self._h = ctypes.c_void_p(h)
        self._ws = None
        self.T_max = 0

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            self.lib.moe_plan_destroy(h)
            self._h = None

    close = __del__

    # ---- set-up -------------------------------------------------------------------------------
    def set_weights(self, w_router, b_router, w_gate, w_up, w_down, s_gate=None, s_up=None, s_down=None):
        E, d, f = self.E, self.d, self.f
        args = [_dev(w_router, "w_router", torch.float32, (E, d)),
                _dev(b_router, "b_router", torch.float32, (E,))]
        if self.weight_dtype == "bf16":
            args += [_dev(w_gate, "w_gate", torch.bfloat16, (E, f, d)), _dev(w_up, "w_up", torch.bfloat16, (E, f, d)),
                     _dev(w_down, "w_down", torch.bfloat16, (E, d, f)), None, None, None]
        elif self.weight_dtype == "fp8":
            f8, bd, bf = torch.float8_e4m3fn, _blocks(d), _blocks(f)
            args += [_dev(w_gate, "w_gate", f8, (E, f, d)), _dev(w_up, "w_up", f8, (E, f, d)),
                     _dev(w_down, "w_down", f8, (E, d, f)),
                     _dev(s_gate, "s_gate", torch.float32, (E, bf, bd)), _dev(s_up, "s_up", torch.float32, (E, bf, bd)),
                     _dev(s_down, "s_down", torch.float32, (E, bd, bf))]
        else:
            args += [_dev(w_gate, "w_gate", torch.uint8, (E, f, d // 2)), _dev(w_up, "w_up", torch.uint8, (E, f, d // 2)),
                     _dev(w_down, "w_down", torch.uint8, (E, d, f // 2)),
                     _dev(s_gate, "s_gate", torch.uint8, (E, f, d // 32)), _dev(s_up, "s_up", torch.uint8, (E, f, d // 32)),
                     _dev(s_down, "s_down", torch.uint8, (E, d, f // 32))]
        _check(self.lib.moe_plan_set_weights(self._h, *args))

    def set_shared(self, d_ff_shared: int, w_gate, w_up, w_down):
        n, d, fs = self.n_shared, self.d, d_ff_shared
        _check(self.lib.moe_plan_set_shared(self._h, fs, _dev(w_gate, "w_gate", torch.bfloat16, (n, fs, d)),
                                            _dev(w_up, "w_up", torch.bfloat16, (n, fs, d)),
                                            _dev(w_down, "w_down", torch.bfloat16, (n, d, fs))))
        self.f_s = fs

    def workspace_bytes(self, T_max: int) -> int:
        return int(self.lib.moe_plan_workspace_bytes(self._h, T_max))

    def set_workspace(self, buf: torch.Tensor, T_max: int):
        _check(self.lib.moe_plan_set_workspace(self._h, _dev(buf, "workspace"), buf.numel() * buf.element_size(), T_max))
        self._ws = buf
        self.T_max = T_max

    def allocate_workspace(self, T_max: int, device=None) -> torch.Tensor:
        buf = torch.empty(self.workspace_bytes(T_max), dtype=torch.uint8, device=device or "cuda")
        self.set_workspace(buf, T_max)
        return buf

    def set_path(self, path: str):
        _check(self.lib.moe_plan_set_path(self._h, PATHS[path]))

    def set_routing(self, score: Optional[str] = "softmax", bias: Optional[torch.Tensor] = None, n_groups: int = 1,
                    topk_groups: int = 1, group_top: int = 1, renormalize: bool = True, scale: float = 1.0):
        """Score and select experts as moe_plan_set_routing says; score=None restores the default
        (the softmax of the k largest logits)."""
        if score is None:
            _check(self.lib.moe_plan_set_routing(self._h, None))
            return
        r = Routing(SCORES[score], _dev(bias, "bias", torch.float32, (self.E,)), n_groups, topk_groups, group_top,
                    int(bool(renormalize)), scale)
        _check(self.lib.moe_plan_set_routing(self._h, ctypes.byref(r)))

    # ---- step ---------------------------------------------------------------------------------
    def forward(self, x: torch.Tensor, n_prefill: int = 0, out: Optional[torch.Tensor] = None, stream=None):
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.forward(x, n_prefill, out)
        T = x.shape[0]
        if out is None:
            out = torch.empty((T, self.d), dtype=torch.bfloat16, device=x.device)
        _check(self.lib.moe_layer_forward(self._h, _dev(x, "x", torch.bfloat16, (T, self.d)), T, n_prefill,
                                          _dev(out, "out", torch.bfloat16, (T, self.d)), _stream()))
        return out

    def forward_routed(self, x: torch.Tensor, ids: torch.Tensor, gates: torch.Tensor,
                       out: Optional[torch.Tensor] = None, stream=None):
        """The layer for given ids and gates [T][k] (moe_layer_forward_routed)."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.forward_routed(x, ids, gates, out)
        T = x.shape[0]
        if out is None:
            out = torch.empty((T, self.d), dtype=torch.bfloat16, device=x.device)
        _check(self.lib.moe_layer_forward_routed(self._h, _dev(x, "x", torch.bfloat16, (T, self.d)), T,
                                                 _dev(ids, "ids", torch.int32, (T, self.k)),
                                                 _dev(gates, "gates", torch.float32, (T, self.k)),
                                                 _dev(out, "out", torch.bfloat16, (T, self.d)), _stream()))
        return out

    def route(self, x: torch.Tensor, want_logits: bool = True, stream=None):
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.route(x, want_logits)
        T = x.shape[0]
        dev = x.device
        logits = torch.empty((T, self.E), dtype=torch.float32, device=dev) if want_logits else None
        ids = torch.empty((T, self.k), dtype=torch.int32, device=dev)
        gates = torch.empty((T, self.k), dtype=torch.float32, device=dev)
        _check(self.lib.moe_route(self._h, _dev(x, "x", torch.bfloat16, (T, self.d)), T, _ptr(logits), _ptr(ids),
                                  _ptr(gates), _stream()))
        return logits, ids, gates

    def route_logits(self, logits: torch.Tensor, stream=None):
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.route_logits(logits)
        T, dev = logits.shape[0], logits.device
        ids = torch.empty((T, self.k), dtype=torch.int32, device=dev)
        gates = torch.empty((T, self.k), dtype=torch.float32, device=dev)
        _check(self.lib.moe_route_logits(self._h, _dev(logits, "logits", torch.float32, (T, self.E)), T, ids.data_ptr(),
                                         gates.data_ptr(), _stream()))
        return ids, gates

    def permute(self, ids: torch.Tensor, stream=None):
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.permute(ids)
        T = ids.shape[0]
        dev = ids.device
        counts = torch.empty(self.E, dtype=torch.int32, device=dev)
        offsets = torch.empty(self.E + 1, dtype=torch.int32, device=dev)
        perm = torch.full((T * self.k,), -1, dtype=torch.int32, device=dev)
        inv = torch.empty(T * self.k, dtype=torch.int32, device=dev)
        _check(self.lib.moe_permute(self._h, _dev(ids, "ids", torch.int32, (T, self.k)), T, _ptr(counts), _ptr(offsets),
                                    _ptr(perm), _ptr(inv), _stream()))
        return counts, offsets, perm, inv

    def experts(self, x: torch.Tensor, offsets: torch.Tensor, perm: torch.Tensor, stream=None):
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.experts(x, offsets, perm)
        T = x.shape[0]
        y = torch.empty((T * self.k, self.d), dtype=torch.float16, device=x.device)
        ys = torch.empty((T, self.d), dtype=torch.float16, device=x.device) if self.n_shared else None
        _check(self.lib.moe_experts(self._h, _dev(x, "x", torch.bfloat16, (T, self.d)), T,
                                    _dev(offsets, "offsets", torch.int32, (self.E + 1,)),
                                    _dev(perm, "perm", torch.int32, (T * self.k,)), _ptr(y), _ptr(ys), _stream()))
        return y, ys

    def combine(self, y: torch.Tensor, gates: torch.Tensor, inv: torch.Tensor, shared_y: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, stream=None):
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.combine(y, gates, inv, shared_y, out)
        T = gates.shape[0]
        if out is None:
            out = torch.empty((T, self.d), dtype=torch.bfloat16, device=y.device)
        _check(self.lib.moe_combine(self._h, _dev(y, "y", torch.float32, (T * self.k, self.d)),
                                    _dev(gates, "gates", torch.float32, (T, self.k)),
                                    _dev(inv, "inv", torch.int32, (T * self.k,)),
                                    _dev(shared_y, "shared_y", torch.float32, (T, self.d)), T,
                                    _dev(out, "out", torch.bfloat16, (T, self.d)), _stream()))
        return out

    # ---- diagnostics ----------------------------------------------------------------------------
    def device_error(self) -> int:
        code = ctypes.c_uint32(0)
        st = self.lib.moe_plan_get_device_error(self._h, ctypes.byref(code))
        if st not in (MOE_OK, MOE_ERR_DEVICE):
            _check(st)
        return int(code.value)

    def enable_timing(self, on: bool = True):
        _check(self.lib.moe_plan_enable_timing(self._h, 1 if on else 0))

    def timing_report(self) -> dict:
        """{kernel name: (launches, total ms)} since the last report; synchronises."""
        buf = ctypes.create_string_buffer(1 << 16)
        self.lib.moe_plan_timing_report(self._h, buf, len(buf))
        rep = {}
        for line in buf.value.decode().splitlines():
            name, n, ms = line.split()
            rep[name] = (int(n), float(ms))
        return rep

    def resolved_path(self) -> tuple:
        """('tc' or 'simt', reason): the kernels the expert FFN runs on for this plan."""
        code = int(self.lib.moe_plan_resolved_path(self._h))
        name = {v: k for k, v in PATHS.items()}.get(code, "?")
        return name, ("" if name == "tc" else self.lib.moe_last_error().decode())

    def last_launch_count(self) -> int:
        return int(self.lib.moe_plan_last_launch_count(self._h))
