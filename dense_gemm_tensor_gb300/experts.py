"""The operators around a mixture-of-experts block, over the C interface of
``include/dgt_experts.h``: ``rms_norm``, ``route``, ``expert_matmul``,
``combine`` and their gradients.

As in ``gemm``, the functions take torch CUDA tensors, derive sizes and
strides from them, allocate their outputs and marshal the arguments; every
step of the arithmetic runs in the library's CUDA kernels, on ``stream`` or the
device's current stream. Rows may be padded (stride(0) > row length);
elements along a row are contiguous. Outputs and scratch are allocated for the
stream the call runs on.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import gemm
from .gemm import GEMM_B_K_MAJOR, GEMM_B_ROW_MAJOR, GEMM_OK, GemmError

GEMM_TYPE_F16, GEMM_TYPE_BF16, GEMM_TYPE_F32, GEMM_TYPE_E4M3 = 0, 1, 2, 3
GEMM_SCORE_SOFTMAX, GEMM_SCORE_SIGMOID = 0, 1
GEMM_ACT_SILU_GATED = 4

# Every symbol the C header declares.
EXPORTS = ("gemm_rmsnorm", "gemm_rmsnorm_backward", "gemm_rmsnorm_backward_workspace", "gemm_route",
           "gemm_route_workspace", "gemm_route_backward", "gemm_f16_grouped", "gemm_bf16_grouped",
           "gemm_e4m3_grouped", "gemm_grouped_workspace", "gemm_f16_grouped_wgrad", "gemm_bf16_grouped_wgrad",
           "gemm_grouped_wgrad_workspace", "gemm_combine", "gemm_combine_backward")

ACTIVATIONS = {**gemm.ACTIVATIONS, "silu_gated": GEMM_ACT_SILU_GATED}
SCORES = {"softmax": GEMM_SCORE_SOFTMAX, "sigmoid": GEMM_SCORE_SIGMOID}

_TYPE = {torch.float16: GEMM_TYPE_F16, torch.bfloat16: GEMM_TYPE_BF16, torch.float32: GEMM_TYPE_F32}
_E4M3 = torch.float8_e4m3fn
_GROUPED_TYPE = {torch.float16: GEMM_TYPE_F16, torch.bfloat16: GEMM_TYPE_BF16, _E4M3: GEMM_TYPE_E4M3}
_GROUPED = {torch.float16: "gemm_f16_grouped", torch.bfloat16: "gemm_bf16_grouped", _E4M3: "gemm_e4m3_grouped"}


class RouteConfig(ctypes.Structure):
    """gemm_route_config_t."""
    _fields_ = [("k", ctypes.c_int), ("score", ctypes.c_int), ("groups", ctypes.c_int), ("kept_groups", ctypes.c_int),
                ("renormalize", ctypes.c_int), ("scale", ctypes.c_float)]


class GroupedEpilogue(ctypes.Structure):
    """gemm_grouped_epilogue_t."""
    _fields_ = [("alpha", ctypes.c_float), ("row_scale", ctypes.c_void_p), ("col_scale", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("activation", ctypes.c_int)]


class Norm(NamedTuple):
    """``rms_norm``'s outputs; ``scale`` is None unless y is float8_e4m3fn."""
    y: torch.Tensor
    h: torch.Tensor
    rstd: torch.Tensor
    scale: torch.Tensor | None


class Routing(NamedTuple):
    """``route``'s outputs: T x k ids (-1: none), weights and slots (-1: none);
    the token of each of the T * k slots (-1 past the last one in use); the
    experts' first slots (experts + 1)."""
    ids: torch.Tensor
    weights: torch.Tensor
    slots: torch.Tensor
    rows: torch.Tensor
    offsets: torch.Tensor


_lib = None
_C = {}  # entry point -> bound C function, filled on first use


def _load():
    """The library, with this header's signatures declared (once)."""
    global _lib
    if _lib is not None:
        return _lib
    lib = gemm.load()
    i, i64, vp, f = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float
    cfg, epi = ctypes.POINTER(RouteConfig), ctypes.POINTER(GroupedEpilogue)
    sig = {
        "gemm_rmsnorm": [i, i64, i64, vp, i64, vp, i64, vp, f, vp, i64, i, vp, i64, vp, vp, vp],
        "gemm_rmsnorm_backward": [i, i64, i64, vp, i64, vp, i64, vp, vp, vp, i64, vp, i64, vp, vp, i64, vp],
        "gemm_route": [i, i64, i, vp, i64, vp, cfg, vp, vp, vp, vp, vp, vp, i64, vp],
        "gemm_route_backward": [i, i64, i, vp, i64, vp, vp, cfg, vp, i64, vp],
        "gemm_combine": [i, i64, i64, i, vp, i64, i64, vp, vp, vp, i64, vp, i64, vp],
        "gemm_combine_backward": [i, i64, i64, i, vp, i64, vp, i64, i64, vp, vp, vp, vp, i64, vp, vp],
    }
    for name in _GROUPED.values():
        sig[name] = [i, vp, i64, i64, i64, vp, i64, i64, vp, vp, i64, i64, vp, i64, i, epi, vp, i64, vp]
    for name in ("gemm_f16_grouped_wgrad", "gemm_bf16_grouped_wgrad"):
        sig[name] = [i, vp, i64, i64, i64, vp, i64, i64, vp, vp, i64, vp, i64, i64, i, vp, i64, vp]
    sizes = {"gemm_rmsnorm_backward_workspace": [i64, i64], "gemm_route_workspace": [i64, i, i],
             "gemm_grouped_workspace": [i, i, i64, i64], "gemm_grouped_wgrad_workspace": [i, i64, i64, i64, i]}
    for name, args in {**sig, **sizes}.items():
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, i64 if name in sizes else i
        _C[name] = fn
    _lib = lib
    return lib


def _call(name: str, *args) -> None:
    """Calls one entry point; raises what it refuses."""
    fn = _C.get(name)
    if fn is None:
        _load()
        fn = _C[name]
    code = fn(*args)
    if code != GEMM_OK:
        raise GemmError(code, name)


def _size(name: str, *args) -> int:
    if not _C:
        _load()
    return _C[name](*args)


def _under(stream, fn, *args, **kw):
    """fn under ``stream``, so that the caching allocator ties what it
    allocates to the stream that uses it."""
    with torch.cuda.stream(stream):
        return fn(*args, **kw)


def _stream(t: torch.Tensor) -> int:
    return gemm._raw_stream(None, t.device.index)


def _matrix(t: torch.Tensor, what: str, dtype=None, shape=None) -> int:
    """Checks a 2-D CUDA tensor with contiguous rows; its leading dimension."""
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}")
    size = t.shape
    if len(size) != 2 or not t.is_cuda:
        raise ValueError(f"{what} must be a 2-D CUDA tensor")
    rows, cols = size
    if shape is not None and size != shape:
        raise ValueError(f"{what} must be {shape[0]} x {shape[1]}")
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        raise ValueError(f"{what} must have unit stride along its rows")
    if rows <= 1:
        return cols
    if s0 < cols:
        raise ValueError(f"{what} must not have rows that overlap")
    return s0


def _vector(t: torch.Tensor, what: str, dtype, n: int):
    """Checks a contiguous CUDA tensor of n elements; its address (None if it has none)."""
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}")
    if t.numel() != n or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous CUDA tensor of {n} elements")
    return t.data_ptr() or None


def _type(t: torch.Tensor, what: str) -> int:
    code = _TYPE.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} must be float16, bfloat16 or float32")
    return code


# ---------------------------------------------------------------- norm

def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, *, eps: float = 1e-6,
             out_dtype: torch.dtype | None = None, h_out: torch.Tensor | None = None,
             stream: torch.cuda.Stream | None = None) -> Norm:
    """h = x + residual (rounded to x's dtype), y = h * rsqrt(mean(h^2) + eps) * weight.

    ``x``, ``residual``: rows x cols; ``weight``: cols, all of one dtype
    (float16, bfloat16 or float32). ``out_dtype`` None or that dtype, or
    float8_e4m3fn: y then holds 8-bit rows and ``scale`` their scales (y * scale
    stands for the norm). ``h_out`` receives h (it may be ``x`` or
    ``residual``); without a residual h is x. ``rstd``: fp32, for the backward pass."""
    if stream is not None:
        return _under(stream, rms_norm, x, weight, residual, eps=eps, out_dtype=out_dtype, h_out=h_out)
    dt = x.dtype
    code = _TYPE.get(dt)
    if code is None:
        raise TypeError("x must be float16, bfloat16 or float32")
    ldx = _matrix(x, "x")
    rows, cols = x.shape
    q8 = out_dtype is _E4M3
    if not q8 and out_dtype is not None and out_dtype is not dt:
        raise TypeError("out_dtype must be x's dtype or float8_e4m3fn")
    w = _vector(weight, "weight", dt, cols)
    dev = x.device
    y = torch.empty((rows, cols), dtype=out_dtype or dt, device=dev)
    rstd = torch.empty((rows,), dtype=torch.float32, device=dev)
    scale = torch.empty((rows,), dtype=torch.float32, device=dev) if q8 else None
    h, ph, pr, ldh, ldr = x, None, None, 0, 0
    if residual is not None:
        ldr, pr = _matrix(residual, "residual", dt, x.shape), residual.data_ptr()
        if h_out is None:
            h, ldh = torch.empty((rows, cols), dtype=dt, device=dev), cols
        else:
            h, ldh = h_out, _matrix(h_out, "h_out", dt, x.shape)
        ph = h.data_ptr()
    _call("gemm_rmsnorm", code, rows, cols, x.data_ptr(), ldx, pr, ldr, w, eps, ph, ldh, GEMM_TYPE_E4M3 if q8 else code,
          y.data_ptr(), cols, scale.data_ptr() if q8 else None, rstd.data_ptr(), gemm._raw_stream(None, dev.index))
    return Norm(y, h, rstd, scale)


def rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor, *,
                      dh: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None):
    """(dx, dweight) of ``rms_norm``: dx is the gradient of x and of the
    residual alike; ``dh`` is the gradient that reaches h by the residual path."""
    if stream is not None:
        return _under(stream, rms_norm_backward, dy, h, weight, rstd, dh=dh)
    dt = h.dtype
    code = _type(h, "h")
    ldh = _matrix(h, "h")
    rows, cols = h.shape
    lddy = _matrix(dy, "dy", dt, h.shape)
    lddh = _matrix(dh, "dh", dt, h.shape) if dh is not None else 0
    w, r = _vector(weight, "weight", dt, cols), _vector(rstd, "rstd", torch.float32, rows)
    need = _size("gemm_rmsnorm_backward_workspace", rows, cols)
    dev = h.device
    dx = torch.empty((rows, cols), dtype=dt, device=dev)
    dw = torch.empty((cols,), dtype=dt, device=dev)
    ws = torch.empty((need,), dtype=torch.uint8, device=dev)
    _call("gemm_rmsnorm_backward", code, rows, cols, dy.data_ptr(), lddy, h.data_ptr(), ldh, w, r,
          dh.data_ptr() if dh is not None else None, lddh, dx.data_ptr(), cols, dw.data_ptr(), ws.data_ptr(), need,
          _stream(h))
    return dx, dw


# ---------------------------------------------------------------- router

def _config(k, score, groups, kept_groups, renormalize, scale) -> RouteConfig:
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}")
    return RouteConfig(int(k), SCORES[score], int(groups), int(kept_groups), int(bool(renormalize)), float(scale))


def route(logits: torch.Tensor, k: int, *, score: str = "softmax", bias: torch.Tensor | None = None, groups: int = 1,
          kept_groups: int = 1, renormalize: bool = True, scale: float = 1.0,
          stream: torch.cuda.Stream | None = None) -> Routing:
    """Chooses each token's k experts from its row of ``logits`` (T x experts,
    float16, bfloat16 or float32) and orders the pairs by expert.

    Experts are ranked by score + ``bias`` (experts floats; it moves the choice
    only), within the ``kept_groups`` best of ``groups`` equal runs of experts;
    the weights are the chosen scores, renormalised to sum to 1 and times
    ``scale``. Ties go to the lowest expert; a logit of -inf takes its expert
    out (see the C header for the exact rules)."""
    if stream is not None:
        return _under(stream, route, logits, k, score=score, bias=bias, groups=groups, kept_groups=kept_groups,
                      renormalize=renormalize, scale=scale)
    code = _type(logits, "logits")
    ld = _matrix(logits, "logits")
    tokens, experts = logits.shape
    cfg = _config(k, score, groups, kept_groups, renormalize, scale)
    b = _vector(bias, "bias", torch.float32, experts) if bias is not None else None
    need = _size("gemm_route_workspace", tokens, experts, cfg.k)
    k = max(cfg.k, 0)
    dev, i32 = logits.device, torch.int32
    ids = torch.empty((tokens, k), dtype=i32, device=dev)
    weights = torch.empty((tokens, k), dtype=torch.float32, device=dev)
    slots = torch.empty((tokens, k), dtype=i32, device=dev)
    rows = torch.empty((tokens * k,), dtype=i32, device=dev)
    offsets = torch.empty((experts + 1,), dtype=i32, device=dev)
    ws = torch.empty((need,), dtype=torch.uint8, device=dev) if need else None
    _call("gemm_route", code, tokens, experts, logits.data_ptr(), ld, b, cfg, ids.data_ptr(), weights.data_ptr(),
          slots.data_ptr(), rows.data_ptr(), offsets.data_ptr(), ws.data_ptr() if need else None, need, _stream(logits))
    return Routing(ids, weights, slots, rows, offsets)


def route_backward(dweights: torch.Tensor, logits: torch.Tensor, ids: torch.Tensor, *, score: str = "softmax",
                   renormalize: bool = True, scale: float = 1.0,
                   stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """dlogits (in the logits' dtype) from the weights' gradient, the logits and
    the ids that ``route`` chose; the choice itself is held fixed."""
    if stream is not None:
        return _under(stream, route_backward, dweights, logits, ids, score=score, renormalize=renormalize, scale=scale)
    code = _type(logits, "logits")
    ld = _matrix(logits, "logits")
    tokens, experts = logits.shape
    if ids.dim() != 2 or ids.shape[0] != tokens:
        raise ValueError("ids must be T x k")
    k = ids.shape[1]
    cfg = _config(k, score, 1, 1, renormalize, scale)
    i, d = _vector(ids, "ids", torch.int32, tokens * k), _vector(dweights, "dweights", torch.float32, tokens * k)
    out = torch.empty((tokens, experts), dtype=logits.dtype, device=logits.device)
    _call("gemm_route_backward", code, tokens, experts, logits.data_ptr(), ld, i, d, cfg, out.data_ptr(), experts,
          _stream(logits))
    return out


# ---------------------------------------------------------------- experts

def _stack(t: torch.Tensor, what: str):
    """Checks a groups x rows x cols CUDA tensor with contiguous rows; its leading dimension and matrix stride."""
    if t.dim() != 3 or not t.is_cuda:
        raise ValueError(f"{what} must be a 3-D CUDA tensor")
    g, r, c = t.shape
    s0, s1, s2 = t.stride()
    if c > 1 and s2 != 1:
        raise ValueError(f"{what} must have unit stride along its rows")
    ld = s1 if r > 1 else c
    return ld, s0 if g > 1 else r * ld


def expert_matmul(A: torch.Tensor, W: torch.Tensor, offsets: torch.Tensor, rows: torch.Tensor | None = None, *,
                  layout: int = GEMM_B_ROW_MAJOR, out: torch.Tensor | None = None, alpha: float = 1.0,
                  a_scale: torch.Tensor | None = None, w_scale: torch.Tensor | None = None,
                  bias: torch.Tensor | None = None, activation: str | None = None,
                  stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Each expert's rows times its matrix: C[s] = act(alpha * a_scale[row(s)] *
    w_scale[e] * (A[row(s)] . W[e]) + bias[e]) for s in [offsets[e], offsets[e+1]).

    ``A``: rows x K; ``rows`` (int32, one per slot) says which row of A a slot
    takes -- ``Routing.rows``, so that A is the tokens' own matrix -- and None
    that slot s takes row s. ``W``: experts x K x N for
    ``layout=GEMM_B_ROW_MAJOR``, experts x N x K for ``GEMM_B_K_MAJOR`` (the
    only one for float8_e4m3fn). float16 and bfloat16 give their own dtype,
    float8_e4m3fn bfloat16. ``a_scale``: one float per row of A; ``w_scale``:
    experts x N floats; ``bias``: experts x N of C's dtype; ``activation``: as
    ``gemm.matmul``'s, or "silu_gated" (W holds gate and value halves, C has
    N / 2 columns). Rows of C past offsets[-1] are zero. With the other layout
    flag the call is the gradient of A (a row per slot)."""
    if stream is not None:
        return _under(stream, expert_matmul, A, W, offsets, rows, layout=layout, out=out, alpha=alpha, a_scale=a_scale,
                      w_scale=w_scale, bias=bias, activation=activation)
    dt = A.dtype
    name = _GROUPED.get(dt)
    if name is None:
        raise TypeError("A must be float16, bfloat16 or float8_e4m3fn")
    if W.dtype is not dt:
        raise TypeError("A and W must have the same dtype")
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(a for a in ACTIVATIONS if a)}")
    lda = _matrix(A, "A")
    ldw, stride_w = _stack(W, "W")
    experts, W1, W2 = W.shape
    a_rows, K = A.shape
    N, WK = (W1, W2) if layout == GEMM_B_K_MAJOR else (W2, W1)
    if WK != K:
        raise ValueError("W's K dimension does not match A")
    out_dt = torch.bfloat16 if dt is _E4M3 else dt
    off = _vector(offsets, "offsets", torch.int32, experts + 1)
    dev = A.device
    if rows is None:
        slots, r, need = a_rows, None, 0
    else:
        slots = rows.numel()
        r = _vector(rows, "rows", torch.int32, slots)
        need = _size("gemm_grouped_workspace", _GROUPED_TYPE[dt], experts, slots, K)
    cols = N // 2 if act == GEMM_ACT_SILU_GATED else N
    if out is None:
        out, ldc = torch.empty((slots, cols), dtype=out_dt, device=dev), cols
    else:
        ldc = _matrix(out, "out", out_dt, (slots, cols))
    ws = torch.empty((need,), dtype=torch.uint8, device=dev) if need else None
    epi = None
    if act or alpha != 1.0 or a_scale is not None or w_scale is not None or bias is not None:
        epi = GroupedEpilogue(
            alpha, _vector(a_scale, "a_scale", torch.float32, a_rows) if a_scale is not None else None,
            _vector(w_scale, "w_scale", torch.float32, experts * N) if w_scale is not None else None,
            _vector(bias, "bias", out_dt, experts * N) if bias is not None else None, act)
    _call(name, experts, off, slots, N, K, A.data_ptr() or None, a_rows, lda, r, W.data_ptr() or None, ldw, stride_w,
          out.data_ptr(), ldc, layout, epi, ws.data_ptr() if need else None, need, gemm._raw_stream(None, dev.index))
    return out


def expert_weight_grad(A: torch.Tensor, dC: torch.Tensor, offsets: torch.Tensor, rows: torch.Tensor | None = None, *,
                       layout: int = GEMM_B_ROW_MAJOR, out: torch.Tensor | None = None,
                       stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The gradient of ``expert_matmul``'s W (of its plain product) from
    ``dC`` (slots x N): experts x K x N for ``layout=GEMM_B_ROW_MAJOR``,
    experts x N x K for ``GEMM_B_K_MAJOR``; zeros for an expert without slots."""
    if stream is not None:
        return _under(stream, expert_weight_grad, A, dC, offsets, rows, layout=layout, out=out)
    dt = A.dtype
    if dt not in (torch.float16, torch.bfloat16):
        raise TypeError("A must be float16 or bfloat16")
    lda = _matrix(A, "A")
    a_rows, K = A.shape
    slots = a_rows if rows is None else rows.numel()
    if dC.dim() != 2 or dC.shape[0] != slots:
        raise ValueError("dC must have one row per slot")
    lddc = _matrix(dC, "dC", dt)
    N = dC.shape[1]
    experts = offsets.numel() - 1
    off = _vector(offsets, "offsets", torch.int32, experts + 1)
    r = _vector(rows, "rows", torch.int32, slots) if rows is not None else None
    shape = (experts, N, K) if layout == GEMM_B_K_MAJOR else (experts, K, N)
    if out is None:
        out = torch.empty(shape, dtype=dt, device=A.device)
    elif out.dtype is not dt or tuple(out.shape) != shape:
        raise ValueError(f"out must be {shape[0]} x {shape[1]} x {shape[2]} of A's dtype")
    need = _size("gemm_grouped_wgrad_workspace", experts, slots, N, K, int(rows is not None))
    ws = torch.empty((need,), dtype=torch.uint8, device=A.device) if need else None
    ldw, stride_w = _stack(out, "out")
    _call("gemm_f16_grouped_wgrad" if dt is torch.float16 else "gemm_bf16_grouped_wgrad", experts, off, slots, N, K,
          A.data_ptr() or None, a_rows, lda, r, dC.data_ptr() or None, lddc, out.data_ptr() or None, ldw, stride_w,
          layout, ws.data_ptr() if need else None, need, _stream(A))
    return out


# ---------------------------------------------------------------- combine

def combine(z: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor | None = None, *,
            residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
            stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """y[t] = residual[t] + sum_j weights[t][j] * z[slots[t][j]] (slots of -1
    add nothing; weights None: all 1). ``out`` may be ``residual``."""
    if stream is not None:
        return _under(stream, combine, z, slots, weights, residual=residual, out=out)
    dt = z.dtype
    code = _type(z, "z")
    ldz = _matrix(z, "z")
    if slots.dim() != 2:
        raise ValueError("slots must be T x k")
    tokens, k = slots.shape
    nslots, cols = z.shape
    i = _vector(slots, "slots", torch.int32, tokens * k)
    w = _vector(weights, "weights", torch.float32, tokens * k) if weights is not None else None
    ldr = _matrix(residual, "residual", dt, (tokens, cols)) if residual is not None else 0
    if out is None:
        out, ldy = torch.empty((tokens, cols), dtype=dt, device=z.device), cols
    else:
        ldy = _matrix(out, "out", dt, (tokens, cols))
    _call("gemm_combine", code, tokens, cols, k, z.data_ptr(), ldz, nslots, i, w,
          residual.data_ptr() if residual is not None else None, ldr, out.data_ptr(), ldy, _stream(z))
    return out


def combine_backward(dy: torch.Tensor, z: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor | None = None,
                     offsets: torch.Tensor | None = None, *, stream: torch.cuda.Stream | None = None):
    """(dz, dweights) of ``combine``. ``offsets`` (``Routing.offsets``): rows of
    dz past offsets[-1] are set to zero; without it every row of z must belong
    to a slot. dweights is None where weights is."""
    if stream is not None:
        return _under(stream, combine_backward, dy, z, slots, weights, offsets)
    dt = z.dtype
    code = _type(z, "z")
    ldz = _matrix(z, "z")
    if slots.dim() != 2:
        raise ValueError("slots must be T x k")
    tokens, k = slots.shape
    nslots, cols = z.shape
    lddy = _matrix(dy, "dy", dt, (tokens, cols))
    i = _vector(slots, "slots", torch.int32, tokens * k)
    w = _vector(weights, "weights", torch.float32, tokens * k) if weights is not None else None
    used = None
    if offsets is not None:
        n = offsets.numel()
        used = _vector(offsets, "offsets", torch.int32, n) + 4 * (n - 1)
    dz = torch.empty((nslots, cols), dtype=dt, device=z.device)
    dw = torch.empty((tokens, k), dtype=torch.float32, device=z.device) if weights is not None else None
    _call("gemm_combine_backward", code, tokens, cols, k, dy.data_ptr(), lddy, z.data_ptr(), ldz, nslots, i, w, used,
          dz.data_ptr(), cols, dw.data_ptr() if dw is not None else None, _stream(z))
    return dz, dw
