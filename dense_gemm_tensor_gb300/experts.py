"""The operators around a mixture-of-experts block, over the C interface of
``include/dgt_experts.h``: ``rms_norm``, ``route``, ``expert_matmul``,
``combine`` and their gradients.

As in ``gemm``, the functions take torch CUDA tensors, derive sizes and
strides from them, allocate their outputs and pass the arguments on; every
step of the arithmetic runs in the library's CUDA kernels, on ``stream`` or the
device's current stream. The checks and allocations are in the compiled module
``_experts`` (``csrc/experts_binding.cpp``). Rows may be padded (stride(0) > row
length); elements along a row are contiguous. Outputs and scratch are allocated
for the stream the call runs on.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import gemm
from .gemm import GEMM_B_ROW_MAJOR, GemmError

GEMM_SCORE_SOFTMAX, GEMM_SCORE_SIGMOID = 0, 1
GEMM_ACT_SILU_GATED = 4

# Every symbol the C header declares.
EXPORTS = ("gemm_rmsnorm", "gemm_rmsnorm_backward", "gemm_rmsnorm_backward_workspace", "gemm_route",
           "gemm_route_workspace", "gemm_route_backward", "gemm_f16_grouped", "gemm_bf16_grouped",
           "gemm_e4m3_grouped", "gemm_grouped_workspace", "gemm_f16_grouped_wgrad", "gemm_bf16_grouped_wgrad",
           "gemm_grouped_wgrad_workspace", "gemm_grouped_rows_workspace", "gemm_grouped_weights_workspace",
           "gemm_grouped_wgrad_rows_workspace", "gemm_combine", "gemm_combine_backward")

ACTIVATIONS = {**gemm.ACTIVATIONS, "silu_gated": GEMM_ACT_SILU_GATED}
SCORES = {"softmax": GEMM_SCORE_SOFTMAX, "sigmoid": GEMM_SCORE_SIGMOID}

_E4M3 = torch.float8_e4m3fn


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
_ext = None


def _load():
    """The library, with this header's signatures declared (once): the C calls with raw pointers."""
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
    for name in ("gemm_f16_grouped", "gemm_bf16_grouped", "gemm_e4m3_grouped"):
        sig[name] = [i, vp, i64, i64, i64, vp, i64, i64, vp, vp, i64, i64, vp, i64, i, epi, vp, i64, vp]
    for name in ("gemm_f16_grouped_wgrad", "gemm_bf16_grouped_wgrad"):
        sig[name] = [i, vp, i64, i64, i64, vp, i64, i64, vp, vp, i64, vp, i64, i64, i, vp, i64, vp]
    sizes = {"gemm_rmsnorm_backward_workspace": [i64, i64], "gemm_route_workspace": [i64, i, i],
             "gemm_grouped_workspace": [i, i, i64, i64], "gemm_grouped_wgrad_workspace": [i, i64, i64, i64, i],
             "gemm_grouped_rows_workspace": [i, i, i64, i64, i64, i64, i],
             "gemm_grouped_weights_workspace": [i, i, i64, i64, i64, i64, i, i],
             "gemm_grouped_wgrad_rows_workspace": [i, i64, i64, i64, i64, i64, i, i64]}
    for name, args in {**sig, **sizes}.items():
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, i64 if name in sizes else i
    _lib = lib
    return lib


def _binding():
    """The compiled binding, given the loaded library's entry points (once)."""
    global _ext
    if _ext is None:
        lib = _load()
        try:
            from . import _experts
        except ImportError as e:
            raise RuntimeError(f"the compiled binding _experts.so cannot be loaded ({e}): build it with "
                               "dense_gemm_tensor_gb300.build.build()") from e
        _experts.bind({name: ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in EXPORTS})
        _ext = _experts
    return _ext


def _under(stream, fn, *args, **kw):
    """fn under ``stream``, so that the caching allocator ties what it
    allocates to the stream that uses it."""
    with torch.cuda.stream(stream):
        return fn(*args, **kw)


def _refuse(code: int, name: str):
    raise GemmError(code, name)


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
    q8 = out_dtype is _E4M3
    if not q8 and out_dtype is not None and out_dtype is not x.dtype:
        raise TypeError("out_dtype must be x's dtype or float8_e4m3fn")
    r = (_ext or _binding()).rms_norm(x, weight, residual, eps, q8, h_out)
    if r.__class__ is int:
        _refuse(r, "gemm_rmsnorm")
    return Norm._make(r)


def rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor, *,
                      dh: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None):
    """(dx, dweight) of ``rms_norm``: dx is the gradient of x and of the
    residual alike; ``dh`` is the gradient that reaches h by the residual path."""
    if stream is not None:
        return _under(stream, rms_norm_backward, dy, h, weight, rstd, dh=dh)
    r = (_ext or _binding()).rms_norm_backward(dy, h, weight, rstd, dh)
    if r.__class__ is int:
        _refuse(r, "gemm_rmsnorm_backward")
    return r


# ---------------------------------------------------------------- router

def _score(score: str) -> int:
    code = SCORES.get(score)
    if code is None:
        raise ValueError(f"score must be one of {sorted(SCORES)}")
    return code


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
    r = (_ext or _binding()).route(logits, k, _score(score), bias, groups, kept_groups, renormalize, scale)
    if r.__class__ is int:
        _refuse(r, "gemm_route")
    return Routing._make(r)


def route_backward(dweights: torch.Tensor, logits: torch.Tensor, ids: torch.Tensor, *, score: str = "softmax",
                   renormalize: bool = True, scale: float = 1.0,
                   stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """dlogits (in the logits' dtype) from the weights' gradient, the logits and
    the ids that ``route`` chose; the choice itself is held fixed."""
    if stream is not None:
        return _under(stream, route_backward, dweights, logits, ids, score=score, renormalize=renormalize, scale=scale)
    r = (_ext or _binding()).route_backward(dweights, logits, ids, _score(score), renormalize, scale)
    if r.__class__ is int:
        _refuse(r, "gemm_route_backward")
    return r[0]


# ---------------------------------------------------------------- experts

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
    flag the call is the gradient of A (a row per slot).

    A and W start on 16-byte boundaries. Rows may have any pitch, but only those
    (and matrices of W, and the value half of row-major gated weights) that are
    16-byte multiples apart are read where they are: others are copied first, in
    every call, so keep weights of an odd width in a padded buffer."""
    if stream is not None:
        return _under(stream, expert_matmul, A, W, offsets, rows, layout=layout, out=out, alpha=alpha, a_scale=a_scale,
                      w_scale=w_scale, bias=bias, activation=activation)
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(a for a in ACTIVATIONS if a)}")
    r = (_ext or _binding()).expert_matmul(A, W, offsets, rows, layout, out, alpha, a_scale, w_scale, bias, act)
    if r.__class__ is int:
        _refuse(r, "gemm_grouped")
    return r[0]


def expert_weight_grad(A: torch.Tensor, dC: torch.Tensor, offsets: torch.Tensor, rows: torch.Tensor | None = None, *,
                       layout: int = GEMM_B_ROW_MAJOR, out: torch.Tensor | None = None,
                       stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The gradient of ``expert_matmul``'s W (of its plain product) from
    ``dC`` (slots x N): experts x K x N for ``layout=GEMM_B_ROW_MAJOR``,
    experts x N x K for ``GEMM_B_K_MAJOR``; zeros for an expert without slots.
    A and dC start on 16-byte boundaries; rows that are not 16-byte multiples
    apart are copied first."""
    if stream is not None:
        return _under(stream, expert_weight_grad, A, dC, offsets, rows, layout=layout, out=out)
    r = (_ext or _binding()).expert_weight_grad(A, dC, offsets, rows, layout, out)
    if r.__class__ is int:
        _refuse(r, "gemm_grouped_wgrad")
    return r[0]


# ---------------------------------------------------------------- combine

def combine(z: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor | None = None, *,
            residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
            stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """y[t] = residual[t] + sum_j weights[t][j] * z[slots[t][j]] (slots of -1
    add nothing; weights None: all 1). ``out`` may be ``residual``."""
    if stream is not None:
        return _under(stream, combine, z, slots, weights, residual=residual, out=out)
    r = (_ext or _binding()).combine(z, slots, weights, residual, out)
    if r.__class__ is int:
        _refuse(r, "gemm_combine")
    return r[0]


def combine_backward(dy: torch.Tensor, z: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor | None = None,
                     offsets: torch.Tensor | None = None, *, stream: torch.cuda.Stream | None = None):
    """(dz, dweights) of ``combine``. ``offsets`` (``Routing.offsets``): rows of
    dz past offsets[-1] are set to zero; without it every row of z must belong
    to a slot. dweights is None where weights is."""
    if stream is not None:
        return _under(stream, combine_backward, dy, z, slots, weights, offsets)
    r = (_ext or _binding()).combine_backward(dy, z, slots, weights, offsets)
    if r.__class__ is int:
        _refuse(r, "gemm_combine_backward")
    return r
