"""The operators of a dense feed-forward block, over the C interface of
``include/dgt_feedforward.h``: ``layer_norm`` and ``gated_matmul`` with their
gradients, and products of 8-bit matrices with a scale for each block of 128
(``quantize_blocks``, ``matmul_blocks``).

As in ``experts``, the functions take torch CUDA tensors on the current device,
derive sizes and strides from them, allocate their outputs and pass the
arguments on; every step of the arithmetic runs in the library's CUDA kernels,
on ``stream`` or the device's current stream. The checks and allocations are in
the compiled module ``_feedforward`` (``csrc/feedforward_binding.cpp``). Rows may
be padded (stride(0) > row length); elements along a row are contiguous. Outputs
and scratch are allocated for the stream the call runs on.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import gemm
from .experts import _refuse, _under
from .gemm import GEMM_B_ROW_MAJOR

GEMM_GATE_SILU, GEMM_GATE_GELU, GEMM_GATE_GELU_TANH, GEMM_GATE_RELU = 0, 1, 2, 3
BLOCK = 128

# Every symbol the C header declares.
EXPORTS = ("gemm_layernorm", "gemm_layernorm_backward", "gemm_layernorm_backward_workspace", "gemm_gated",
           "gemm_gated_workspace", "gemm_gated_backward", "gemm_gated_backward_workspace", "gemm_e4m3_blocks",
           "gemm_quantize_blocks")

GATES = {"silu": GEMM_GATE_SILU, "gelu": GEMM_GATE_GELU, "gelu_tanh": GEMM_GATE_GELU_TANH, "relu": GEMM_GATE_RELU}

_E4M3 = torch.float8_e4m3fn


class LayerNorm(NamedTuple):
    """``layer_norm``'s outputs; ``scale`` is None unless y is float8_e4m3fn."""
    y: torch.Tensor
    h: torch.Tensor
    mean: torch.Tensor
    rstd: torch.Tensor
    scale: torch.Tensor | None


class Gated(NamedTuple):
    """``gated_matmul``'s outputs; ``up`` (M x 2F) is None unless it is kept."""
    c: torch.Tensor
    up: torch.Tensor | None


class GatedGrads(NamedTuple):
    """``gated_matmul_backward``'s outputs; None for those not asked for."""
    dA: torch.Tensor | None
    dW: torch.Tensor | None
    dbias: torch.Tensor | None


class Blocks(NamedTuple):
    """An 8-bit matrix and the scales of its blocks."""
    q: torch.Tensor
    scale: torch.Tensor


_lib = None
_ext = None


def _load():
    """The library, with this header's signatures declared (once): the C calls with raw pointers."""
    global _lib
    if _lib is not None:
        return _lib
    lib = gemm.load()
    i, i64, vp, f = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float
    sig = {
        "gemm_layernorm": [i, i64, i64, vp, i64, vp, i64, vp, vp, f, vp, i64, i, vp, i64, vp, vp, vp, vp],
        "gemm_layernorm_backward": [i, i64, i64, vp, i64, vp, i64, vp, vp, vp, vp, i64, vp, i64, vp, vp, vp, i64, vp],
        "gemm_gated": [i, i64, i64, i64, vp, i64, vp, i64, i, i, vp, vp, i64, vp, i64, vp, i64, vp],
        "gemm_gated_backward": [i, i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, i, i, vp, i64, vp, i64, vp, vp,
                                i64, vp],
        "gemm_e4m3_blocks": [i64, i64, i64, vp, i64, vp, i64, i64, vp, i64, vp, i64, i64, i, vp, i64, vp],
        "gemm_quantize_blocks": [i, i64, i64, vp, i64, i, i, vp, i64, vp, i64, i64, vp],
    }
    sizes = {"gemm_layernorm_backward_workspace": [i64, i64], "gemm_gated_workspace": [i, i64, i64, i64, i64, i64, i],
             "gemm_gated_backward_workspace": [i, i64, i64, i64, i64, i64, i, i, i, i]}
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
            from . import _feedforward
        except ImportError as e:
            raise RuntimeError(f"the compiled binding _feedforward.so cannot be loaded ({e}): build it with "
                               "dense_gemm_tensor_gb300.build.build()") from e
        _feedforward.bind({name: ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in EXPORTS})
        _ext = _feedforward
    return _ext


def _gate(activation: str) -> int:
    code = GATES.get(activation)
    if code is None:
        raise ValueError(f"activation must be one of {sorted(GATES)}")
    return code


# ---------------------------------------------------------------- norm

def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
               residual: torch.Tensor | None = None, *, eps: float = 1e-5, out_dtype: torch.dtype | None = None,
               h_out: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None) -> LayerNorm:
    """h = x + residual (rounded to x's dtype), y = (h - mean(h)) * rsqrt(var(h) + eps) * weight + bias.

    ``x``, ``residual``: rows x cols; ``weight``, ``bias``: cols, all of one
    dtype (float16, bfloat16 or float32). ``out_dtype`` None or that dtype, or
    float8_e4m3fn: y then holds 8-bit rows and ``scale`` their scales (y * scale
    stands for the norm; ``scale[:, None].expand(-1, blocks)`` makes them an
    operand of ``matmul_blocks``). ``h_out`` receives h (it may be ``x`` or
    ``residual``); without a residual h is x. ``mean`` and ``rstd``: fp32, for
    the backward pass."""
    if stream is not None:
        return _under(stream, layer_norm, x, weight, bias, residual, eps=eps, out_dtype=out_dtype, h_out=h_out)
    q8 = out_dtype is _E4M3
    if not q8 and out_dtype is not None and out_dtype is not x.dtype:
        raise TypeError("out_dtype must be x's dtype or float8_e4m3fn")
    r = (_ext or _binding()).layer_norm(x, weight, bias, residual, eps, q8, h_out)
    if r.__class__ is int:
        _refuse(r, "gemm_layernorm")
    return LayerNorm._make(r)


def layer_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor,
                        rstd: torch.Tensor, *, dh: torch.Tensor | None = None,
                        stream: torch.cuda.Stream | None = None):
    """(dx, dweight, dbias) of ``layer_norm``: dx is the gradient of x and of
    the residual alike; ``dh`` is the gradient that reaches h by the residual path."""
    if stream is not None:
        return _under(stream, layer_norm_backward, dy, h, weight, mean, rstd, dh=dh)
    r = (_ext or _binding()).layer_norm_backward(dy, h, weight, mean, rstd, dh)
    if r.__class__ is int:
        _refuse(r, "gemm_layernorm_backward")
    return r


# ---------------------------------------------------------------- gated product

def gated_matmul(A: torch.Tensor, W: torch.Tensor, *, layout: int = GEMM_B_ROW_MAJOR, activation: str = "silu",
                 bias: torch.Tensor | None = None, keep: bool = False, out: torch.Tensor | None = None,
                 stream: torch.cuda.Stream | None = None) -> Gated:
    """C = act(gate) * value, where [gate | value] = A . W + bias, in one kernel.

    ``A``: M x K, float16 or bfloat16. ``W`` holds the gate's F columns, then
    the value's: K x 2F for ``layout=GEMM_B_ROW_MAJOR``, 2F x K for
    ``GEMM_B_K_MAJOR``. ``activation``: "silu", "gelu", "gelu_tanh" or "relu".
    ``bias``: 2F elements. ``keep`` returns [gate | value] too (M x 2F, rounded),
    which ``gated_matmul_backward`` takes.

    A and W start on 16-byte boundaries. Rows may have any pitch, but only those
    (and the value half of row-major weights) that are 16-byte multiples apart
    are read where they are: others are copied first, in every call."""
    if stream is not None:
        return _under(stream, gated_matmul, A, W, layout=layout, activation=activation, bias=bias, keep=keep, out=out)
    r = (_ext or _binding()).gated_matmul(A, W, layout, _gate(activation), bias, keep, out)
    if r.__class__ is int:
        _refuse(r, "gemm_gated")
    return Gated._make(r)


def gated_matmul_backward(dC: torch.Tensor, A: torch.Tensor, W: torch.Tensor, up: torch.Tensor, *,
                          layout: int = GEMM_B_ROW_MAJOR, activation: str = "silu", bias: bool = False,
                          rows: bool = True, weights: bool = True,
                          stream: torch.cuda.Stream | None = None) -> GatedGrads:
    """The gradients of ``gated_matmul`` from ``dC`` (M x F) and the ``up`` that
    it kept: dA unless ``rows`` is False, dW (W's shape) unless ``weights`` is
    False, and dbias where ``bias`` is True. The gradient of [gate | value] is
    rounded to the operands' dtype before the products."""
    if stream is not None:
        return _under(stream, gated_matmul_backward, dC, A, W, up, layout=layout, activation=activation, bias=bias,
                      rows=rows, weights=weights)
    r = (_ext or _binding()).gated_matmul_backward(dC, A, W, up, layout, _gate(activation), rows, weights, bias)
    if r.__class__ is int:
        _refuse(r, "gemm_gated_backward")
    return GatedGrads._make(r)


# ---------------------------------------------------------------- 8-bit blocks

def quantize_blocks(x: torch.Tensor, *, rows: int = 1, transpose: bool = False,
                    stream: torch.cuda.Stream | None = None) -> Blocks:
    """x (or x^T with ``transpose``) in float8_e4m3fn, with a scale for each
    block of ``rows`` (1 or 128) rows x 128 columns: q * scale stands for it.

    ``x``: float16, bfloat16 or float32. q's rows start on 16-byte boundaries, as
    ``matmul_blocks`` takes them. ``scale``: rows x blocks of a row for ``rows=1``
    (the blocks' columns contiguous), runs of 128 rows x blocks for ``rows=128``."""
    if stream is not None:
        return _under(stream, quantize_blocks, x, rows=rows, transpose=transpose)
    if rows not in (1, BLOCK):
        raise ValueError("rows must be 1 or 128")
    r = (_ext or _binding()).quantize_blocks(x, rows, transpose)
    if r.__class__ is int:
        _refuse(r, "gemm_quantize_blocks")
    return Blocks._make(r)


def matmul_blocks(A: torch.Tensor, B: torch.Tensor, a_scale: torch.Tensor, b_scale: torch.Tensor, *,
                  out: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """C = A . B^T with a scale for each block of 128 along K, in bfloat16.

    ``A``: M x K, ``B``: N x K, float8_e4m3fn, their rows on 16-byte boundaries.
    ``a_scale``: M x ceil(K / 128) floats. ``b_scale``: N x ceil(K / 128), or
    ceil(N / 128) x ceil(K / 128) for blocks of 128 x 128. Scales may have any
    strides (``expand`` repeats one). A product's gradients are this product too:
    dA of ``dC`` and ``B`` quantised along N, dB of ``dC`` and ``A`` along M
    (``quantize_blocks`` with ``transpose``)."""
    if stream is not None:
        return _under(stream, matmul_blocks, A, B, a_scale, b_scale, out=out)
    r = (_ext or _binding()).matmul_blocks(A, B, a_scale, b_scale, out)
    if r.__class__ is int:
        _refuse(r, "gemm_e4m3_blocks")
    return r[0]
