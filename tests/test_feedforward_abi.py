"""The feed-forward operators without a GPU: the oracle against differences and
worked examples, the C interface's exports, workspace sizes and refusals, and
the Python functions' refusals."""

import os
import re
import sys

import numpy as np
import pytest
import torch

import dense_gemm_tensor_gb300
from dense_gemm_tensor_gb300 import build, feedforward, gemm
from oracle import feedforward as of

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dgt_feedforward.h")
INVALID, MISALIGNED, OK = gemm.GEMM_ERR_INVALID_VALUE, gemm.GEMM_ERR_MISALIGNED, gemm.GEMM_OK
P = 1 << 20  # an aligned address that no check dereferences


@pytest.fixture(scope="module")
def lib():
    build.build()
    return feedforward._load()


# ---------------------------------------------------------------- the oracle

def _numeric(f, x, step=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = step
        g[i] = (f(x + e) - f(x - e)) / (2 * step)
    return g


def test_layer_norm_gradient_against_differences():
    rng = np.random.default_rng(0)
    x, w, b, d = rng.normal(size=(3, 7)) + 2, rng.normal(size=7), rng.normal(size=7), rng.normal(size=(3, 7))
    y, mean, rstd = of.layer_norm(x, w, b, 1e-3)
    dx, dw, db = of.layer_norm_grad(d, x, w, mean, rstd)
    # differences with a step h are off by h^2 times a third derivative of order 1, and 1e-16 / h
    assert np.abs(dx - _numeric(lambda t: (of.layer_norm(t, w, b, 1e-3)[0] * d).sum(), x)).max() < 1e-8
    assert np.abs(dw - _numeric(lambda t: (of.layer_norm(x, t, b, 1e-3)[0] * d).sum(), w)).max() < 1e-8
    assert np.abs(db - _numeric(lambda t: (of.layer_norm(x, w, t, 1e-3)[0] * d).sum(), b)).max() < 1e-8


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
def test_gated_gradient_against_differences(act):
    rng = np.random.default_rng(1)
    a, w, bias, d = (rng.normal(size=s) for s in ((4, 5), (5, 6), (6,), (4, 3)))
    up = of.gated(a, w, bias, act)[1]
    dup = of.gated_grad(d, up, act)
    loss = lambda a, w, bias: (of.gated(a, w, bias, act)[0] * d).sum()  # noqa: E731
    assert np.abs(dup @ w.T - _numeric(lambda t: loss(t, w, bias), a)).max() < 1e-7
    assert np.abs(a.T @ dup - _numeric(lambda t: loss(a, t, bias), w)).max() < 1e-7
    assert np.abs(dup.sum(0) - _numeric(lambda t: loss(a, w, t), bias)).max() < 1e-7


def test_gates_at_worked_values():
    x = np.array([0.0, 1.0, -2.0])
    assert np.allclose(of.gate(x, "silu")[0], [0, 0.7310585786300049, -0.2384058440442351], atol=1e-15)
    assert np.allclose(of.gate(x, "gelu")[0], [0, 0.8413447460685429, -0.0455002638963584], atol=1e-15)
    assert np.allclose(of.gate(x, "gelu_tanh")[0], [0, 0.8411919906082768, -0.0454023059122250], atol=1e-14)
    assert np.array_equal(of.gate(x, "relu")[1], [0, 1, 0])


def test_blocks_at_worked_values():
    a, b = np.zeros((2, 130)), np.zeros((129, 130))
    a[0, 0], a[0, 129], b[128, 0], b[128, 129], b[0, 0] = 2, 3, 5, 7, 11
    sa, sb = np.array([[2.0, 4.0], [1.0, 1.0]]), np.array([[1.0, 1.0], [0.5, 0.25]])
    c, s = of.matmul_blocks(a, b, sa, sb, 128)
    assert c[0, 128] == 2 * 5 * 2 * 0.5 + 3 * 7 * 4 * 0.25 and c[0, 0] == 2 * 11 * 2 and c[1].max() == 0
    assert np.array_equal(of.block_scales(a * 448, 1), [[2, 3], [1e-12 / 448, 1e-12 / 448]])
    assert np.array_equal(of.block_scales(b * 448, 128), [[11, 1e-12 / 448], [5, 7]])


# ---------------------------------------------------------------- the C interface

def test_header_declarations_match_binding(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:int|int64_t)\s+(gemm_[a-z_0-9]+)\s*\(", text, flags=re.M))
    assert sorted(names) == sorted(feedforward.EXPORTS)
    for name in names:
        assert hasattr(lib, name)


def _norm(lib, type=1, rows=2, cols=8, x=P, ldx=8, res=None, ldr=8, w=2 * P, b=None, h=None, ldh=8, y_type=1, y=3 * P,
          ldy=8, scale=None, mean=None, rstd=None):
    return lib.gemm_layernorm(type, rows, cols, x, ldx, res, ldr, w, b, 1e-5, h, ldh, y_type, y, ldy, scale, mean, rstd,
                              None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), INVALID), (dict(type=-1), INVALID), (dict(y_type=0), INVALID), (dict(rows=-1), INVALID),
    (dict(rows=1 << 31), INVALID), (dict(cols=-1), INVALID), (dict(cols=16385, ldx=20000, ldy=20000), INVALID),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(ldx=7), INVALID),
    (dict(ldy=7), INVALID), (dict(res=4 * P, ldr=7), INVALID), (dict(res=4 * P, h=5 * P, ldh=7), INVALID),
    (dict(y_type=3), INVALID), (dict(scale=6 * P), INVALID), (dict(y=P + 2), INVALID), (dict(y=2 * P), INVALID),
    (dict(b=3 * P + 4), INVALID), (dict(res=4 * P, y=4 * P), INVALID), (dict(res=4 * P, h=P + 16), INVALID),
    (dict(mean=3 * P), INVALID), (dict(rstd=P + 4), INVALID),
    (dict(x=P + 1), MISALIGNED), (dict(y=3 * P + 1), MISALIGNED), (dict(b=6 * P + 1), MISALIGNED),
    (dict(rstd=6 * P + 2), MISALIGNED), (dict(mean=6 * P + 2), MISALIGNED),
    (dict(rows=0, x=None, y=None), OK), (dict(cols=0), OK),
])
def test_layer_norm_arguments(lib, kw, code):
    assert _norm(lib, **kw) == code


def _norm_grad(lib, type=1, rows=2, cols=8, dy=P, lddy=8, h=2 * P, ldh=8, w=3 * P, mean=9 * P, rstd=4 * P, dh=None,
               lddh=8, dx=5 * P, lddx=8, dw=6 * P, db=8 * P, ws=7 * P, bytes=128):
    return lib.gemm_layernorm_backward(type, rows, cols, dy, lddy, h, ldh, w, mean, rstd, dh, lddh, dx, lddx, dw, db, ws,
                                       bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), INVALID), (dict(rows=-1), INVALID), (dict(cols=16385), INVALID), (dict(dy=None), INVALID),
    (dict(h=None), INVALID), (dict(mean=None), INVALID), (dict(rstd=None), INVALID), (dict(dx=None), INVALID),
    (dict(dw=None), INVALID), (dict(db=6 * P), INVALID), (dict(lddy=7), INVALID), (dict(ldh=7), INVALID),
    (dict(lddx=7), INVALID), (dict(dh=P, lddh=7), INVALID), (dict(bytes=127), INVALID), (dict(ws=None), INVALID),
    (dict(dx=P + 2), INVALID), (dict(dx=2 * P + 16), INVALID), (dict(dx=9 * P), INVALID), (dict(dx=8 * P), INVALID),
    (dict(h=2 * P + 1), MISALIGNED), (dict(db=8 * P + 1), MISALIGNED), (dict(mean=9 * P + 2), MISALIGNED),
    (dict(ws=7 * P + 4), MISALIGNED), (dict(cols=0), OK),
])
def test_layer_norm_backward_arguments(lib, kw, code):
    assert _norm_grad(lib, **kw) == code


def _gated(lib, type=1, M=4, F=8, K=8, A=P, lda=8, W=2 * P, ldw=8, layout=1, act=0, bias=None, C=3 * P, ldc=8, up=None,
           ldup=16, ws=None, bytes=0):
    return lib.gemm_gated(type, M, F, K, A, lda, W, ldw, layout, act, bias, C, ldc, up, ldup, ws, bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=2), INVALID), (dict(type=3), INVALID), (dict(M=-1), INVALID), (dict(F=-1), INVALID), (dict(K=-1), INVALID),
    (dict(M=1 << 31), INVALID), (dict(F=1 << 30), INVALID), (dict(layout=2), INVALID), (dict(act=4), INVALID),
    (dict(act=-1), INVALID), (dict(A=None), INVALID), (dict(W=None), INVALID), (dict(C=None), INVALID),
    (dict(lda=7), INVALID), (dict(ldw=7), INVALID), (dict(layout=0, ldw=15), INVALID), (dict(ldc=7), INVALID),
    (dict(up=5 * P, ldup=15), INVALID), (dict(C=P + 16), INVALID), (dict(C=2 * P), INVALID), (dict(bias=3 * P), INVALID),
    (dict(up=3 * P + 32), INVALID), (dict(up=P), INVALID), (dict(up=5 * P, bias=5 * P), INVALID),
    (dict(A=P + 8), MISALIGNED), (dict(W=2 * P + 2), MISALIGNED), (dict(C=3 * P + 1), MISALIGNED),
    (dict(up=5 * P + 1), MISALIGNED), (dict(bias=5 * P + 1), MISALIGNED), (dict(lda=12), MISALIGNED),
    (dict(ldw=12), MISALIGNED), (dict(layout=0, F=12, ldw=24, ldc=12), MISALIGNED),  # the value half off a boundary
    (dict(lda=12, ws=6 * P, bytes=4 * 128 - 1), MISALIGNED), (dict(lda=12, ws=3 * P, bytes=4 * 128), INVALID),
    (dict(lda=12, ws=6 * P + 16, bytes=4 * 128), MISALIGNED), (dict(M=0, C=None), OK), (dict(F=0), OK),
])
def test_gated_arguments(lib, kw, code):
    assert _gated(lib, **kw) == code


def _gated_grad(lib, type=1, M=4, F=8, K=8, dC=P, lddc=8, up=2 * P, ldup=16, A=3 * P, lda=8, W=4 * P, ldw=8, layout=1,
                act=0, dA=5 * P, ldda=8, dW=6 * P, lddw=8, db=7 * P, ws=8 * P, bytes=1 << 16):
    return lib.gemm_gated_backward(type, M, F, K, dC, lddc, up, ldup, A, lda, W, ldw, layout, act, dA, ldda, dW, lddw,
                                   db, ws, bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=2), INVALID), (dict(M=-1), INVALID), (dict(layout=2), INVALID), (dict(act=4), INVALID),
    (dict(dC=None), INVALID), (dict(up=None), INVALID), (dict(A=None), INVALID), (dict(W=None), INVALID),
    (dict(lddc=7), INVALID), (dict(ldup=15), INVALID), (dict(lda=7), INVALID), (dict(ldw=7), INVALID),
    (dict(ldda=7), INVALID), (dict(lddw=7), INVALID), (dict(layout=0, ldw=16, lddw=15), INVALID), (dict(ws=None), INVALID),
    (dict(bytes=256), INVALID), (dict(dA=P), INVALID), (dict(dW=3 * P + 8), INVALID), (dict(dA=6 * P), INVALID),
    (dict(db=2 * P + 6), INVALID), (dict(ws=4 * P), INVALID), (dict(ws=7 * P), INVALID), (dict(dC=P + 1), MISALIGNED),
    (dict(up=2 * P + 1), MISALIGNED), (dict(A=3 * P + 8), MISALIGNED), (dict(W=4 * P + 8), MISALIGNED),
    (dict(dA=5 * P + 1), MISALIGNED), (dict(db=7 * P + 1), MISALIGNED), (dict(ws=8 * P + 64), MISALIGNED),
    (dict(dA=None, dW=None, db=None, dC=None), OK), (dict(F=0, dA=None), OK), (dict(M=0, dW=None, db=None), OK),
])
def test_gated_backward_arguments(lib, kw, code):
    assert _gated_grad(lib, **kw) == code


def test_gated_workspaces(lib):
    size, grad = lib.gemm_gated_workspace, lib.gemm_gated_backward_workspace
    assert size(1, 4, 8, 8, 8, 8, 1) == size(1, 4, 8, 8, 8, 16, 0) == size(1, 0, 8, 8, 8, 8, 1) == 0
    assert size(1, 4, 8, 9, 9, 16, 1) == 4 * 128                          # rows of A of 18 bytes
    assert size(1, 4, 8, 9, 16, 9, 1) == 16 * 128                         # of W
    assert size(1, 4, 12, 8, 8, 24, 0) == 8 * 128                         # a value half of 24 bytes, off a boundary
    assert grad(1, 4, 8, 8, 8, 8, 1, 1, 0, 0) == 4 * 128                  # dup
    assert grad(1, 4, 8, 8, 8, 8, 1, 0, 0, 1) == 4 * 128 + 4 * 2 * 8 * 4  # and partial sums of dbias
    assert grad(1, 4, 8, 8, 8, 8, 1, 1, 1, 0) == 4 * 128
    assert grad(1, 4, 8, 9, 9, 16, 1, 0, 1, 0) == 4 * 128 + 4 * 128      # rows of A of 18 bytes
    assert grad(1, 4, 8, 8, 8, 8, 1, 0, 0, 0) == grad(1, 0, 8, 8, 8, 8, 1, 1, 1, 1) == 0
    assert lib.gemm_layernorm_backward_workspace(3, 64) == 3 * 2 * 64 * 4
    assert lib.gemm_layernorm_backward_workspace(0, 64) == 0


def _blocks(lib, M=4, N=8, K=32, A=P, lda=32, sa=2 * P, as_row=1, as_block=4, B=3 * P, ldb=32, sb=4 * P, bs_row=1,
            bs_block=8, b_rows=1, C=5 * P, ldc=8):
    return lib.gemm_e4m3_blocks(M, N, K, A, lda, sa, as_row, as_block, B, ldb, sb, bs_row, bs_block, b_rows, C, ldc, None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID), (dict(M=1 << 31), INVALID),
    (dict(b_rows=2), INVALID), (dict(b_rows=0), INVALID), (dict(A=None), INVALID), (dict(B=None), INVALID),
    (dict(sa=None), INVALID), (dict(sb=None), INVALID), (dict(C=None), INVALID), (dict(lda=31), INVALID),
    (dict(ldb=31), INVALID), (dict(ldc=7), INVALID), (dict(as_row=-1), INVALID), (dict(bs_block=-1), INVALID),
    (dict(C=P + 16), INVALID), (dict(C=3 * P), INVALID), (dict(C=2 * P), INVALID), (dict(C=4 * P + 16), INVALID),
    (dict(lda=40), MISALIGNED), (dict(ldb=40), MISALIGNED), (dict(A=P + 8), MISALIGNED), (dict(B=3 * P + 1), MISALIGNED),
    (dict(sa=2 * P + 2), MISALIGNED), (dict(sb=4 * P + 1), MISALIGNED), (dict(C=5 * P + 1), MISALIGNED),
    (dict(M=0, A=None, C=None), OK), (dict(N=0), OK),
])
def test_matmul_blocks_arguments(lib, kw, code):
    assert _blocks(lib, **kw) == code


def _quantize(lib, type=1, rows=4, cols=200, x=P, ldx=200, tall=1, transpose=0, q=2 * P, ldq=208, s=3 * P, s_row=1,
              s_block=4):
    return lib.gemm_quantize_blocks(type, rows, cols, x, ldx, tall, transpose, q, ldq, s, s_row, s_block, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), INVALID), (dict(rows=-1), INVALID), (dict(cols=-1), INVALID), (dict(tall=2), INVALID),
    (dict(transpose=2), INVALID), (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID),
    (dict(ldx=199), INVALID), (dict(ldq=199), INVALID), (dict(transpose=1, ldq=3), INVALID), (dict(s_row=-1), INVALID),
    (dict(s_block=3), INVALID), (dict(s_row=0), INVALID), (dict(s_row=1, s_block=1), INVALID), (dict(q=P), INVALID),
    (dict(s=P + 4), INVALID), (dict(s=2 * P), INVALID), (dict(x=P + 1), MISALIGNED), (dict(s=3 * P + 2), MISALIGNED),
    (dict(rows=0, x=None), OK), (dict(cols=0), OK),
])
def test_quantize_blocks_arguments(lib, kw, code):
    assert _quantize(lib, **kw) == code


def test_no_device_is_reported(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for call in (_norm, _norm_grad, _gated, _gated_grad, _blocks, _quantize):
        assert call(lib) == gemm.GEMM_ERR_UNSUPPORTED_DEVICE
    assert _quantize(lib, s_row=2, s_block=1) == gemm.GEMM_ERR_UNSUPPORTED_DEVICE  # scales row by row


# ---------------------------------------------------------------- Python

def test_python_refusals():
    """What the binding refuses by itself, on CPU tensors: types, shapes, strides and memory."""
    x = torch.zeros(2, 8, dtype=torch.bfloat16)
    w, q = torch.zeros(16, 8, dtype=torch.bfloat16), torch.zeros(2, 16).to(torch.float8_e4m3fn)
    one = torch.ones(2, 1)
    for error, call in (
            (TypeError, lambda: feedforward.layer_norm(x.double(), x[0].double())),
            (TypeError, lambda: feedforward.layer_norm(x, x[0], out_dtype=torch.float16)),
            (ValueError, lambda: feedforward.layer_norm(x, x[0])),  # not CUDA
            (TypeError, lambda: feedforward.layer_norm_backward(x, x.int(), x[0], one[:, 0], one[:, 0])),
            (TypeError, lambda: feedforward.gated_matmul(x.float(), w.float())),
            (TypeError, lambda: feedforward.gated_matmul(x, w.half(), layout=1)),
            (ValueError, lambda: feedforward.gated_matmul(x, w, layout=1)),
            (ValueError, lambda: feedforward.gated_matmul(x, w, layout=1, activation="tanh")),
            (ValueError, lambda: feedforward.gated_matmul_backward(x, x, w, w, layout=1, activation=None)),
            (TypeError, lambda: feedforward.matmul_blocks(x, q, one, one)),
            (ValueError, lambda: feedforward.matmul_blocks(q, q, one, one)),
            (TypeError, lambda: feedforward.quantize_blocks(x.int())),
            (ValueError, lambda: feedforward.quantize_blocks(x)),
            (ValueError, lambda: feedforward.quantize_blocks(x, rows=64)),
            (TypeError, lambda: feedforward.quantize_blocks(None))):
        with pytest.raises(error):
            call()


def test_an_unbuilt_tree_says_what_to_do(lib, monkeypatch):
    monkeypatch.setattr(feedforward, "_ext", None)
    monkeypatch.delattr(dense_gemm_tensor_gb300, "_feedforward", raising=False)
    monkeypatch.setitem(sys.modules, "dense_gemm_tensor_gb300._feedforward", None)
    with pytest.raises(RuntimeError, match=r"_feedforward.so .*build\.build\(\)"):
        feedforward.quantize_blocks(torch.zeros(2, 8))
