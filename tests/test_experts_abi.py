"""The C interface of the mixture-of-experts operators without a GPU: exports,
workspace sizes and refused arguments; and the Python functions' refusals."""

import os
import re

import pytest
import torch

from dense_gemm_tensor_gb300 import build, experts, gemm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dgt_experts.h")
INVALID, MISALIGNED = gemm.GEMM_ERR_INVALID_VALUE, gemm.GEMM_ERR_MISALIGNED
P = 1 << 20  # an aligned address that no check dereferences


@pytest.fixture(scope="module")
def lib():
    build.build()
    return experts._load()


def test_header_declarations_match_binding(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:int|int64_t)\s+(gemm_[a-z_0-9]+)\s*\(", text, flags=re.M))
    assert sorted(names) == sorted(experts.EXPORTS)
    for name in names:
        assert hasattr(lib, name)


def test_workspace_sizes(lib):
    assert lib.gemm_route_workspace(0, 8, 2) == 0
    assert lib.gemm_route_workspace(32, 64, 8) == 0          # one block does it all
    assert lib.gemm_route_workspace(33, 64, 8) == 2 * 64 * 4  # blocks of 32 tokens
    assert lib.gemm_route_workspace(1 << 20, 64, 8) == 152 * 64 * 4
    assert lib.gemm_grouped_workspace(1, 4, 63, 64) == 0           # few rows a group: gathered on the way
    assert lib.gemm_grouped_workspace(1, 4, 512, 65) == 512 * 256  # rows of 130 bytes, 128-byte pitch
    assert lib.gemm_grouped_workspace(3, 4, 512, 65) == 512 * 128
    # a slab of 64 rows of dC and of A for each group, and the rows of A in slot order
    assert lib.gemm_grouped_wgrad_workspace(2, 3, 65, 64, 0) == 2 * 64 * (256 + 128)
    assert lib.gemm_grouped_wgrad_workspace(2, 3, 65, 64, 1) == 2 * 64 * (256 + 128) + 3 * 128
    assert lib.gemm_grouped_wgrad_workspace(2, 0, 65, 64, 1) == 0
    assert lib.gemm_rmsnorm_backward_workspace(0, 64) == 0
    assert lib.gemm_rmsnorm_backward_workspace(3, 64) == 3 * 64 * 4
    assert lib.gemm_rmsnorm_backward_workspace(10 ** 6, 64) == 608 * 64 * 4
    assert lib.gemm_rmsnorm_backward_workspace(10 ** 6, 5000) == 456 * 5000 * 4


def _norm(lib, type=1, rows=2, cols=8, x=P, ldx=8, res=None, ldr=8, w=2 * P, h=None, ldh=8, y_type=1, y=3 * P, ldy=8,
          scale=None, rstd=None):
    return lib.gemm_rmsnorm(type, rows, cols, x, ldx, res, ldr, w, 1e-6, h, ldh, y_type, y, ldy, scale, rstd, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), INVALID), (dict(type=7), INVALID), (dict(y_type=0), INVALID), (dict(rows=-1), INVALID),
    (dict(cols=-1), INVALID), (dict(cols=16385, ldx=20000, ldy=20000), INVALID), (dict(x=None), INVALID),
    (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(ldx=7), INVALID), (dict(ldy=7), INVALID),
    (dict(res=4 * P, ldr=7), INVALID), (dict(res=4 * P, h=5 * P, ldh=7), INVALID),
    (dict(y_type=3), INVALID),                         # 8-bit rows need their scales
    (dict(scale=6 * P), INVALID),                      # and only they have them
    (dict(y=P + 2), INVALID), (dict(res=4 * P, y=4 * P), INVALID), (dict(res=4 * P, h=P + 16), INVALID),
    (dict(x=P + 1), MISALIGNED), (dict(y=3 * P + 1), MISALIGNED), (dict(rstd=6 * P + 2), MISALIGNED),
    (dict(rows=0, x=None, y=None), gemm.GEMM_OK), (dict(cols=0), gemm.GEMM_OK),
])
def test_rms_norm_arguments(lib, kw, code):
    assert _norm(lib, **kw) == code


def _norm_grad(lib, type=1, rows=2, cols=8, dy=P, lddy=8, h=2 * P, ldh=8, w=3 * P, rstd=4 * P, dh=None, lddh=8,
               dx=5 * P, lddx=8, dw=6 * P, ws=7 * P, bytes=64):
    return lib.gemm_rmsnorm_backward(type, rows, cols, dy, lddy, h, ldh, w, rstd, dh, lddh, dx, lddx, dw, ws, bytes,
                                     None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), INVALID), (dict(rows=-1), INVALID), (dict(cols=16385), INVALID), (dict(dy=None), INVALID),
    (dict(h=None), INVALID), (dict(rstd=None), INVALID), (dict(dx=None), INVALID), (dict(dw=None), INVALID),
    (dict(lddy=7), INVALID), (dict(ldh=7), INVALID), (dict(lddx=7), INVALID), (dict(dh=P, lddh=7), INVALID),
    (dict(bytes=63), INVALID), (dict(ws=None), INVALID), (dict(dx=P + 2), INVALID), (dict(dx=2 * P + 16), INVALID),
    (dict(h=2 * P + 1), MISALIGNED), (dict(ws=7 * P + 4), MISALIGNED), (dict(cols=0), gemm.GEMM_OK),
])
def test_rms_norm_backward_arguments(lib, kw, code):
    assert _norm_grad(lib, **kw) == code


def _route(lib, type=2, tokens=4, E=8, logits=P, ld=8, bias=None, k=2, score=0, groups=1, kept=1, ids=2 * P,
           weights=3 * P, slots=4 * P, rows=5 * P, offsets=6 * P, ws=None, bytes=0):
    cfg = experts.RouteConfig(k, score, groups, kept, 1, 1.0)
    return lib.gemm_route(type, tokens, E, logits, ld, bias, cfg, ids, weights, slots, rows, offsets, ws, bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), INVALID), (dict(tokens=-1), INVALID), (dict(E=0), INVALID), (dict(E=1025, ld=1025), INVALID),
    (dict(k=0), INVALID), (dict(k=33, E=64, ld=64), INVALID), (dict(k=9), INVALID), (dict(score=2), INVALID),
    (dict(groups=3), INVALID), (dict(groups=0), INVALID), (dict(groups=64, E=64, ld=64), INVALID),
    (dict(groups=4, kept=5), INVALID), (dict(groups=4, kept=0), INVALID),
    (dict(groups=4, kept=1, k=3), INVALID),            # more than the kept groups hold
    (dict(ld=7), INVALID), (dict(logits=None), INVALID), (dict(ids=None), INVALID), (dict(weights=None), INVALID),
    (dict(slots=None), INVALID), (dict(rows=None), INVALID), (dict(offsets=None), INVALID),
    (dict(tokens=129), INVALID),                       # needs a workspace
    (dict(tokens=129, ws=7 * P, bytes=5 * 32 - 1), INVALID), (dict(tokens=1 << 30, k=2), INVALID),
    (dict(logits=P + 2), MISALIGNED), (dict(bias=P + 2), MISALIGNED), (dict(offsets=6 * P + 1), MISALIGNED),
])
def test_route_arguments(lib, kw, code):
    assert _route(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(E=0), INVALID), (dict(type=3), INVALID), (dict(dw=None), INVALID), (dict(out=None), INVALID),
    (dict(ldd=7), INVALID), (dict(out=P + 8), INVALID), (dict(out=4 * P + 2), MISALIGNED),
    (dict(tokens=0), gemm.GEMM_OK),
])
def test_route_backward_arguments(lib, kw, code):
    a = dict(type=2, tokens=4, E=8, logits=P, ld=8, ids=2 * P, dw=3 * P, out=4 * P, ldd=8) | kw
    cfg = experts.RouteConfig(2, 0, 1, 1, 1, 1.0)
    assert lib.gemm_route_backward(a["type"], a["tokens"], a["E"], a["logits"], a["ld"], a["ids"], a["dw"], cfg,
                                   a["out"], a["ldd"], None) == code


def _grouped(lib, name="gemm_bf16_grouped", groups=2, off=P, slots=4, N=8, K=8, A=2 * P, a_rows=4, lda=8, rows=None,
             W=3 * P, ldw=8, sw=64, C=4 * P, ldc=8, layout=1, act=0, row_scale=None, col_scale=None, bias=None, ws=None, bytes=0):
    epi = experts.GroupedEpilogue(1.0, row_scale, col_scale, bias, act)
    return getattr(lib, name)(groups, off, slots, N, K, A, a_rows, lda, rows, W, ldw, sw, C, ldc, layout, epi, ws, bytes,
                              None)


@pytest.mark.parametrize("kw,code", [
    (dict(groups=0), INVALID), (dict(groups=1025), INVALID), (dict(slots=-1), INVALID), (dict(N=-8), INVALID),
    (dict(K=1 << 31), INVALID), (dict(layout=2), INVALID), (dict(act=5), INVALID), (dict(act=-1), INVALID),
    (dict(act=4, N=7), INVALID), (dict(off=None), INVALID), (dict(A=None), INVALID), (dict(W=None), INVALID),
    (dict(C=None), INVALID), (dict(a_rows=3), INVALID), (dict(lda=0), INVALID), (dict(ldw=0), INVALID),
    (dict(ldc=7), INVALID), (dict(sw=56), INVALID), (dict(sw=-64), INVALID), (dict(C=2 * P + 16), INVALID),
    (dict(C=3 * P + 64), INVALID), (dict(name="gemm_e4m3_grouped", layout=0), INVALID),
    (dict(lda=12), MISALIGNED), (dict(ldw=12, sw=96), MISALIGNED), (dict(sw=68), MISALIGNED), (dict(A=2 * P + 8), MISALIGNED),
    (dict(W=3 * P + 2), MISALIGNED), (dict(C=4 * P + 1), MISALIGNED), (dict(rows=P + 2), MISALIGNED),
    (dict(bias=P + 1), MISALIGNED), (dict(row_scale=P + 2), MISALIGNED), (dict(col_scale=P + 2), MISALIGNED),
    (dict(act=4, N=24, ldw=24, sw=192, ldc=12, layout=0), MISALIGNED),  # the value half starts off a 16-byte boundary
    (dict(name="gemm_e4m3_grouped", lda=8), MISALIGNED),
    (dict(rows=5 * P, ws=6 * P, bytes=4 * 128 - 1), INVALID), (dict(rows=5 * P, ws=4 * P, bytes=4 * 128), INVALID),
    (dict(rows=5 * P, ws=6 * P + 16, bytes=4 * 128), MISALIGNED),
    (dict(slots=0, A=None, C=None), gemm.GEMM_OK), (dict(N=0), gemm.GEMM_OK),
])
def test_grouped_arguments(lib, kw, code):
    assert _grouped(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(groups=0), INVALID), (dict(layout=3), INVALID), (dict(off=None), INVALID), (dict(A=None), INVALID),
    (dict(dC=None), INVALID), (dict(dW=None), INVALID), (dict(a_rows=3), INVALID), (dict(lddc=0), INVALID),
    (dict(lddw=7), INVALID), (dict(sdw=56), INVALID), (dict(dW=2 * P), INVALID), (dict(lda=12), MISALIGNED),
    (dict(dC=3 * P + 8), MISALIGNED), (dict(dW=4 * P + 1), MISALIGNED), (dict(N=0), gemm.GEMM_OK),
    (dict(ws=None), INVALID), (dict(bytes=2 * 64 * 256 - 1), INVALID), (dict(rows=5 * P), INVALID),
    (dict(ws=4 * P, bytes=2 * 64 * 256), INVALID), (dict(ws=7 * P + 64), MISALIGNED),
])
def test_weight_grad_arguments(lib, kw, code):
    a = dict(groups=2, off=P, slots=4, N=8, K=8, A=2 * P, a_rows=4, lda=8, rows=None, dC=3 * P, lddc=8, dW=4 * P,
             lddw=8, sdw=64, layout=1, ws=7 * P, bytes=2 * 64 * 256) | kw
    assert lib.gemm_bf16_grouped_wgrad(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), INVALID), (dict(tokens=-1), INVALID), (dict(k=0), INVALID), (dict(k=33), INVALID),
    (dict(z=None), INVALID), (dict(slots=None), INVALID), (dict(y=None), INVALID), (dict(ldz=7), INVALID),
    (dict(ldy=7), INVALID), (dict(res=P, ldr=7), INVALID), (dict(y=P + 16), INVALID), (dict(res=5 * P, y=5 * P + 16), INVALID),
    (dict(z=P + 1), MISALIGNED), (dict(weights=P + 2), MISALIGNED), (dict(tokens=0, y=None), gemm.GEMM_OK),
])
def test_combine_arguments(lib, kw, code):
    a = dict(type=1, tokens=4, cols=8, k=2, z=P, ldz=8, nslots=8, slots=2 * P, weights=3 * P, res=None, ldr=8, y=4 * P,
             ldy=8) | kw
    assert lib.gemm_combine(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), INVALID), (dict(k=0), INVALID), (dict(dy=None), INVALID), (dict(z=None), INVALID),
    (dict(dz=None), INVALID), (dict(slots=None), INVALID), (dict(lddy=7), INVALID), (dict(lddz=7), INVALID),
    (dict(dz=P + 16), INVALID), (dict(dz=2 * P), INVALID), (dict(used=P + 2), MISALIGNED),
    (dict(tokens=0, used=None), gemm.GEMM_OK),
])
def test_combine_backward_arguments(lib, kw, code):
    a = dict(type=1, tokens=4, cols=8, k=2, dy=P, lddy=8, z=2 * P, ldz=8, nslots=8, slots=3 * P, weights=4 * P,
             used=5 * P, dz=6 * P, lddz=8, dweights=7 * P) | kw
    assert lib.gemm_combine_backward(*a.values(), None) == code


def test_no_device_is_reported(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    want = gemm.GEMM_ERR_UNSUPPORTED_DEVICE
    assert _norm(lib) == want and _norm_grad(lib) == want and _route(lib) == want and _grouped(lib) == want


def test_python_refusals():
    """What the binding refuses by itself, on CPU tensors: types, shapes, strides and memory."""
    f16, i32 = torch.zeros(2, 8, dtype=torch.float16), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        experts.rms_norm(f16.double(), f16[0].double())
    with pytest.raises(ValueError):
        experts.rms_norm(f16, f16[0])  # not CUDA
    with pytest.raises(TypeError):
        experts.expert_matmul(f16.float(), torch.zeros(2, 8, 8), i32)
    with pytest.raises(TypeError):
        experts.expert_matmul(f16, torch.zeros(2, 8, 8), i32)
    with pytest.raises(ValueError):
        experts.expert_matmul(f16, torch.zeros(2, 8, 8, dtype=torch.float16), i32, activation="tanh")
    with pytest.raises(ValueError):
        experts.expert_matmul(f16, torch.zeros(2, 8, 8, dtype=torch.float16), i32)
    with pytest.raises(TypeError):
        experts.expert_weight_grad(f16.float(), f16.float(), i32)
    with pytest.raises(TypeError):
        experts.route(torch.zeros(2, 4, dtype=torch.int32), 2)
    with pytest.raises(TypeError):
        experts.combine(torch.zeros(2, 4, dtype=torch.int32), i32.view(3, 1))
    with pytest.raises(ValueError):
        experts.route(torch.zeros(2, 4), 2, score="tanh")
    with pytest.raises(TypeError):
        experts.rms_norm([1.0], f16[0])
    with pytest.raises(TypeError):
        experts.rms_norm(f16, f16[0], out_dtype=torch.float32)


def test_binding_takes_every_argument():
    ext = experts._binding()
    with pytest.raises(TypeError):
        ext.rms_norm(torch.zeros(2, 8))
    with pytest.raises(ValueError):
        ext.bind({})
