"""The feed-forward operators on the GPU at the ends of what their interface allows:
scales far from 1, the quantiser's operands in the product, outputs in their inputs' buffers.
Helpers and tolerances are those of test_gpu_feedforward.py."""

import numpy as np
import pytest
import torch

from dense_gemm_tensor_gb300 import feedforward as ff
from dense_gemm_tensor_gb300 import gemm
from oracle import feedforward as of
from test_gpu_feedforward import E4M3, _accept, _gen, _lib, _normal, _np, _pitch16  # noqa: F401

pytestmark = pytest.mark.gpu


# few rows by every width, pairs of CTAs with 128- and with 256-wide tiles
@pytest.mark.parametrize("M,N,K", [(5, 200, 300), (20, 130, 2100), (64, 257, 384), (70, 300, 2100), (300, 129, 300),
                                   (1000, 9000, 300)])
@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("power", [115, -115])
def test_matmul_blocks_takes_the_product_of_its_scales(M, N, K, b_rows, power):
    """One operand's scales of about 2^115 and the other's of 2^-115: a block's sum (here up to 1e6) times one alone
    may pass fp32's range, times their product it does not. Powers of two change no rounding, so that the result is that of
    scales about 1 bit for bit."""
    a = (100 * torch.rand((M, K), generator=_gen(1))).to(E4M3)
    b = (100 * torch.rand((N, K), generator=_gen(2))).to(E4M3)
    blocks = -(-K // 128)
    sa = 0.5 + torch.rand((M, blocks), generator=_gen(3))
    sb = 0.5 + torch.rand((N if b_rows == 1 else -(-N // 128), blocks), generator=_gen(4))
    want, s = of.matmul_blocks(_np(a.float()), _np(b.float()), _np(sa), _np(sb), b_rows)
    ad, bd = _pitch16(a), _pitch16(b)
    one = ff.matmul_blocks(ad, bd, sa.cuda(), sb.cuda())
    _accept(one, want, s, "bf16")
    assert torch.equal(ff.matmul_blocks(ad, bd, (sa * 2.0 ** power).cuda(), (sb * 2.0 ** -power).cuda()), one)


# the quantiser and the product together: tails along every dimension, few rows and pairs
@pytest.mark.parametrize("M,N,K", [(200, 260, 300), (20, 130, 257), (385, 129, 1000), (129, 300, 40)])
def test_products_of_quantised_operands(M, N, K):
    """A product and its gradients against the float64 product of what the quantised operands stand for, by the ordinary
    acceptance rule. On 200 x 260 x 300 it refuses 50398 of 52000 entries of a product without its last block, or with
    that block's scale doubled, where a bound for the unquantised product refuses 3."""
    a, w, dc = _normal((M, K), "bf16", 5), _normal((N, K), "bf16", 6, 0.1), _normal((M, N), "bf16", 7)

    def product(x, y, tall=1, tx=False, ty=False):
        qx = ff.quantize_blocks(x.cuda(), transpose=tx)
        qy = ff.quantize_blocks(y.cuda(), rows=tall, transpose=ty)
        got = ff.matmul_blocks(qx.q, qy.q, qx.scale, qy.scale)
        vx, vy = (_np(q.q.float()) * of.spread(_np(q.scale), q.q.shape, t) for q, t in ((qx, 1), (qy, tall)))
        # (each stands for its matrix: half a spacing of E4M3 off, 2^-4 of a value or 2^-10 of its scale)
        for v, t, q, rows in ((vx, x.t() if tx else x, qx, 1), (vy, y.t() if ty else y, qy, tall)):
            assert np.all(np.abs(v - _np(t)) <= 2.0 ** -4 * 1.001 * np.abs(_np(t)) +
                          2.0 ** -10 * of.spread(_np(q.scale), q.q.shape, rows))
        _accept(got, vx @ vy.T, np.abs(vx) @ np.abs(vy).T, "bf16")

    product(a, w, tall=128)                            # A W^T
    product(dc, w, tall=128, ty=True)                  # dA = dC W
    product(dc, a, tx=True, ty=True)                   # dW = dC^T A
    product(a, w)                                      # both in 1 x 128


# ---------------------------------------------------------------- layer norm in place

def _buffer(t, pad):
    """t with rows `pad` elements further apart, on the GPU: (the whole buffer, the matrix in it)."""
    full = torch.full((t.shape[0], t.shape[1] + pad), 7.0, dtype=t.dtype, device="cuda")
    full[:, :t.shape[1]] = t.cuda()
    return full, full[:, :t.shape[1]]


IN_PLACE = [(1500, 99), (3000, 33), (40, 1023), (9, 8191), (7, 1), (700, 96), (3, 16383), (33, 5120)]


@pytest.mark.parametrize("rows,cols", IN_PLACE)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_layer_norm_in_place(rows, cols, dtype, pad):
    """Outputs in the buffers that the header allows (h in x's or the residual's, y in x's) are those of outputs apart, bit
    for bit. In rows of odd width a 16-byte piece holds the end of one row and the start of the next, whose block may be
    writing it."""
    lib, code = ff._load(), {"f16": 0, "bf16": 1, "f32": 2}[dtype]
    x, r = _normal((rows, cols), dtype, 20) + 1, _normal((rows, cols), dtype, 21)
    w, b = _normal((cols,), dtype, 22).cuda(), _normal((cols,), dtype, 23).cuda()

    def call(h_in=None, y_in=None, residual=True):
        (fx, xd), (fr, rd), (fh, hd), (fy, yd) = (_buffer(t, pad) for t in (x, r, torch.zeros_like(x), torch.zeros_like(x)))
        hd, yd = {"x": xd, "r": rd, None: hd}[h_in], xd if y_in == "x" else yd
        mean, rstd = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
        ld = cols + pad
        torch.cuda.synchronize()
        st = lib.gemm_layernorm(code, rows, cols, xd.data_ptr(), ld, rd.data_ptr() if residual else None, ld, w.data_ptr(),
                                b.data_ptr(), 1e-5, hd.data_ptr() if residual else None, ld, code, yd.data_ptr(), ld, None,
                                mean.data_ptr(), rstd.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert st == gemm.GEMM_OK
        torch.cuda.synchronize()
        assert all((f[:, cols:] == 7.0).all() for f in (fx, fr, fh, fy))
        return (yd, mean, rstd) + ((hd,) if residual else ())

    for residual, places in ((True, [("x", None), ("r", None), (None, "x"), ("r", "x")]), (False, [(None, "x")])):
        want = call(residual=residual)
        for h_in, y_in in places:
            for got, ref in zip(call(h_in, y_in, residual), want):
                assert torch.equal(got, ref), (h_in, y_in)


@pytest.mark.parametrize("rows,cols", IN_PLACE)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_layer_norm_backward_in_place(rows, cols, dtype, pad):
    """dx in dh's or dy's buffer, as above; there the next row's copy is under way while this one's result is stored."""
    lib, code = ff._load(), {"f16": 0, "bf16": 1, "f32": 2}[dtype]
    dy, h, dh = (_normal((rows, cols), dtype, 30 + i) for i in range(3))
    w = _normal((cols,), dtype, 33).cuda()
    mean, rstd = torch.randn(rows, generator=_gen(34)).cuda(), (0.5 + torch.rand(rows, generator=_gen(35))).cuda()
    need = lib.gemm_layernorm_backward_workspace(rows, cols)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")

    def call(into=None, path=True):
        (fy, yd), (fh, hd), (fp, pd), (fx, xd) = (_buffer(t, pad) for t in (dy, h, dh, torch.zeros_like(dy)))
        xd = {"dy": yd, "dh": pd, None: xd}[into]
        dw, db = torch.zeros_like(w), torch.zeros_like(w)
        ld = cols + pad
        torch.cuda.synchronize()
        st = lib.gemm_layernorm_backward(code, rows, cols, yd.data_ptr(), ld, hd.data_ptr(), ld, w.data_ptr(), mean.data_ptr(),
                                         rstd.data_ptr(), pd.data_ptr() if path else None, ld, xd.data_ptr(), ld, dw.data_ptr(),
                                         db.data_ptr(), ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
        assert st == gemm.GEMM_OK
        torch.cuda.synchronize()
        assert all((f[:, cols:] == 7.0).all() for f in (fy, fh, fp, fx))
        return xd, dw, db

    for path, places in ((True, ["dh", "dy"]), (False, ["dy"])):
        want = call(path=path)
        for into in places:
            for got, ref in zip(call(into, path), want):
                assert torch.equal(got, ref), into
