"""The feed-forward operators on the GPU at the ends of what their interface allows:
scales far from 1, the quantiser's operands in the product. Helpers and tolerances are those of test_gpu_feedforward.py."""

import numpy as np
import pytest
import torch

from dense_gemm_tensor_gb300 import feedforward as ff
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
    acceptance rule: a block left out, or one with another's scale, is far outside it."""
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
