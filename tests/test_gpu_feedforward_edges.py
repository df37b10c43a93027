"""The feed-forward operators on the GPU at the ends of what their interface allows:
scales far from 1. Helpers and tolerances are those of test_gpu_feedforward.py."""

import numpy as np
import pytest
import torch

from dense_gemm_tensor_gb300 import feedforward as ff
from oracle import feedforward as of
from test_gpu_feedforward import E4M3, _accept, _gen, _lib, _np, _pitch16  # noqa: F401

pytestmark = pytest.mark.gpu


# few rows by every width, pairs of CTAs with 128- and with 256-wide tiles
@pytest.mark.parametrize("M,N,K", [(5, 200, 300), (20, 130, 2100), (64, 257, 384), (70, 300, 2100), (300, 129, 300),
                                   (1000, 9000, 300)])
@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("power", [115, -115])
def test_matmul_blocks_takes_the_product_of_its_scales(M, N, K, b_rows, power):
    """One operand's scales of about 2^115 and the other's of 2^-115: a block's sum (here up to 1e6) times either alone
    passes fp32's range, times their product it does not. Powers of two change no rounding, so that the result is that of
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
