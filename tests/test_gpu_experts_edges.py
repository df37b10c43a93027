"""The mixture-of-experts operators on the GPU at the edges of what they take:
values near the ends of the types' ranges, several host threads, no tokens,
operands of any width. Each case against the float64 oracle (oracle/experts.py);
tolerances as in test_gpu_experts.py where none is given.
"""

import numpy as np
import pytest
import torch

import oracle
from dense_gemm_tensor_gb300 import experts, gemm
from oracle import experts as ox

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_gemm_tensor_gb300 import build
    build.build()
    gemm.load()
    gemm.set_debug(0, 0)
    gemm.reset_device_status()
    yield
    assert gemm.device_status() == 0


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _normal(shape, dtype, seed, std=1.0):
    return (torch.randn(shape, generator=_gen(seed)) * std).to(DT[dtype])


def _np(t):
    return t.detach().cpu().double().numpy()


def _close(got, want, s, fmt, factor=1e-5):
    got, want = _np(got), np.asarray(want)
    allowed = 0.5 * oracle.ulp(want, fmt) + factor * np.asarray(s)
    bad = ~(np.abs(got - want) <= allowed)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


# ---------------------------------------------------------------- norm

# by the layout of the rows: whole pieces; contiguous of any width; padded of any width
@pytest.mark.parametrize("rows,cols,pad", [(5, 512, 0), (40, 5120, 0), (9, 333, 0), (7, 77, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e15, 1e17, 1e-13, 1e-14, 1.0])
def test_rms_norm_backward_of_large_and_small_rows(rows, cols, pad, dtype, size):
    """Rows whose norm's cube leaves fp32: the mean's term is of the size of dy's own, since dy goes along with h."""
    base = torch.randn((rows, cols), generator=_gen(1))
    h = (size * base).to(DT[dtype])
    dy = (base + 0.5 * torch.randn((rows, cols), generator=_gen(2))).to(DT[dtype])
    w = _normal((cols,), dtype, 3, 0.1) + 1
    rstd = torch.from_numpy(1 / np.sqrt((_np(h) ** 2).mean(1))).float()

    def dev(t):
        full = torch.zeros((rows, cols + pad), dtype=t.dtype)
        full[:, :cols] = t
        return full.cuda()[:, :cols]

    dx, dw = experts.rms_norm_backward(dev(dy), dev(h), w.cuda(), rstd.cuda())
    want_x, want_w = ox.rms_norm_grad(_np(dy), _np(h), _np(w), _np(rstd))
    g, xh, r = np.abs(_np(dy) * _np(w)), np.abs(_np(h) * _np(rstd)[:, None]), _np(rstd)[:, None]
    _close(dx, want_x, r * (g + xh * (g * xh).mean(1, keepdims=True)), dtype)
    _close(dw, want_w, (np.abs(_np(dy)) * xh).sum(0), dtype)
