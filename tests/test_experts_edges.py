"""The mixture-of-experts operators' edges that need no GPU: refusals of the C
interface, workspace sizes and the build of the compiled binding."""

import pytest

from dense_gemm_tensor_gb300 import build, experts, gemm

INVALID, MISALIGNED = gemm.GEMM_ERR_INVALID_VALUE, gemm.GEMM_ERR_MISALIGNED
P = 1 << 20  # an aligned address that no check dereferences


@pytest.fixture(scope="module")
def lib():
    build.build()
    return experts._load()


def _grouped(lib, name="gemm_bf16_grouped", groups=2, off=P, slots=4, N=8, K=8, A=2 * P, a_rows=4, lda=8, rows=None,
             W=3 * P, ldw=8, sw=64, C=4 * P, ldc=8, layout=1, act=0, row_scale=None, col_scale=None, bias=None, ws=None, bytes=0):
    epi = experts.GroupedEpilogue(1.0, row_scale, col_scale, bias, act)
    return getattr(lib, name)(groups, off, slots, N, K, A, a_rows, lda, rows, W, ldw, sw, C, ldc, layout, epi, ws, bytes,
                              None)


def test_row_scales_of_a_matrix_without_rows(lib):
    """Slots that name rows of an A of no rows have no scale to read, whatever K is."""
    for K in (0, 8):
        assert _grouped(lib, K=K, A=None, a_rows=0, rows=5 * P, row_scale=6 * P) == INVALID
