"""The mixture-of-experts operators' edges that need no GPU: refusals of the C
interface, workspace sizes and the build of the compiled binding."""

import subprocess
import sys

import pytest
import torch

import dense_gemm_tensor_gb300
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


def test_workspace_of_rows_of_any_pitch(lib):
    rows, grad = lib.gemm_grouped_rows_workspace, lib.gemm_grouped_wgrad_rows_workspace
    for gathered in (0, 1):
        assert rows(1, 4, 5, 65, 5, 65, gathered) == 5 * 256      # rows of 130 bytes are copied at a 128-byte pitch
        assert rows(3, 4, 5, 65, 5, 65, gathered) == 5 * 128
        assert rows(1, 4, 5, 65, 1, 65, gathered) == 0            # the pitch of one row says nothing
        assert rows(1, 4, 5, 65, 5, 72, gathered) == 0            # rows of 144 bytes are read where they are
        assert rows(1, 4, 0, 65, 0, 65, gathered) == 0
    assert rows(1, 4, 512, 65, 9, 72, 1) == lib.gemm_grouped_workspace(1, 4, 512, 65) == 512 * 256
    slabs = 2 * 64 * (256 + 128)
    assert grad(2, 3, 65, 64, 3, 64, 0, 72) == lib.gemm_grouped_wgrad_workspace(2, 3, 65, 64, 0) == slabs
    assert grad(2, 3, 65, 64, 3, 64, 1, 72) == slabs + 3 * 128
    assert grad(2, 3, 65, 64, 3, 64, 0, 65) == slabs + 3 * 256
    assert grad(2, 3, 65, 60, 3, 60, 0, 65) == slabs + 3 * (128 + 256)
    assert grad(2, 1, 65, 60, 1, 60, 0, 65) == slabs


def test_rows_of_any_pitch_need_their_workspace(lib):
    for kw in (dict(), dict(rows=5 * P)):
        assert _grouped(lib, lda=12, ws=6 * P, bytes=4 * 128 - 1, **kw) == MISALIGNED
        assert _grouped(lib, lda=12, ws=4 * P, bytes=4 * 128, **kw) == INVALID            # it is C
        assert _grouped(lib, lda=12, A=2 * P + 8, ws=6 * P, bytes=4 * 128, **kw) == MISALIGNED
    grad = dict(groups=2, off=P, slots=4, N=8, K=8, A=2 * P, a_rows=4, lda=8, rows=None, dC=3 * P, lddc=12, dW=4 * P,
                lddw=8, sdw=64, layout=1, ws=7 * P, bytes=2 * 64 * 256 + 4 * 128 - 1)
    assert lib.gemm_bf16_grouped_wgrad(*grad.values(), None) == MISALIGNED
    grad["bytes"], grad["dC"] = 2 * 64 * 256 + 4 * 128, 3 * P + 2
    assert lib.gemm_bf16_grouped_wgrad(*grad.values(), None) == MISALIGNED


def test_workspace_of_weights_that_are_copied(lib):
    def size(type=1, E=3, N=40, K=24, ldw=None, sw=None, layout=1, act=0):
        w_rows, w_cols = (N, K) if layout else (K, N)
        ldw = w_cols if ldw is None else ldw
        return lib.gemm_grouped_weights_workspace(type, E, N, K, ldw, w_rows * ldw if sw is None else sw, layout, act)

    assert size() == size(layout=0) == size(E=1, sw=1) == 0
    assert size(K=25) == 3 * 40 * 128                        # rows of 50 bytes
    assert size(layout=0, N=65) == 3 * 24 * 256
    assert size(sw=40 * 24 + 4) == 3 * 40 * 128              # matrices off 16-byte multiples
    assert size(K=25, N=1, sw=32) == size(E=1, K=25, N=1) == 0  # one row a matrix
    assert size(type=3) == 3 * 40 * 128 and size(type=3, K=32) == 0
    assert size(layout=0, act=4, N=40) == 3 * 24 * 2 * 128   # halves of 40 bytes, each on a boundary of its own
    assert size(layout=0, act=4, N=32) == size(act=4, N=42) == 0
    assert size(K=0) == 0


def test_copied_weights_need_their_workspace(lib):
    copied = 2 * 8 * 128
    for kw in (dict(ldw=12, sw=96), dict(sw=68)):
        assert _grouped(lib, ws=6 * P, bytes=copied - 1, **kw) == MISALIGNED
        assert _grouped(lib, ws=4 * P, bytes=copied, **kw) == INVALID                     # it is C
        assert _grouped(lib, W=3 * P + 8, ws=6 * P, bytes=copied, **kw) == MISALIGNED
        assert _grouped(lib, lda=12, ws=6 * P, bytes=copied + 4 * 128 - 1, **kw) == MISALIGNED
    gated = dict(act=4, N=24, ldw=24, sw=192, ldc=12, layout=0)
    assert _grouped(lib, ws=6 * P, bytes=2 * copied - 1, **gated) == MISALIGNED
    assert _grouped(lib, ws=4 * P, bytes=2 * copied, **gated) == INVALID


@pytest.fixture
def compiled(monkeypatch, tmp_path):
    """The binding's build with its files in tmp_path and a compiler that only leaves a file; the list of its runs."""
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_experts.so"))
    monkeypatch.setattr(build, "BINDING_STAMP", str(tmp_path / "b" / "experts_binding.txt"))
    runs = []

    def run(cmd, **kw):
        runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    return runs


def test_the_binding_is_built_anew_for_another_torch(compiled, monkeypatch):
    build._build_binding()
    build._build_binding()
    assert len(compiled) == 1
    monkeypatch.setattr(build, "_binding_stamp", lambda: "another torch")
    build._build_binding()
    build._build_binding()
    assert len(compiled) == 2


def test_the_library_is_built_without_torch(compiled, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    build._build_binding()
    assert compiled == []


def test_an_unbuilt_tree_says_what_to_do(lib, monkeypatch, tmp_path):
    x = torch.zeros(2, 8)
    monkeypatch.setattr(experts, "_ext", None)
    monkeypatch.delattr(dense_gemm_tensor_gb300, "_experts", raising=False)
    monkeypatch.setitem(sys.modules, "dense_gemm_tensor_gb300._experts", None)
    with pytest.raises(RuntimeError, match=r"_experts.so .*build\.build\(\)"):
        experts.route(x, 2)
    monkeypatch.setattr(experts, "_lib", None)
    monkeypatch.setattr(gemm, "_lib", None)
    monkeypatch.setattr(gemm, "_LIB_PATH", str(tmp_path / "none.so"))
    with pytest.raises(RuntimeError, match=r"none.so is missing: build it"):
        experts.route(x, 2)
