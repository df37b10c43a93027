"""The mixture-of-experts block end to end on a GB300: its serving pass and its
gradients against the block written out in 64 bits on the CPU, given the
experts that its router chose.

Tolerances are relative errors of whole matrices (Frobenius norm). Every
intermediate matrix is rounded to the 16-bit type once, by at most half a unit
in the last place, u = 2^-9 (bfloat16) or 2^-12 (float16) relative to each
element; the forward pass has seven such roundings on the way to y (n, logits, up,
inner, z, the sum, h) and the logits' moves the weights by about |logit| u, so
8 u; each gradient passes those and at most eight more of its own, 16 u.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

UNIT = {"bf16": 2.0 ** -9, "f16": 2.0 ** -12}
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def f64(t):
    return t.detach().double().cpu()


def written_out(block, x, residual, ids, up=None, n_rows=None):
    """(y, leaves) of the block in 64 bits, for the ids chosen."""
    leaves = [f64(t).requires_grad_() for t in (x, block.norm, block.router, block.up if up is None else up, block.down)]
    xx, norm, router, w_up, w_down = leaves
    h = xx + f64(residual)
    n = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * norm
    p = torch.softmax(n @ router, 1)
    rows = n if n_rows is None else n_rows
    y = h
    chosen = torch.gather(p, 1, ids.clamp_min(0).long())
    weights = chosen / (chosen.sum(1, keepdim=True) + 1e-20)
    for j in range(ids.shape[1]):
        out = []
        for t in range(x.shape[0]):
            e = int(ids[t, j])
            gate, value = (w_up[e] @ rows[t]).chunk(2)
            out.append(weights[t, j] * (w_down[e] @ (torch.nn.functional.silu(gate) * value)))
        y = y + torch.stack(out)
    return y, leaves


def error(got, want):
    want = want.detach().numpy()
    return np.linalg.norm(f64(got).numpy() - want) / np.linalg.norm(want)


def setup(dtype, tokens, hidden, inner, n, k):
    from dense_gemm_tensor_gb300 import moe
    block = moe.MoeBlock.random(hidden, inner, n, k, DT[dtype], seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    return (block, *(torch.randn(tokens, hidden, generator=g, device="cuda").to(DT[dtype]) for _ in range(3)))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,hidden,inner,n,k", [(1, 128, 64, 4, 2), (33, 136, 72, 5, 3), (150, 256, 128, 16, 2)])
def test_serving_pass(dtype, tokens, hidden, inner, n, k):
    block, x, residual, _ = setup(dtype, tokens, hidden, inner, n, k)
    y, saved = block.forward(x, residual)
    want, _ = written_out(block, x, residual, saved.routing.ids.cpu())
    assert error(y, want) < 8 * UNIT[dtype]
    assert error(block.serve(x, residual), want) < 8 * UNIT[dtype]


def test_serving_pass_8_bit():
    from dense_gemm_tensor_gb300 import experts
    block, x, residual, _ = setup("bf16", 40, 256, 128, 8, 2)
    block = block.quantize()
    n = experts.rms_norm(x, block.norm, residual)
    n8 = experts.rms_norm(n.h, block.norm, out_dtype=torch.float8_e4m3fn)
    rows = f64(n8.y.float()) * f64(n8.scale)[:, None]
    up = f64(block.up8.float()) * f64(block.up8_scale)[..., None]
    _, saved = block.forward(x, residual)
    want, _ = written_out(block, x, residual, saved.routing.ids.cpu(), up=up, n_rows=rows)
    assert error(block.serve(x, residual), want) < 8 * UNIT["bf16"]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,hidden,inner,n,k", [(5, 128, 64, 4, 2), (37, 136, 72, 5, 3), (150, 256, 128, 16, 2)])
def test_gradients(dtype, tokens, hidden, inner, n, k):
    block, x, residual, dy = setup(dtype, tokens, hidden, inner, n, k)
    _, saved = block.forward(x, residual)
    got = block.backward(dy, saved)
    want, leaves = written_out(block, x, residual, saved.routing.ids.cpu())
    want.backward(f64(dy))
    for g, leaf, name in zip(got, leaves, got._fields):
        assert error(g, leaf.grad) < 16 * UNIT[dtype], name


def test_step_in_a_graph():
    block, x, residual, dy = setup("bf16", 64, 256, 128, 8, 2)

    def step():
        y, saved = block.forward(x, residual)
        return (y, *block.backward(dy, saved))

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
