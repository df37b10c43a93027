"""The feed-forward operators on the GPU against the float64 oracle
(oracle/feedforward.py): every direction, type and layout at sizes and inputs
where they can go wrong.

Tolerances, per entry, with U = half an ulp of the output type at the reference:

* layer norm and its gradient: U + 1e-5 * S, S the sum of the absolute values of
  the terms. fp32 sums here run over at most 32 values a thread and a tree over
  the threads, under 64 roundings of 2^-24 (4e-6), and a handful more come from
  the factors; the mean's error, 1e-5 of mean |h|, is a term of every h - mean.
* 8-bit rows and blocks: q * scale is off by half a spacing of E4M3: 2^-4 of the
  value, or 2^-10 * scale below the smallest normal number. Blocks' scales are
  one division of an exact maximum, and q one multiplication by one reciprocal:
  both are compared for equality with the same fp32 steps.
* products: the acceptance rule of oracle/check.py (1e-3 S and an ulp), with S
  taken through the epilogue: c = act(g) v is off by (L s_g)(|v| + 1e-3 s_v) +
  |act(g)| s_v, L the activation's largest slope. The gradient's products
  take dup rounded to 16 bits, U of each of its entries: 2^-8 (2^-11) of sum
  |dup| |w| at most in place of nothing, beside dup's own fp32 error, 1e-4 of
  |dC v| and |dC act| (the hardware's exponential: 4e-5).
"""

import numpy as np
import pytest
import torch

import oracle
from dense_gemm_tensor_gb300 import feedforward as ff
from dense_gemm_tensor_gb300 import gemm
from oracle import feedforward as of

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
E4M3 = torch.float8_e4m3fn


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


def _pad(t, extra, fill=float("nan")):
    """A CUDA view of t whose rows sit `extra` elements apart further, the gaps holding `fill`."""
    full = torch.full((t.shape[0], t.shape[1] + extra), fill, dtype=torch.float32).to(t.dtype)
    full[:, :t.shape[1]] = t
    return full.cuda()[:, :t.shape[1]]


def _pitch16(t, more=0):
    """A CUDA view of t whose rows start on 16-byte boundaries; NaN between them."""
    per = 16 // t.element_size()
    return _pad(t, -t.shape[1] % per + per * more)


def _close(got, want, s, fmt, factor=1e-5):
    got, want = _np(got), np.asarray(want)
    allowed = 0.5 * oracle.ulp(want, fmt) + factor * np.asarray(s)
    bad = ~(np.abs(got - want) <= allowed)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


def _accept(C, want, s, dtype):
    r = oracle.check(_np(C), want, s, dtype)
    assert r["ok"], r


# ---------------------------------------------------------------- layer norm

NORM_SHAPES = [(1, 1), (1, 7), (3, 64), (2, 1000), (5, 4096), (300, 264), (33, 5120), (4, 8200), (2, 16384), (700, 96),
               (3, 16383), (1500, 99), (9, 8191), (40, 1023), (2, 6001), (3, 10999)]


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_layer_norm(rows, cols, dtype, pad):
    x, r = _normal((rows, cols), dtype, 1) + 1, _normal((rows, cols), dtype, 2, 3.0)
    w, b = _normal((cols,), dtype, 3), _normal((cols,), dtype, 4)
    h = (x.float() + r.float()).to(DT[dtype])
    want, mean, rstd = of.layer_norm(_np(h), _np(w), _np(b), 1e-3)
    n = ff.layer_norm(_pad(x, pad), w.cuda(), b.cuda(), _pad(r, pad), eps=1e-3)
    assert torch.equal(n.h.cpu(), h) and n.scale is None
    size = np.abs(_np(h)).mean(1)
    s = (np.abs(_np(h)) + size[:, None]) * rstd[:, None] * np.abs(_np(w)) + np.abs(_np(b))
    _close(n.y, want, s, dtype)
    _close(n.mean, mean, size, "f32")
    # the variance's error: relative, and the mean's error times the deviations, which sum to that error again
    _close(n.rstd, rstd, rstd * (1 + 1e-5 * size ** 2 * rstd ** 2), "f32")
    # without a residual h is x; without a bias; eight-bit rows
    want, mean, rstd = of.layer_norm(_np(x), _np(w), None, 1e-3)
    xc = _pad(x, pad)
    n = ff.layer_norm(xc, w.cuda(), eps=1e-3, out_dtype=E4M3)
    assert n.h is xc
    top = np.maximum(np.abs(want).max(axis=1), 1e-12) / 448
    off = 1e-5 * (np.abs(_np(x)) + np.abs(_np(x)).mean(1)[:, None]) * rstd[:, None] * np.abs(_np(w))
    assert np.all(np.abs(_np(n.scale) - top) <= 2e-7 * top + off.max(1) / 448)
    got = _np(n.y.float()) * _np(n.scale)[:, None]
    assert np.all(np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * top[:, None] + 2 * off)


def test_layer_norm_in_place_and_odd_rows():
    x, r, w = _normal((9, 512), "bf16", 4), _normal((9, 512), "bf16", 5), _normal((512,), "bf16", 6)
    h = (x.float() + r.float()).bfloat16()
    want, _, _ = of.layer_norm(_np(h), _np(w), None, 1e-5)
    for into in (0, 1):
        xc, rc = x.cuda(), r.cuda()
        n = ff.layer_norm(xc, w.cuda(), None, rc, h_out=(xc, rc)[into])
        assert n.h is (xc, rc)[into] and torch.equal(n.h.cpu(), h)
        _close(n.y, want, np.abs(want) + 1, "bf16")
    # a row of one value is its bias; an infinity or NaN stays in its row
    b = _normal((512,), "bf16", 7)
    x[1], x[2] = 0, 7.5
    x[3, 5] = float("inf")
    x[4, 6] = float("nan")
    n = ff.layer_norm(x.cuda(), w.cuda(), b.cuda())
    y = n.y.cpu()
    assert torch.equal(y[1], b) and torch.equal(y[2], b) and torch.isnan(y[4]).all() and torch.isnan(y[3]).all()
    keep = [0, 5, 6, 7, 8]
    want, _, _ = of.layer_norm(_np(x[keep]), _np(w), _np(b), 1e-5)
    _close(n.y[keep], want, 4 * (np.abs(_np(x[keep])) + 1) * np.abs(_np(w)) + np.abs(_np(b)), "bf16")
    q = ff.layer_norm(x.cuda(), w.cuda(), out_dtype=E4M3)
    assert torch.isnan(q.scale[4]) and torch.all(q.y[1].float() == 0)
    assert ff.layer_norm(x[:0].cuda(), w.cuda()).y.shape == (0, 512)
    empty = ff.layer_norm(x[:, :0].cuda(), w[:0].cuda(), out_dtype=E4M3)
    assert empty.y.shape == (9, 0) and torch.isnan(empty.mean).all() and torch.isnan(empty.rstd).all()


@pytest.mark.parametrize("cols", [264, 1023, 5120])
def test_layer_norm_of_rows_far_from_zero(cols):
    """Deviations of 1 about 4096, in fp32: mean(h^2) - mean(h)^2 would keep nothing of them."""
    h = (torch.randn((40, cols), generator=_gen(8)) + 4096).float()
    w = torch.ones(cols)
    want, mean, rstd = of.layer_norm(_np(h), _np(w), None, 1e-5)
    n = ff.layer_norm(h.cuda(), w.cuda())
    _close(n.mean, mean, np.abs(mean), "f32")
    # the mean is off by at most 1e-5 of 4096 (its sum's roundings), each deviation by that
    assert np.abs(_np(n.mean) - mean).max() <= 1e-5 * 4096
    assert np.abs(_np(n.y) - want).max() <= 1.1 * 1e-5 * 4096 + 1e-4
    assert np.abs(_np(n.rstd) / rstd - 1).max() <= (1e-5 * 4096) ** 2 + 1e-5


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad,path", [(0, True), (1, False), (8, True)])
def test_layer_norm_backward(rows, cols, dtype, pad, path):
    h, dy = _normal((rows, cols), dtype, 7, 2.0) + 1, _normal((rows, cols), dtype, 8)
    w, dh = _normal((cols,), dtype, 9), _normal((rows, cols), dtype, 10)
    mean = h.double().mean(1).float()
    rstd = torch.rsqrt((h.double() - mean.double()[:, None]).square().mean(1) + 1e-3).float()
    dx, dw, db = ff.layer_norm_backward(_pad(dy, pad), _pad(h, pad), w.cuda(), mean.cuda(), rstd.cuda(),
                                        dh=_pad(dh, pad) if path else None)
    want = of.layer_norm_grad(_np(dy), _np(h), _np(w), _np(mean), _np(rstd), _np(dh) if path else None)
    g, r = np.abs(_np(dy) * _np(w)), _np(rstd)[:, None]
    xh = np.abs(_np(h) - _np(mean)[:, None]) * r
    _close(dx, want[0], r * (g + g.mean(1, keepdims=True) + xh * (g * xh).mean(1, keepdims=True)) +
           (np.abs(_np(dh)) if path else 0), dtype)
    _close(dw, want[1], (np.abs(_np(dy)) * xh).sum(0), dtype)
    _close(db, want[2], np.abs(_np(dy)).sum(0), dtype)


@pytest.mark.parametrize("rows,cols", [(47, 1), (30, 2), (44, 3), (20, 7), (50, 33), (40, 1023), (9, 2050), (50, 40)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_layer_norm_rows_stay_apart(rows, cols, dtype, bad):
    """What a row holds, and what lies behind the matrix, reaches no other row: the others are the same bit for bit."""
    def behind(t):  # the same matrix with `bad` right behind it
        if t.dtype == torch.float32 and t.dim() == 1:
            return t.cuda()
        return torch.cat((t.flatten(), torch.full((64,), bad, dtype=t.dtype))).cuda()[:t.numel()].view(t.shape)

    ts = [_normal((rows, cols), dtype, 900 + i) for i in range(5)]
    w, b = _normal(cols, dtype, 906), _normal(cols, dtype, 907)

    def run(x, res, dy, dh, h, **kw):
        outs = []
        for q in (None, E4M3):
            n = ff.layer_norm(behind(x), behind(w), behind(b), behind(res), out_dtype=q)
            outs += [n.y.view(torch.uint8) if q else n.y, n.mean, n.rstd] + ([n.scale] if q else [])
        n = ff.layer_norm(behind(h), behind(w), behind(b))
        outs += [n.y]
        return outs + [ff.layer_norm_backward(behind(dy), behind(h), behind(w), n.mean, n.rstd, dh=behind(dh))[0]]

    want = run(*ts)
    assert not any(torch.isnan(t.float()).any() for t in want)
    at = rows // 2
    poisoned = [t.clone() for t in ts]
    for t in poisoned:
        t[at] = bad
    rest = [i for i in range(rows) if i != at]
    for got, ref in zip(run(*poisoned), want):
        assert torch.equal(got[rest].float(), ref[rest].float())


@pytest.mark.parametrize("cols", [40, 33, 1023])
def test_layer_norm_backward_of_huge_constant_rows(cols):
    """h - mean is 0 and rstd eps^-1/2: no step of any path may pass fp32's range."""
    h = torch.full((20, cols), 2.0 ** 123, dtype=torch.bfloat16, device="cuda")
    dy = _normal((20, cols), "bf16", 911).cuda()
    w = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    mean = torch.full((20,), 2.0 ** 123, device="cuda")
    rstd = torch.full((20,), 316.0, device="cuda")
    dx, dw, db = ff.layer_norm_backward(dy, h, w, mean, rstd)
    g = dy.double()
    want = 316.0 * (g - g.mean(1, keepdim=True))
    assert ((dx.double() - want).abs() <= want.abs() * 2.0 ** -8 + 316.0 * 1e-5 * (g.abs() + g.abs().mean(1, keepdim=True))).all()
    assert (dw == 0).all() and not torch.isnan(db.float()).any()


def test_layer_norm_backward_of_no_rows():
    z, v = torch.zeros(0, 64, device="cuda", dtype=torch.bfloat16), torch.zeros(0, device="cuda")
    dx, dw, db = ff.layer_norm_backward(z, z, torch.ones(64, device="cuda", dtype=torch.bfloat16), v, v)
    assert dx.shape == (0, 64) and torch.all(dw == 0) and torch.all(db == 0)


# ---------------------------------------------------------------- gated product

GATED = [(1, 64, 40), (9, 200, 136), (130, 136, 197), (300, 72, 333), (5, 8, 1), (128, 1000, 100), (257, 64, 64),
         (33, 1, 70), (64, 2048, 96), (17, 300, 520), (48, 513, 130)]


def _gated_case(M, K, F, dtype, layout, seed, more=0):
    a, w = _normal((M, K), dtype, seed), _normal((K, 2 * F), dtype, seed + 1, 1.5 * K ** -0.5)
    return a, w, _pitch16(a, more), _pitch16(w.t().contiguous() if layout else w, more)


def _gated_s(up, s, act):
    f = up.shape[1] // 2
    g, v = up[:, :f], up[:, f:]
    return of.LIPSCHITZ[act] * s[:, :f] * (np.abs(v) + 1e-3 * s[:, f:]) + np.abs(of.gate(g, act)[0]) * s[:, f:]


@pytest.mark.parametrize("M,K,F", GATED)
@pytest.mark.parametrize("dtype,layout", [("bf16", 0), ("bf16", 1), ("f16", 0), ("f16", 1)])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
def test_gated_matmul(M, K, F, dtype, layout, act):
    a, w, ad, wd = _gated_case(M, K, F, dtype, layout, 20, more=M % 2)
    bias = _normal((2 * F,), dtype, 22)
    want, up, s = of.gated(_np(a), _np(w), _np(bias), act)
    r = ff.gated_matmul(ad, wd, layout=layout, activation=act, bias=bias.cuda(), keep=True)
    _accept(r.c, want, _gated_s(up, s, act), dtype)
    _accept(r.up, up, s, dtype)
    want, up, s = of.gated(_np(a), _np(w), None, act)
    buf = torch.full((M + 1, F + 3), 7.0, dtype=DT[dtype], device="cuda")
    r = ff.gated_matmul(ad, wd, layout=layout, activation=act, out=buf[:M, :F])
    assert r.up is None and r.c.data_ptr() == buf.data_ptr()
    _accept(r.c, want, _gated_s(up, s, act), dtype)
    assert torch.all(buf[M:] == 7.0) and torch.all(buf[:, F:] == 7.0)


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("M", [3, 200])
def test_gated_matmul_of_any_pitch(layout, M):
    """Contiguous rows off 16-byte boundaries: both operands are copied first."""
    a, w, ad, wd = _gated_case(M, 77, 51, "bf16", layout, 30)
    one = ff.gated_matmul(ad, wd, layout=layout, keep=True)
    r = ff.gated_matmul(ad.contiguous(), wd.contiguous(), layout=layout, keep=True)
    assert torch.equal(r.c, one.c) and torch.equal(r.up, one.up)
    want, up, s = of.gated(_np(a), _np(w), None, "silu")
    _accept(r.c, want, _gated_s(up, s, "silu"), "bf16")
    dc = _normal((M, 51), "bf16", 33).cuda()
    for x, y in zip(ff.gated_matmul_backward(dc, ad, wd, one.up, layout=layout, bias=True),
                    ff.gated_matmul_backward(dc, ad.contiguous(), wd.contiguous(), one.up, layout=layout, bias=True)):
        assert torch.equal(x, y)


def test_gated_matmul_without_terms_or_rows():
    bias = _normal((24,), "bf16", 35)
    a, w = torch.zeros(5, 0, device="cuda", dtype=torch.bfloat16), torch.zeros(24, 0, device="cuda", dtype=torch.bfloat16)
    r = ff.gated_matmul(a, w, layout=1, bias=bias.cuda(), keep=True)
    want = of.gate(_np(bias[:12]), "silu")[0] * _np(bias[12:])
    _close(r.c, np.broadcast_to(want, (5, 12)), 5 * np.abs(want), "bf16")
    assert torch.equal(r.up.cpu(), bias.expand(5, 24))
    g = ff.gated_matmul_backward(r.c, a, w, r.up, layout=1, bias=True)
    dup = of.gated_grad(_np(r.c), _np(r.up), "silu").sum(0)
    assert g.dA.shape == (5, 0) and g.dW.shape == (24, 0)
    _close(g.dbias, dup, 10 * np.abs(dup), "bf16")
    # no rows
    x, w = torch.zeros(0, 16, device="cuda", dtype=torch.bfloat16), _normal((24, 16), "bf16", 36).cuda()
    r = ff.gated_matmul(x, w, layout=1, keep=True)
    assert r.c.shape == (0, 12) and r.up.shape == (0, 24)
    g = ff.gated_matmul_backward(r.c, x, w, r.up, layout=1, bias=True)
    assert g.dA.shape == (0, 16) and torch.all(g.dW == 0) and torch.all(g.dbias == 0)
    # no columns: the gradient of the rows is of no terms
    x = _normal((5, 16), "bf16", 37).cuda()
    r = ff.gated_matmul(x, w[:0], layout=1, keep=True)
    assert r.c.shape == (5, 0)
    assert torch.all(ff.gated_matmul_backward(r.c, x, w[:0], r.up, layout=1).dA == 0)


@pytest.mark.parametrize("M,K,F", GATED)
@pytest.mark.parametrize("dtype,layout", [("bf16", 0), ("bf16", 1), ("f16", 0), ("f16", 1)])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
def test_gated_matmul_backward(M, K, F, dtype, layout, act):
    a, w, ad, wd = _gated_case(M, K, F, dtype, layout, 40)
    up, dc = _normal((M, 2 * F), dtype, 42, 1.5), _normal((M, F), dtype, 43)
    up[0, 0] = 0.0
    r = ff.gated_matmul_backward(_pad(dc, M % 3), ad, wd, _pad(up, 2 * (F % 3)), layout=layout, activation=act, bias=True)
    dup = of.gated_grad(_np(dc), _np(up), act)
    # what dup may be off by: its rounding, and 1e-4 of the factors of its terms
    size = np.concatenate((np.abs(_np(dc) * _np(up[:, F:])), np.abs(_np(dc)) * np.abs(of.gate(_np(up[:, :F]), act)[0])), 1)
    off = HALF[dtype] * np.abs(dup) + 1e-4 * size + 2.0 ** -24
    for got, want, s, more in ((r.dA, dup @ _np(w).T, np.abs(dup) @ np.abs(_np(w)).T, off @ np.abs(_np(w)).T),
                               (r.dW.t() if layout else r.dW, _np(a).T @ dup, np.abs(_np(a)).T @ np.abs(dup),
                                np.abs(_np(a)).T @ off)):
        bad = ~(np.abs(_np(got) - want) <= oracle.allowed_error(want, s, dtype) + more)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3])
    want = dup.sum(0)
    assert np.all(np.abs(_np(r.dbias) - want) <= 0.5 * oracle.ulp(want, dtype) + 1e-4 * size.sum(0))
    # each output alone is the same
    alone = dict(dA=dict(weights=False), dW=dict(rows=False), dbias=dict(rows=False, weights=False, bias=True))
    for name, kw in alone.items():
        one = ff.gated_matmul_backward(_pad(dc, M % 3), ad, wd, _pad(up, 2 * (F % 3)), layout=layout, activation=act, **kw)
        assert torch.equal(getattr(one, name), getattr(r, name))
        assert all(v is None for k, v in one._asdict().items() if k != name)


def test_gated_gradient_of_extreme_gates():
    """Gates far out have slopes 0 and 1, whatever the exponential does there; a NaN stays in its entry."""
    up = torch.zeros(4, 16, dtype=torch.bfloat16)
    up[0, :8] = torch.tensor([-1e30, -100, -20, 20, 100, 1e30, float("inf"), float("nan")])
    up[:, 8:] = 1.0
    dc, a = torch.ones(4, 8, dtype=torch.bfloat16), torch.zeros(4, 8, dtype=torch.bfloat16)
    a[0] = 1.0
    w = torch.zeros(16, 8, dtype=torch.bfloat16)
    for act in ("silu", "gelu", "gelu_tanh", "relu"):
        # dW's row j is dup[0][j] (A has one row of ones)
        g = ff.gated_matmul_backward(dc.cuda(), a.cuda(), w.cuda(), up.cuda(), layout=1, activation=act)
        slope = _np(g.dW)[:8, 0]
        assert np.allclose(slope[:7], [0, 0, 0, 1, 1, 1, 1], atol=1e-6), (act, slope)
        assert np.isnan(slope[7])


# ---------------------------------------------------------------- 8-bit blocks

SIZES = [(1, 1), (1, 128), (3, 129), (130, 256), (5, 1000), (128, 127), (257, 300), (2, 16), (64, 4096), (300, 17)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tall", [1, 128])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_quantize_blocks(rows, cols, dtype, tall, transpose, pad):
    x = _normal((rows, cols), dtype, 50) * torch.exp(2 * torch.randn(cols, generator=_gen(51))).to(DT[dtype])
    x[0, :min(cols, 128)] = 0
    b = ff.quantize_blocks(_pad(x, pad), rows=tall, transpose=transpose)
    t = (x.t() if transpose else x).float()
    assert b.q.shape == t.shape and b.q.dtype == E4M3 and (b.q.stride(0) % 16 == 0 or t.shape[0] == 1)
    scale = torch.from_numpy(np.float32(np.maximum(of.block_scales(_np(t), tall) * 448, np.float32(1e-12)))) / 448
    assert torch.equal(b.scale.cpu(), scale)
    inv = torch.from_numpy(of.spread(_np(1.0 / scale), t.shape, tall)).float()
    assert torch.equal(b.q.cpu().float(), (t * inv).clamp(-448, 448).to(E4M3).float())
    err = np.abs(_np(b.q.float()) * of.spread(_np(b.scale), t.shape, tall) - _np(t))
    assert np.all(err <= 2.0 ** -4 * np.abs(_np(t)) * 1.001 + 2.0 ** -10 * of.spread(_np(scale), t.shape, tall))


def test_quantize_blocks_of_infinities_and_none():
    x = _normal((4, 300), "f32", 52)
    x[1, 130], x[2, 5] = float("nan"), float("inf")
    b = ff.quantize_blocks(x.cuda())
    s, q = b.scale.cpu(), b.q.float().cpu()
    assert torch.isnan(s[1, 1]) and torch.isnan(q[1, 128:256]).all() and torch.isinf(s[2, 0])
    assert torch.isnan(q[2, 5]) and torch.all(q[2, :5] == 0)
    ok = torch.ones(4, 3, dtype=torch.bool)
    ok[1, 1] = ok[2, 0] = False
    assert torch.isfinite(s[ok]).all() and torch.isfinite(q[0]).all()
    for shape in ((0, 300), (4, 0)):
        e = ff.quantize_blocks(torch.zeros(shape, device="cuda"))
        assert e.q.shape == shape and e.scale.shape == (shape[0], -(-shape[1] // 128))


BLOCKS = [(1, 1, 1), (1, 128, 128), (16, 130, 256), (17, 64, 300), (33, 200, 129), (64, 257, 1000), (65, 100, 127),
          (130, 300, 700), (300, 129, 2100), (7, 1000, 4096), (128, 128, 16), (1, 3, 8000), (400, 17, 384), (2, 40, 1150)]


def _operand(n, K, tall, seed, expand=False):
    x = torch.randn((n, K), generator=_gen(seed)) * torch.exp(torch.randn(K, generator=_gen(seed + 1)))
    scale = torch.from_numpy(of.block_scales(_np(x), tall)).float()
    q = (x / torch.from_numpy(of.spread(_np(scale), x.shape, tall)).float()).to(E4M3)
    return q, scale


@pytest.mark.parametrize("M,N,K", BLOCKS)
@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("columns", [True, False])
def test_matmul_blocks(M, N, K, b_rows, columns):
    a, sa = _operand(M, K, 1, 60)
    b, sb = _operand(N, K, b_rows, 62)
    want, s = of.matmul_blocks(_np(a.float()), _np(b.float()), _np(sa), _np(sb), b_rows)
    lay = (lambda t: t.cuda().t().contiguous().t()) if columns else (lambda t: t.cuda())
    buf = torch.full((M + 1, N + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    C = ff.matmul_blocks(_pitch16(a, M % 2), _pitch16(b, N % 2), lay(sa), lay(sb), out=buf[:M, :N])
    _accept(C, want, s, "bf16")
    assert torch.all(buf[M:] == 7.0) and torch.all(buf[:, N:] == 7.0)
    assert torch.equal(ff.matmul_blocks(_pitch16(a), _pitch16(b), sa.cuda(), sb.cuda()), C)


@pytest.mark.parametrize("M", [5, 300])
def test_matmul_blocks_with_a_scale_for_a_row(M):
    """Scales of stride 0, as the norm's 8-bit rows have them; columns past K and rows of the other operand do not count."""
    x, w = _normal((M, 640), "bf16", 70) + 1, _normal((640,), "bf16", 71)
    n = ff.layer_norm(x.cuda(), w.cuda(), out_dtype=E4M3)
    b, sb = _operand(200, 640, 128, 72)
    C = ff.matmul_blocks(n.y, b.cuda(), n.scale[:, None].expand(-1, 5), sb.cuda())
    want, s = of.matmul_blocks(_np(n.y.float()), _np(b.float()), np.repeat(_np(n.scale)[:, None], 5, 1), _np(sb), 128)
    _accept(C, want, s, "bf16")


def test_matmul_blocks_keeps_special_values_in_their_rows():
    a, sa = _operand(70, 300, 1, 74)
    b, sb = _operand(140, 300, 1, 76)
    plain = ff.matmul_blocks(_pitch16(a), _pitch16(b), sa.cuda(), sb.cuda())
    sa[3, 1], sb[139, 2] = float("nan"), float("inf")
    a.view(torch.uint8)[8, 299] = 0x7F  # NaN
    C = ff.matmul_blocks(_pitch16(a), _pitch16(b), sa.cuda(), sb.cuda())
    assert torch.isnan(C[3]).all() and torch.isnan(C[8]).all() and not torch.isfinite(C[:, 139]).any()
    rows = [i for i in range(70) if i not in (3, 8)]
    assert torch.equal(C[rows, :139], plain[rows, :139])


def test_matmul_blocks_of_no_terms():
    e = torch.zeros(5, 0, device="cuda").to(E4M3)
    f = torch.zeros(7, 0, device="cuda").to(E4M3)
    s = lambda n: torch.zeros(n, 0, device="cuda")  # noqa: E731
    out = torch.full((5, 9), 3.0, device="cuda", dtype=torch.bfloat16)
    C = ff.matmul_blocks(e, f, s(5), s(7), out=out[:, :7])
    assert torch.all(C == 0) and torch.all(out[:, 7:] == 3.0)
    assert ff.matmul_blocks(e[:0], f, s(0), s(1)).shape == (0, 7)


# ---------------------------------------------------------------- together

def _block(x, res, w, b, up, down, **kw):
    n = ff.layer_norm(x, w, b, res, **kw)
    g = ff.gated_matmul(n.y, up, layout=1, keep=True, **kw)
    y = gemm.matmul(g.c, down, layout=1, **kw)
    return y, n, g


def _block_backward(dy, n, g, w, up, down, **kw):
    """Gradients of the block and of h, whose other path (the next residual) brings dy too."""
    dc = gemm.matmul(dy, down, **kw)
    gg = ff.gated_matmul_backward(dc, n.y, up, g.up, layout=1, **kw)
    dx, dw, db = ff.layer_norm_backward(gg.dA, n.h, w, n.mean, n.rstd, dh=dy, **kw)
    return dx, dw, db, gg.dW


def _block_inputs(M=200, H=128, F=136):
    return [t.cuda() for t in (_normal((M, H), "bf16", 90), _normal((M, H), "bf16", 91), 1 + _normal((H,), "bf16", 92, 0.1),
                               _normal((H,), "bf16", 93, 0.1), _normal((2 * F, H), "bf16", 94, H ** -0.5),
                               _normal((H, F), "bf16", 95, F ** -0.5))]


def test_block_and_its_gradients():
    x, res, w, b, up, down = args = _block_inputs()
    y, n, g = _block(*args)
    dy = _normal(y.shape, "bf16", 96).cuda()
    got = _block_backward(dy, n, g, w, up, down)
    leaves = [t.double().requires_grad_() for t in (x, w, b, up, down)]
    x64, w64, b64, up64, down64 = leaves
    h = x64 + res.double()
    ny = torch.nn.functional.layer_norm(h, (h.shape[1],), w64, b64, 1e-5)
    gate, value = (ny @ up64.t()).chunk(2, dim=1)
    want = (torch.nn.functional.silu(gate) * value) @ down64.t()
    (want + h).backward(dy.double())
    # a chain of five or six roundings to bfloat16 (2^-9 in the mean) on either way
    assert (y.double() - want).norm() <= 8 * 2.0 ** -9 * want.norm()
    for t, leaf in zip(got, (x64, w64, b64, up64)):
        assert (t.double() - leaf.grad).norm() <= 16 * 2.0 ** -9 * leaf.grad.norm()


def test_eight_bit_product_and_its_gradients():
    """C = A W^T with both in blocks, and dA, dW as the same product on operands quantised along the other dimension."""
    a, w, dc = _normal((200, 300), "bf16", 100), _normal((260, 300), "bf16", 101, 0.1), _normal((200, 260), "bf16", 102)
    qa, qw = ff.quantize_blocks(a.cuda()), ff.quantize_blocks(w.cuda(), rows=128)
    C = ff.matmul_blocks(qa.q, qw.q, qa.scale, qw.scale)
    d, wt = ff.quantize_blocks(dc.cuda()), ff.quantize_blocks(w.cuda(), rows=128, transpose=True)
    dA = ff.matmul_blocks(d.q, wt.q, d.scale, wt.scale)
    dt, at = ff.quantize_blocks(dc.cuda(), transpose=True), ff.quantize_blocks(a.cuda(), transpose=True)
    dW = ff.matmul_blocks(dt.q, at.q, dt.scale, at.scale)
    for got, want, s in ((C, _np(a) @ _np(w).T, np.abs(_np(a)) @ np.abs(_np(w)).T),
                         (dA, _np(dc) @ _np(w), np.abs(_np(dc)) @ np.abs(_np(w))),
                         (dW, _np(dc).T @ _np(a), np.abs(_np(dc)).T @ np.abs(_np(a)))):
        # each operand is off by half a spacing of E4M3, 2^-4 of its value (or 2^-10 of its scale): both, and the product
        assert np.all(np.abs(_np(got) - want) <= (2 * 2.0 ** -4 + 2.0 ** -8 + 2.0 ** -8) * s + 2.0 ** -6 * s.mean())


@pytest.mark.parametrize("M", [16, 200])
def test_repeats_bit_for_bit_on_any_stream(M):
    args = _block_inputs(M)
    qa, qw = ff.quantize_blocks(args[0]), ff.quantize_blocks(args[4], rows=128)

    def everything(**kw):
        y, n, g = _block(*args, **kw)
        q = ff.quantize_blocks(args[0], **kw)
        c = ff.matmul_blocks(qa.q, qw.q, qa.scale, qw.scale, **kw)
        return (y, n.mean, *_block_backward(y, n, g, args[2], args[4], args[5], **kw), q.q.float(), c)

    first = everything()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = everything(stream=side)
    with torch.cuda.stream(side):
        third = everything()
    torch.cuda.synchronize()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_in_a_cuda_graph():
    args = _block_inputs(40)
    qw = ff.quantize_blocks(args[4], rows=128)

    def step():
        y, n, g = _block(*args)
        grads = _block_backward(y, n, g, args[2], args[4], args[5])
        q = ff.quantize_blocks(args[0])
        t = ff.quantize_blocks(args[0], transpose=True)
        return (y, *grads, ff.matmul_blocks(q.q, qw.q, q.scale, qw.scale), t.scale)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    args[0].copy_(_normal((40, 128), "bf16", 97))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in got]
    for a, b in zip(got, step()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("M,K,F", [(5, 100, 70), (70, 333, 65), (300, 200, 136), (600, 77, 201)])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_gated_rows_and_columns_stay_apart(M, K, F, layout, bad):
    a, w, ad, wd = _gated_case(M, K, F, "bf16", layout, 160)
    dc = _normal((M, F), "bf16", 163).cuda()

    def run(a, w, dc):
        r = ff.gated_matmul(a, w, layout=layout, keep=True)
        return r.c, r.up, ff.gated_matmul_backward(dc, a, w, r.up, layout=layout, weights=False).dA

    # (a clone drops the pitch, and another pitch may take another kernel, with another order of sums: both are clones)
    want = run(ad.clone(), wd, dc)
    at, rest = M // 2, [i for i in range(M) if i != M // 2]
    ad2, dc2 = ad.clone(), dc.clone()
    ad2[at] = bad
    dc2[at] = bad
    for got, ref in zip(run(ad2, wd, dc2), want):
        assert torch.equal(got[rest], ref[rest])
    col, others = F // 3, [j for j in range(F) if j != F // 3]
    wd2 = wd.clone()
    if layout:
        wd2[F + col] = bad
    else:
        wd2[:, F + col] = bad
    got, ref = (ff.gated_matmul(ad, t, layout=layout).c for t in (wd2, wd.clone()))
    assert torch.equal(got[:, others], ref[:, others])


def test_in_inference_mode():
    args = _block_inputs(40)
    y, n, g = _block(*args)
    q = ff.layer_norm(args[0], args[2], args[3], args[1], out_dtype=E4M3)
    with torch.inference_mode():
        y2, n2, g2 = _block(*args)
        q2 = ff.layer_norm(args[0], args[2], args[3], args[1], out_dtype=E4M3)
        blocks = ff.quantize_blocks(args[0])
        assert q2.scale.is_inference() and n2.mean.is_inference() and blocks.q.is_inference()
        doubled = (n2.mean * 2).cpu()
    assert torch.equal(y, y2) and torch.equal(g.c, g2.c)
    for a, b in ((n.mean, n2.mean), (n.rstd, n2.rstd), (q.mean, q2.mean), (q.rstd, q2.rstd), (q.scale, q2.scale)):
        assert a.is_contiguous() and torch.equal(a, b)
    assert torch.equal(doubled, n.mean.cpu() * 2)
    n.mean.zero_()  # the statistics share memory, and no element of it
    q.rstd.zero_()
    assert torch.equal(n.rstd, n2.rstd) and torch.equal(q.mean, q2.mean) and torch.equal(q.scale, q2.scale)


@pytest.mark.parametrize("rows,cols", [(0, 64), (3, 0), (0, 0)])
def test_layer_norm_of_nothing(rows, cols):
    x, w = torch.empty(rows, cols, device="cuda").bfloat16(), torch.empty(cols, device="cuda").bfloat16()
    for kw in ({}, {"out_dtype": E4M3}):
        n = ff.layer_norm(x, w, residual=x, **kw)
        assert n.y.shape == n.h.shape == x.shape and n.mean.shape == n.rstd.shape == (rows,)
        assert n.scale is None or n.scale.shape == (rows,)
        if cols == 0:
            assert torch.isnan(n.mean).all() and torch.isnan(n.rstd).all()
            assert n.scale is None or (n.scale == torch.tensor(1e-12 / 448, device="cuda")).all()
    dx, dw, db = ff.layer_norm_backward(x, x, w, n.mean, n.rstd)
    assert dx.shape == x.shape and not dw.any() and not db.any()


def test_a_stalled_product_reports_a_timeout():
    """A producer that loads nothing: the kernel gives up within its limit and says so in the status word."""
    a, w = _normal((300, 64), "bf16", 98).cuda(), _normal((128, 64), "bf16", 99).cuda()
    few, big = ff.quantize_blocks(_normal((9, 2048), "bf16", 98).cuda()), ff.quantize_blocks(_normal((300, 2048), "bf16", 99).cuda())
    calls = (lambda: ff.gated_matmul(a, w, layout=1), lambda: ff.gated_matmul(a[:9], w, layout=1),
             lambda: ff.matmul_blocks(few.q, big.q, few.scale, big.scale),
             lambda: ff.matmul_blocks(big.q, big.q, big.scale, big.scale))
    before = [c() for c in calls]
    try:
        for call in calls:
            gemm.set_debug(1, 50_000_000)
            call()
            assert gemm.device_status() & 0xF == 1
            gemm.set_debug(0, 0)
            gemm.reset_device_status()
    finally:
        gemm.set_debug(0, 0)
        gemm.reset_device_status()
    for call, want in zip(calls, before):
        got = call()
        assert torch.equal(got.c, want.c) if isinstance(got, ff.Gated) else torch.equal(got, want)


def test_refusals_on_the_device():
    a, w = _normal((8, 64), "bf16", 101).cuda(), _normal((128, 64), "bf16", 102).cuda()
    v, up = torch.ones(64, device="cuda", dtype=torch.bfloat16), torch.zeros(8, 128, device="cuda", dtype=torch.bfloat16)
    q = ff.quantize_blocks(a)
    one = torch.ones(8, device="cuda")
    for error, call in (
            (TypeError, lambda: ff.layer_norm(a, v.float())),
            (ValueError, lambda: ff.layer_norm(a, v[:63])),
            (ValueError, lambda: ff.layer_norm(a, v, v[:63])),
            (ValueError, lambda: ff.layer_norm(a, v, None, a[:7])),
            (ValueError, lambda: ff.layer_norm(a, v, h_out=a)),  # there is no residual
            (ValueError, lambda: ff.layer_norm(a.t(), v[:8])),
            (ValueError, lambda: ff.layer_norm_backward(a, a, v, one[:7], one)),
            (TypeError, lambda: ff.layer_norm_backward(None, a, v, one, one)),
            (gemm.GemmError, lambda: ff.gated_matmul(a[:, 1:], w[:, 1:].contiguous(), layout=1)),  # off a 16-byte boundary
            (ValueError, lambda: ff.gated_matmul(a, w)),
            (ValueError, lambda: ff.gated_matmul(a, w[:127], layout=1)),
            (ValueError, lambda: ff.gated_matmul(a, w, layout=1, bias=v)),
            (gemm.GemmError, lambda: ff.gated_matmul(a, a.t().contiguous(), layout=2)),
            (ValueError, lambda: ff.gated_matmul_backward(a, a, w, up[:7], layout=1)),
            (TypeError, lambda: ff.gated_matmul_backward(a, a, w, None, layout=1)),
            (TypeError, lambda: ff.matmul_blocks(a, q.q, q.scale, q.scale)),
            (ValueError, lambda: ff.matmul_blocks(q.q, q.q, q.scale[:7], q.scale)),
            (ValueError, lambda: ff.matmul_blocks(q.q, q.q, q.scale, q.scale[:2])),
            (ValueError, lambda: ff.matmul_blocks(q.q, q.q[:, :32], q.scale, q.scale)),
            (gemm.GemmError, lambda: ff.matmul_blocks(q.q[:, :20].contiguous(), q.q[:, :20].contiguous(), q.scale, q.scale)),
            (gemm.GemmError, lambda: ff.matmul_blocks(q.q, q.q, q.scale, q.scale, out=q.q.view(torch.bfloat16)[:, :8])),
            (ValueError, lambda: ff.quantize_blocks(a, rows=2)),
            (ValueError, lambda: ff.quantize_blocks(a.t()))):
        with pytest.raises(error):
            call()
    # host memory through the C call
    host = torch.zeros(64, dtype=torch.bfloat16)
    code = ff._load().gemm_quantize_blocks(1, 2, 32, host.data_ptr(), 32, 1, 0, q.q.data_ptr(), 32, one.data_ptr(), 1, 2, None)
    assert code == gemm.GEMM_ERR_NOT_DEVICE_MEMORY


# ---------------------------------------------------------------- at the edges

# slabs (or blocks) that clusters of one to eight CTAs share, and tiles that leave no room for a cluster
@pytest.mark.parametrize("slabs", [1, 2, 3, 4, 6, 8, 10, 12, 14, 16, 17])
@pytest.mark.parametrize("M", [3, 20, 40])
def test_few_rows_by_every_split(M, slabs):
    K, F = 64 * slabs - 5, 70
    a, w, ad, wd = _gated_case(M, K, F, "bf16", slabs % 2, 120)
    want, up, s = of.gated(_np(a), _np(w), None, "silu")
    r = ff.gated_matmul(ad, wd, layout=slabs % 2, keep=True)
    _accept(r.c, want, _gated_s(up, s, "silu"), "bf16")
    _accept(r.up, up, s, "bf16")
    K = 128 * slabs - 9
    a, sa = _operand(M, K, 1, 122)
    b, sb = _operand(150, K, 128 if slabs % 2 else 1, 124)
    want, s = of.matmul_blocks(_np(a.float()), _np(b.float()), _np(sa), _np(sb), 128 if slabs % 2 else 1)
    _accept(ff.matmul_blocks(_pitch16(a), _pitch16(b), sa.cuda(), sb.cuda()), want, s, "bf16")


@pytest.mark.parametrize("M,F", [(5, 10100), (40, 20000), (70, 9000), (150, 4200)])
def test_few_rows_of_many_tiles(M, F):
    """More tiles than SMs, and than twice as many; tiles along the rows too."""
    a, w, ad, wd = _gated_case(M, 136, F, "bf16", 1, 130)
    want, up, s = of.gated(_np(a), _np(w), None, "relu")
    _accept(ff.gated_matmul(ad, wd, layout=1, activation="relu").c, want, _gated_s(up, s, "relu"), "bf16")
    dc = _normal((M, F), "bf16", 132)
    up = _normal((M, 2 * F), "bf16", 133)
    dup = of.gated_grad(_np(dc), _np(up), "relu")  # products of 16-bit numbers: dup is rounded once
    got = ff.gated_matmul_backward(dc.cuda(), ad, wd, up.cuda(), layout=1, activation="relu", weights=False).dA
    bad = ~(np.abs(_np(got) - dup @ _np(w).T) <=
            oracle.allowed_error(dup @ _np(w).T, np.abs(dup) @ np.abs(_np(w)).T, "bf16") + HALF["bf16"] * np.abs(dup) @ np.abs(_np(w)).T)
    assert not bad.any()


# pairs of CTAs: a round of 256-wide tiles, of 128-wide ones, several rounds, ragged ends on both sides
@pytest.mark.parametrize("M,N,K", [(1000, 9000, 300), (2100, 2300, 520), (4100, 4000, 130), (515, 4001, 1027), (257, 9999, 129)])
@pytest.mark.parametrize("b_rows", [1, 128])
def test_matmul_blocks_of_many_rows(M, N, K, b_rows):
    a, sa = _operand(M, K, 1, 140)
    b, sb = _operand(N, K, b_rows, 142)
    want, s = of.matmul_blocks(_np(a.float()), _np(b.float()), _np(sa), _np(sb), b_rows)
    for extra in (0, 3):
        buf = torch.full((M + 1, N + extra), 7.0, dtype=torch.bfloat16, device="cuda")
        C = ff.matmul_blocks(_pitch16(a), _pitch16(b), sa.t().contiguous().cuda().t(), sb.cuda(), out=buf[:M, :N])
        _accept(C, want, s, "bf16")
        assert torch.all(buf[M:] == 7.0) and torch.all(buf[:, N:] == 7.0)


def test_offsets_past_32_bits():
    """Matrices of more than 2^31 elements: their last rows against the same rows alone (enough of them that both take
    the same kernel: those for few rows add up in another order)."""
    M, K, F, tail_rows = (1 << 31) // 1024 + 40, 16, 1024, 10000
    a = torch.randn((M, K), device="cuda").bfloat16()
    w = _normal((2 * F, K), "bf16", 150).cuda()
    one = ff.gated_matmul(a, w, layout=1, keep=True)
    few = ff.gated_matmul(a[-tail_rows:].contiguous(), w, layout=1, keep=True)
    assert torch.equal(one.c[-tail_rows:], few.c) and torch.equal(one.up[-tail_rows:], few.up)
    big = ff.gated_matmul_backward(one.c, a, w, one.up, layout=1, weights=False).dA
    small = ff.gated_matmul_backward(few.c, a[-tail_rows:].contiguous(), w, few.up, layout=1, weights=False).dA
    assert torch.equal(big[-tail_rows:], small)
    q, tail = ff.quantize_blocks(one.c), ff.quantize_blocks(few.c)
    assert torch.equal(q.q[-tail_rows:].view(torch.uint8), tail.q.view(torch.uint8)) and torch.equal(q.scale[-tail_rows:], tail.scale)
    t = ff.quantize_blocks(one.c, rows=128, transpose=True)
    first = one.c[M - M % 128 if M % 128 else M - 128:].float().abs()
    assert t.q.shape == (F, M)
    want = torch.from_numpy(of.block_scales(_np(first.t()), 128)).float()
    assert torch.allclose(t.scale[:, -1:].cpu(), want, rtol=1e-6)
    b = ff.quantize_blocks(_normal((64, F), "bf16", 151).cuda())
    c = ff.matmul_blocks(q.q, b.q, q.scale, b.scale)
    assert torch.equal(c[-tail_rows:], ff.matmul_blocks(tail.q, b.q, tail.scale, b.scale))
    del t, c
    n = ff.layer_norm(one.c, torch.ones(F, device="cuda").bfloat16())
    assert torch.equal(n.y[-tail_rows:], ff.layer_norm(few.c, torch.ones(F, device="cuda").bfloat16()).y)


def test_from_several_threads():
    """The calls from host threads at once, each on its own stream."""
    import threading
    cases, errors = [], []
    for i in range(4):
        args = _block_inputs(100 + 60 * i, 128 + 64 * i, 136 + 40 * i)
        qa, qw = ff.quantize_blocks(args[0]), ff.quantize_blocks(args[4], rows=128)
        y, n, g = _block(*args)
        grads = _block_backward(y, n, g, args[2], args[4], args[5])
        cases.append((args, qa, qw, y, grads, ff.matmul_blocks(qa.q, qw.q, qa.scale, qw.scale)))
    torch.cuda.synchronize()

    def work(args, qa, qw, y0, grads0, c0):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    y, n, g = _block(*args)
                    grads = _block_backward(y, n, g, args[2], args[4], args[5])
                    c = ff.matmul_blocks(qa.q, qw.q, qa.scale, qw.scale)
                    torch.cuda.current_stream().synchronize()
                    if not (torch.equal(y, y0) and torch.equal(c, c0) and all(torch.equal(a, b) for a, b in zip(grads, grads0))):
                        errors.append("another result")
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=c) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[:2]


def test_two_graphs_replayed_in_turn():
    """Graphs that hold the same calls on other inputs keep their own scratch."""
    graphs = []
    for seed in (0, 1):
        args = [t + seed for t in _block_inputs(70)]
        y, n, g = _block(*args)
        want = (y, *_block_backward(y, n, g, args[2], args[4], args[5]))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, n, g = _block(*args)
            got = (y, *_block_backward(y, n, g, args[2], args[4], args[5]))
        graphs.append((graph, got, want, args))
    for _ in range(3):
        for graph, _, _, _ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for _, got, want, _ in graphs:
        for a, b in zip(got, want):
            assert torch.equal(a, b)
