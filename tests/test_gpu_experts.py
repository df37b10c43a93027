"""The mixture-of-experts operators on the GPU against the float64 oracle
(oracle/experts.py): every direction, type and layout at sizes and inputs where
they can go wrong.

Tolerances, per entry, with U = half an ulp of the output type at the reference:

* norm, combine and their gradients: U + 1e-5 * S, S the sum of the absolute
  values of the terms. fp32 sums here run over at most 32 values a thread and a
  tree over the threads, under 64 roundings of 2^-24 (4e-6), and a handful more
  come from the factors; 1e-5 covers both.
* 8-bit rows: q * scale is off by half a spacing of E4M3: 2^-4 of the value, or
  2^-10 * scale below the smallest normal number; plus the norm's own 1e-5.
* router: weights 2e-6 relative (a score is four or five fp32 operations and a
  sum of at most 1024 by halves), gradients 1e-5 * S; the choice is accepted
  when no expert left out, and none placed later, beats one by more than 1e-6
  (a rounding of a key below 2 is 1.2e-7); exact ties must go to the lowest index.
* products and their gradient: the acceptance rule of oracle/check.py, with S
  taken through the epilogue (GELU's Lipschitz constant 1.13, SiLU's 1.1).
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
    gemm.set_tuning(0, 0, 0, 0)
    assert gemm.device_status() == 0


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _normal(shape, dtype, seed, std=1.0):
    return (torch.randn(shape, generator=_gen(seed)) * std).to(DT[dtype] if isinstance(dtype, str) else dtype)


def _np(t):
    return t.detach().cpu().double().numpy()


def _pad(t, extra, fill=float("nan")):
    """A CUDA view of t whose rows sit `extra` elements apart further, the gaps holding `fill`."""
    full = torch.full((*t.shape[:-1], t.shape[-1] + extra), fill, dtype=t.dtype)
    full[..., :t.shape[-1]] = t
    return full.cuda()[..., :t.shape[-1]]


def _close(got, want, s, fmt, factor=1e-5):
    got, want = _np(got) if torch.is_tensor(got) else got, np.asarray(want)
    allowed = 0.5 * oracle.ulp(want, fmt) + factor * np.asarray(s)
    bad = ~(np.abs(got - want) <= allowed)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


# ---------------------------------------------------------------- norm

NORM_SHAPES = [(1, 1), (1, 7), (3, 64), (2, 1000), (5, 4096), (300, 264), (33, 5120), (4, 8200), (2, 16384), (700, 96), (3, 16383), (1500, 99), (9, 8191), (40, 1023)]


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_rms_norm(rows, cols, dtype, pad):
    x, r = _normal((rows, cols), dtype, 1), _normal((rows, cols), dtype, 2, 3.0)
    w = _normal((cols,), dtype, 3)
    h = (x.float() + r.float()).to(DT[dtype])
    want, rstd = ox.rms_norm(_np(h), _np(w), 1e-5)
    n = experts.rms_norm(_pad(x, pad), w.cuda(), _pad(r, pad), eps=1e-5)
    assert torch.equal(n.h.cpu(), h) and n.scale is None
    _close(n.y, want, np.abs(want), dtype)
    _close(n.rstd, rstd, rstd, "f32")
    # without a residual, h is x; eight-bit rows
    want, _ = ox.rms_norm(_np(x), _np(w), 1e-5)
    xc = _pad(x, pad)
    n = experts.rms_norm(xc, w.cuda(), eps=1e-5, out_dtype=torch.float8_e4m3fn)
    assert n.h is xc
    top = np.maximum(np.abs(want).max(axis=1), 1e-12) / 448
    assert np.all(np.abs(_np(n.scale) - top) <= 2e-5 * top)
    got = _np(n.y.float()) * _np(n.scale)[:, None]
    assert np.all(np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * top[:, None] + 2e-5 * np.abs(want))


def test_rms_norm_in_place_and_odd_rows():
    x, r, w = _normal((9, 512), "bf16", 4), _normal((9, 512), "bf16", 5), _normal((512,), "bf16", 6)
    h = (x.float() + r.float()).bfloat16()
    want, _ = ox.rms_norm(_np(h), _np(w), 1e-6)
    for into in (0, 1):
        xc, rc = x.cuda(), r.cuda()
        n = experts.rms_norm(xc, w.cuda(), rc, h_out=(xc, rc)[into])
        assert n.h is (xc, rc)[into] and torch.equal(n.h.cpu(), h)
        _close(n.y, want, np.abs(want), "bf16")
    # a row of zeros has norm zero; an infinity or NaN stays in its row
    x[1] = 0
    x[3, 5] = float("inf")
    x[4, 6] = float("nan")
    n = experts.rms_norm(x.cuda(), w.cuda())
    y = n.y.float().cpu()
    assert torch.all(y[1] == 0) and torch.isnan(y[4]).all() and torch.isnan(y[3, 5])
    keep = [0, 2, 5, 6, 7, 8]
    want, _ = ox.rms_norm(_np(x[keep]), _np(w), 1e-6)
    _close(n.y[keep], want, np.abs(want), "bf16")
    q = experts.rms_norm(x.cuda(), w.cuda(), out_dtype=torch.float8_e4m3fn)
    assert torch.isnan(q.scale[4]) and torch.all(q.y[1].float() == 0)
    assert np.all(np.abs(_np(q.scale[keep]) - np.abs(want).max(1) / 448) <= 2e-5 * _np(q.scale[keep]))
    assert experts.rms_norm(x[:0].cuda(), w.cuda()).y.shape == (0, 512)


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad,path", [(0, True), (1, False), (8, True)])
def test_rms_norm_backward(rows, cols, dtype, pad, path):
    h, dy = _normal((rows, cols), dtype, 7, 2.0), _normal((rows, cols), dtype, 8)
    w, dh = _normal((cols,), dtype, 9), _normal((rows, cols), dtype, 10)
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
    dx, dw = experts.rms_norm_backward(_pad(dy, pad), _pad(h, pad), w.cuda(), rstd.cuda(),
                                       dh=_pad(dh, pad) if path else None)
    want_x, want_w = ox.rms_norm_grad(_np(dy), _np(h), _np(w), _np(rstd), _np(dh) if path else None)
    g, xh, r = np.abs(_np(dy) * _np(w)), np.abs(_np(h) * _np(rstd)[:, None]), _np(rstd)[:, None]
    _close(dx, want_x, r * (g + xh * (g * xh).mean(1, keepdims=True)) + (np.abs(_np(dh)) if path else 0), dtype)
    _close(dw, want_w, (np.abs(_np(dy)) * xh).sum(0), dtype)


def test_rms_norm_backward_of_no_rows():
    z = torch.zeros(0, 64, device="cuda", dtype=torch.bfloat16)
    dx, dw = experts.rms_norm_backward(z, z, torch.ones(64, device="cuda", dtype=torch.bfloat16),
                                       torch.zeros(0, device="cuda"))
    assert dx.shape == (0, 64) and torch.all(dw == 0)


# ---------------------------------------------------------------- router

def _check_choice(r, logits, kind, bias, groups, kept, k, tie_gap=1e-6):
    ids = r.ids.cpu().numpy()
    key = ox.keys(logits, kind, bias, groups, kept)
    left = np.isfinite(key).sum(axis=1)
    assert np.array_equal((ids >= 0).sum(axis=1), np.minimum(left, k))
    for t in range(len(ids)):
        got = ids[t][ids[t] >= 0]
        assert len(set(got)) == len(got) and np.all(ids[t][len(got):] == -1)
        v = key[t][got]
        assert np.all(np.isfinite(v))
        assert np.all(v[1:] <= v[:-1] + tie_gap)
        rest = np.delete(key[t], got)
        if len(got) and len(rest):
            assert rest.max() <= v.min() + tie_gap
    return ids


def _check_order(r, ids, experts_n):
    slots, rows, offsets = ox.order(ids, experts_n)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.rows.cpu().numpy(), rows)
    assert np.array_equal(r.slots.cpu().numpy(), slots)


ROUTES = [(32, 1024, 32, 1, 1), (20000, 16, 3, 1, 1), (33, 256, 8, 4, 2), (1, 1, 1, 1, 1), (1, 8, 2, 1, 1), (5, 64, 8, 8, 3), (128, 100, 7, 1, 1), (129, 33, 3, 1, 1), (200, 256, 8, 8, 4),
          (700, 500, 20, 5, 2), (150, 1024, 32, 32, 5), (2000, 16, 2, 16, 5)]


@pytest.mark.parametrize("tokens,E,k,groups,kept", ROUTES)
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_route(tokens, E, k, groups, kept, kind, dtype):
    logits = _normal((tokens, E), dtype, tokens + E)
    if tokens > 2:
        logits[-1] = -float("inf")          # nothing left
        logits[1, 1:] = -float("inf")       # one expert left
        logits[2, ::2] = torch.finfo(logits.dtype).min  # the type's lowest value is an ordinary logit
    # a bias that is the same within a group, so that group keys of distinct groups stay apart
    bias = (torch.arange(E) // max(1, E // groups)).float() * 3 if groups > 1 else _normal((E,), "f32", 3, 0.1)
    r = experts.route(_pad(logits, 3), k, score=kind, bias=bias.cuda(), groups=groups, kept_groups=kept, scale=2.5)
    ids = _check_choice(r, _np(logits), kind, _np(bias), groups, kept, k, 1e-6 if groups == 1 else 1e-5)
    want = ox.route_weights(_np(logits), ids, kind, True, 2.5)
    assert np.all(np.abs(_np(r.weights) - want) <= 2e-6 * want + 1e-30)
    _check_order(r, ids, E)
    r = experts.route(logits.cuda(), min(k, E), score=kind, renormalize=False)
    ids = _check_choice(r, _np(logits), kind, None, 1, 1, k)
    want = ox.route_weights(_np(logits), ids, kind, False)
    assert np.all(np.abs(_np(r.weights) - want) <= 2e-6 * want + 1e-30)
    _check_order(r, ids, E)


@pytest.mark.parametrize("E", [8, 32, 40, 300])
def test_route_ties_go_to_the_lowest_index(E):
    # few distinct values, so that every token has exact ties inside and across lanes
    logits = torch.randint(0, 3, (300, E), generator=_gen(E)).float()
    for kind in ("softmax", "sigmoid"):
        r = experts.route(logits.cuda(), 6, score=kind)
        assert np.array_equal(r.ids.cpu().numpy(), ox.choose(ox.keys(_np(logits), kind), 6))
    flat = experts.route(torch.zeros(2, E, device="cuda"), 4, groups=4, kept_groups=2)
    assert flat.ids.tolist() == [[0, 1, 2, 3]] * 2 if E // 4 >= 2 else True


def test_route_not_a_number_and_infinity():
    logits = torch.zeros(4, 8)
    logits[1, 3] = float("nan")
    logits[2, 5] = float("inf")
    r = experts.route(logits.cuda(), 2, score="sigmoid")
    assert r.ids[0].tolist() == [0, 1] and r.ids[1].tolist() == [0, 1] and r.ids[2].tolist() == [5, 0]
    assert torch.isnan(r.weights[1]).all() and torch.isfinite(r.weights[[0, 2, 3]]).all()
    r = experts.route(logits.cuda(), 2)
    assert torch.isnan(r.weights[1:3]).all() and r.ids[1].tolist() == [-1, -1]
    assert r.ids[0].tolist() == [0, 1] and int(r.offsets[-1]) == 4


def test_route_of_no_tokens():
    r = experts.route(torch.zeros(0, 8, device="cuda"), 2)
    assert r.ids.shape == (0, 2) and r.offsets.tolist() == [0] * 9 and r.rows.numel() == 0


@pytest.mark.parametrize("tokens,E,k,groups,kept", ROUTES)
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype,renormalize", [("f32", True), ("f32", False), ("f16", True)])
def test_route_backward(tokens, E, k, groups, kept, kind, dtype, renormalize):
    logits = _normal((tokens, E), dtype, tokens)
    if tokens > 2:
        logits[-1] = -float("inf")
        logits[1, 1:] = -float("inf")
    dw = _normal((tokens, k), "f32", 11)
    ids = ox.choose(ox.keys(_np(logits), kind), k)
    got = experts.route_backward(dw.cuda(), _pad(logits, 5), torch.from_numpy(ids).int().cuda(), score=kind,
                                 renormalize=renormalize, scale=1.5)
    want = ox.route_grad(_np(dw), _np(logits), ids, kind, renormalize, 1.5)
    # terms: |dw| of each choice through 1 / (sum of scores), its mean, and the softmax's mean
    s = ox.scores(_np(logits), kind)
    c = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), 1), 0)
    d = 1.5 * np.abs(_np(dw))
    if renormalize:
        total = c.sum(1, keepdims=True) + 1e-20
        d = (d + (d * c).sum(1, keepdims=True) / total) / total
    full = np.zeros_like(s)
    np.add.at(full, (np.arange(tokens)[:, None], np.maximum(ids, 0)), np.where(ids >= 0, d, 0))
    scale = s * (full + (full * s).sum(1, keepdims=True))
    _close(got, want, scale, dtype)


# ---------------------------------------------------------------- products

def _routing(tokens, E, k, seed, empty=(), unused=0):
    """ids, and the oracle's order of them: `empty` experts get nothing, the last `unused` pairs of tokens none."""
    rng = np.random.default_rng(seed)
    open_ = [e for e in range(E) if e not in empty]
    ids = np.stack([rng.permutation(open_)[:k] for _ in range(tokens)]) if tokens else np.zeros((0, k), int)
    if unused:
        ids[-unused:] = -1
    return (ids, *ox.order(ids, E))


def _dev_order(rows, offsets):
    return torch.from_numpy(rows).int().cuda(), torch.from_numpy(offsets).int().cuda()


def _pitch16(t, extra=0):
    """A CUDA view with 16-byte rows: the pitch is rounded up (NaN in the gaps)."""
    per = 16 // t.element_size()
    full = -(-t.shape[-1] // per) * per + extra * per
    if t.dtype == torch.float8_e4m3fn:
        buf = torch.full((*t.shape[:-1], full), 0x7F, dtype=torch.uint8).view(t.dtype)
    else:
        buf = torch.full((*t.shape[:-1], full), float("nan"), dtype=t.dtype)
    buf[..., :t.shape[-1]] = t
    return buf.cuda()[..., :t.shape[-1]]


def _accept(got, ref, s, dtype):
    res = oracle.check(_np(got).reshape(-1, got.shape[-1]), ref.reshape(-1, ref.shape[-1]), s.reshape(-1, s.shape[-1]),
                       "bf16" if dtype == "e4m3" else dtype)
    assert res["ok"], res


# tokens, experts, k, K, N: one row; a few rows each; groups around the tile heights; large enough for pair tiles
PRODUCTS = [(1, 4, 2, 64, 64), (7, 6, 3, 200, 72), (70, 5, 2, 136, 264), (300, 3, 2, 520, 392), (130, 1, 1, 64, 520),
            (900, 4, 2, 96, 328), (260, 40, 4, 80, 136)]


@pytest.mark.parametrize("tokens,E,k,K,N", PRODUCTS)
@pytest.mark.parametrize("dtype,layout", [("bf16", 0), ("bf16", 1), ("f16", 0), ("f16", 1), ("e4m3", 1)])
@pytest.mark.parametrize("gather", [True, False])
def test_expert_matmul(tokens, E, k, K, N, dtype, layout, gather):
    _, _, rows, offsets = _routing(tokens, E, k, 1, empty=(1,) if E > 3 else (), unused=tokens // 9)
    a = _normal((tokens if gather else tokens * k, K), dtype, 2)
    w = _normal((E, N, K) if layout else (E, K, N), dtype, 3)
    r, off = _dev_order(rows, offsets)
    buf = torch.full((tokens * k + 1, N + 3), 7.0, dtype=torch.bfloat16 if dtype == "e4m3" else DT[dtype], device="cuda")
    C = buf[:tokens * k, :N]
    experts.expert_matmul(_pitch16(a), _pitch16(w), off, r if gather else None, layout=layout, out=C)
    c, s = ox.grouped(_np(a.float()), _np(w.float()), offsets, rows if gather else None, layout)
    _accept(C, c, s, dtype)
    assert torch.all(C[offsets[-1]:] == 0)
    assert torch.all(buf[:, N:] == 7.0) and torch.all(buf[tokens * k:] == 7.0)


# few slots and a long contraction; all of them in one group, or spread; one slot is a matrix of one row
@pytest.mark.parametrize("slots", [1, 31, 32, 33])
@pytest.mark.parametrize("E", [1, 7])
@pytest.mark.parametrize("dtype,layout", [("bf16", 0), ("bf16", 1), ("f16", 0), ("f16", 1), ("e4m3", 1)])
@pytest.mark.parametrize("gather", [True, False])
def test_expert_matmul_of_few_slots(slots, E, dtype, layout, gather):
    K, N = 2056, 208  # (row-major halves start on 16 bytes)
    _, _, rows, offsets = _routing(slots, E, 1, 41)
    a, w = _normal((slots, K), dtype, 42), _normal((E, N, K) if layout else (E, K, N), dtype, 43)
    r, off = _dev_order(rows, offsets)
    args = (_pitch16(a), _pitch16(w), off, r if gather else None)
    c, s = ox.grouped(_np(a.float()), _np(w.float()), offsets, rows if gather else None, layout)
    _accept(experts.expert_matmul(*args, layout=layout), c, s, dtype)
    g, v = 1e-2 * c[:, :N // 2], 1e-2 * c[:, N // 2:]
    s, silu = 1e-2 * s, g / (1 + np.exp(-g))
    C = experts.expert_matmul(*args, layout=layout, alpha=1e-2, activation="silu_gated")
    _accept(C, silu * v, 1.1 * s[:, :N // 2] * (np.abs(v) + 1e-3 * s[:, N // 2:]) + np.abs(silu) * s[:, N // 2:], dtype)


def _epilogue(c, s, act, lip):
    return {"none": lambda x: x, "relu": oracle.relu, "gelu": oracle.gelu, "gelu_tanh": oracle.gelu_tanh}[act](c), s * lip


@pytest.mark.parametrize("tokens,E,k,K,N", [(9, 4, 2, 72, 80), (400, 3, 2, 136, 328)])
@pytest.mark.parametrize("dtype,layout", [("bf16", 0), ("f16", 1), ("e4m3", 1)])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh"])
def test_expert_matmul_epilogue(tokens, E, k, K, N, dtype, layout, act):
    _, _, rows, offsets = _routing(tokens, E, k, 5, empty=(0,), unused=1)
    a, w = _normal((tokens, K), dtype, 6), _normal((E, N, K) if layout else (E, K, N), dtype, 7, 0.3)
    out = "bf16" if dtype == "e4m3" else dtype
    bias = _normal((E, N), out, 8)
    rs, cs = torch.rand(tokens, generator=_gen(9)) + 0.5, torch.rand((E, N), generator=_gen(10)) + 0.5
    r, off = _dev_order(rows, offsets)
    C = experts.expert_matmul(_pitch16(a), _pitch16(w), off, r, layout=layout, alpha=0.75, a_scale=rs.cuda(),
                              w_scale=cs.cuda(), bias=bias.cuda(), activation=act)
    c, s = ox.grouped(_np(a.float()), _np(w.float()), offsets, rows, layout)
    n = offsets[-1]
    e = np.searchsorted(offsets, np.arange(n), side="right") - 1
    f = 0.75 * _np(rs)[rows[:n], None] * _np(cs)[e]
    c[:n], s[:n] = c[:n] * f + _np(bias)[e], s[:n] * f + np.abs(_np(bias)[e])
    want, s = _epilogue(c, s, act, 1.13 if act.startswith("gelu") else 1.0)
    want[n:] = 0
    _accept(C, want, s, dtype)


@pytest.mark.parametrize("tokens,E,k,K,F", [(1, 4, 2, 64, 40), (9, 5, 2, 200, 136), (400, 3, 2, 136, 200), (500, 2, 2, 64, 72)])
@pytest.mark.parametrize("dtype,layout", [("bf16", 0), ("bf16", 1), ("f16", 0), ("f16", 1), ("e4m3", 1)])
def test_expert_matmul_gated(tokens, E, k, K, F, dtype, layout):
    F -= 3 if layout else 0  # the halves' boundary is free in K-major weights
    _, _, rows, offsets = _routing(tokens, E, k, 11)
    a, w = _normal((tokens, K), dtype, 12), _normal((E, 2 * F, K) if layout else (E, K, 2 * F), dtype, 13, 0.2)
    bias = _normal((E, 2 * F), "bf16" if dtype == "e4m3" else dtype, 14)
    r, off = _dev_order(rows, offsets)
    C = experts.expert_matmul(_pitch16(a), _pitch16(w), off, r, layout=layout, bias=bias.cuda(), activation="silu_gated")
    c, s = ox.grouped(_np(a.float()), _np(w.float()), offsets, rows, layout)
    e = np.searchsorted(offsets, np.arange(len(rows)), side="right") - 1
    c, s = c + _np(bias)[e], s + np.abs(_np(bias)[e])
    g, v = c[:, :F], c[:, F:]
    silu = g / (1 + np.exp(-g))
    _accept(C, silu * v, 1.1 * s[:, :F] * (np.abs(v) + 1e-3 * s[:, F:]) + np.abs(silu) * s[:, F:], dtype)


@pytest.mark.parametrize("tokens,E,k,K,N", PRODUCTS + [(65, 1, 1, 256, 256), (64, 1, 1, 264, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("gather", [True, False])
def test_expert_weight_grad(tokens, E, k, K, N, dtype, layout, gather):
    _, _, rows, offsets = _routing(tokens, E, k, 21, empty=(2,) if E > 3 else (), unused=tokens // 9)
    a, dc = _normal((tokens if gather else tokens * k, K), dtype, 22), _normal((tokens * k, N), dtype, 23)
    dc[offsets[-1]:] = float("nan")  # rows of no group
    r, off = _dev_order(rows, offsets)
    shape = (E, N, K) if layout else (E, K, N)
    buf = torch.full((E, shape[1] + 1, shape[2] + 5), 7.0, dtype=DT[dtype], device="cuda")
    dw = buf[:, :shape[1], :shape[2]]
    experts.expert_weight_grad(_pitch16(a), _pitch16(dc), off, r if gather else None, layout=layout, out=dw)
    want, s = ox.grouped_wgrad(_np(a), np.nan_to_num(_np(dc)), offsets, rows if gather else None, layout)
    _accept(dw, want, s, dtype)
    assert torch.all(buf[:, shape[1]:] == 7.0) and torch.all(buf[:, :, shape[2]:] == 7.0)


def test_input_gradient_is_the_product_with_the_other_layout():
    _, slots, rows, offsets = _routing(90, 4, 2, 31)
    w, dc = _normal((4, 136, 200), "bf16", 32), _normal((180, 136), "bf16", 33)
    _, off = _dev_order(rows, offsets)
    ds = experts.expert_matmul(_pitch16(dc), w.cuda(), off, layout=0)
    c, s = ox.grouped(_np(dc), _np(w), offsets, None, 0)
    _accept(ds, c, s, "bf16")
    da = experts.combine(ds, torch.from_numpy(slots).int().cuda())
    y, ys = ox.combine(_np(ds), slots)
    _close(da, y, ys, "bf16")


@pytest.mark.parametrize("tokens", [6, 400])
def test_other_groups_do_not_leak(tokens):
    """NaN and infinity in one group's rows and weights leave the other groups' results as they were."""
    _, _, rows, offsets = _routing(tokens, 3, 1, 41)
    r, off = _dev_order(rows, offsets)
    a, w, dc = _normal((tokens, 72), "bf16", 42), _normal((3, 72, 80), "bf16", 43), _normal((tokens, 80), "bf16", 44)
    c0 = experts.expert_matmul(a.cuda(), w.cuda(), off, r)
    dw0 = experts.expert_weight_grad(a.cuda(), dc.cuda(), off, r)
    lo, hi = offsets[1], offsets[2]
    a[rows[lo:hi]] = float("inf")
    dc[lo:hi] = float("nan")
    w[1] = float("nan")
    c1 = experts.expert_matmul(a.cuda(), w.cuda(), off, r)
    dw1 = experts.expert_weight_grad(a.cuda(), dc.cuda(), off, r)
    keep = np.r_[0:lo, hi:tokens]
    assert torch.equal(c0[keep], c1[keep]) and torch.isnan(c1[lo:hi]).all()
    assert torch.equal(dw0[[0, 2]], dw1[[0, 2]]) and torch.isnan(dw1[1]).all()


def test_products_of_nothing():
    w = _normal((3, 16, 24), "bf16", 51).cuda()
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    a = _normal((5, 16), "bf16", 52).cuda()
    C = experts.expert_matmul(a, w, off)  # every group empty: all rows are past the last group
    assert C.shape == (5, 24) and torch.all(C == 0)
    assert experts.expert_matmul(a[:0], w, off).shape == (0, 24)
    dw = experts.expert_weight_grad(a, _normal((5, 24), "bf16", 53).cuda(), off)
    assert dw.shape == (3, 16, 24) and torch.all(dw == 0)
    dw = experts.expert_weight_grad(a[:0], torch.empty(0, 24, device="cuda", dtype=torch.bfloat16), off)
    assert torch.all(dw == 0)
    # K = 0: the epilogue of zero
    off = torch.tensor([0, 2, 2, 4], dtype=torch.int32, device="cuda")
    bias = _normal((3, 24), "bf16", 54).cuda()
    C = experts.expert_matmul(torch.empty(5, 0, device="cuda", dtype=torch.bfloat16),
                              torch.empty(3, 0, 24, device="cuda", dtype=torch.bfloat16), off, bias=bias, activation="relu")
    assert torch.equal(C, torch.cat([bias[[0, 0, 2, 2]].clamp(min=0), torch.zeros_like(bias[:1])]))


def test_wrong_numbers_stay_inside_the_buffers():
    """Offsets and rows outside their ranges are clamped: the guards around C are untouched and the good group is right."""
    a, w = _normal((8, 64), "bf16", 61).cuda(), _normal((3, 64, 64), "bf16", 62).cuda()
    off = torch.tensor([0, 4, 1 << 30, 1 << 30], dtype=torch.int32, device="cuda")
    rows = torch.tensor([0, 1, 2, 3, -7, 1 << 30, 99, 8], dtype=torch.int32, device="cuda")
    buf = torch.full((10, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    experts.expert_matmul(a, w, off, rows, out=buf[1:9])
    c, s = ox.grouped(_np(a[:4]), _np(w[:1]), [0, 4])
    _accept(buf[1:5], c, s, "bf16")
    assert torch.all(buf[0] == 7.0) and torch.all(buf[9] == 7.0)
    dw = experts.expert_weight_grad(a, a, off, rows)
    want, s = ox.grouped_wgrad(_np(a[:4]), _np(a[:4]), [0, 4])
    _accept(dw[:1], want, s, "bf16")


def test_long_outputs():
    """Element offsets past 2^31 (a C whose padded rows span 5 GB)."""
    slots, ld = 70001, 36864
    _, off = _dev_order(np.zeros(1, int), np.array([0, 30000, slots]))
    a, w = _normal((slots, 64), "bf16", 71).cuda(), _normal((2, 64, 72), "bf16", 72).cuda()
    buf = torch.zeros(slots * ld, dtype=torch.bfloat16, device="cuda").view(slots, ld)
    C = experts.expert_matmul(a, w, off, out=buf[:, :72])
    want = torch.cat([a[:30000].float() @ w[0].float(), a[30000:].float() @ w[1].float()])
    assert (C.float() - want).abs().max() <= 2 ** -8 * want.abs().max()
    assert torch.all(buf[-1, 72:] == 0)
    y = experts.combine(buf[:, :72], torch.tensor([[slots - 1, 5], [3, slots - 2]], dtype=torch.int32, device="cuda"))
    want = torch.stack([C[slots - 1].float() + C[5].float(), C[3].float() + C[slots - 2].float()])
    assert (y.float() - want).abs().max() <= 2 ** -8 * want.abs().max()


# ---------------------------------------------------------------- combine

@pytest.mark.parametrize("tokens,cols,k", [(1, 1, 1), (1, 64, 3), (5, 100, 8), (33, 1000, 9), (300, 2048, 2), (7, 4104, 32),
                                            (64, 24, 6), (40, 1001, 5), (9, 2051, 2), (3, 4099, 8), (100, 13, 4)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad", [0, 1])
def test_combine_and_backward(tokens, cols, k, dtype, pad):
    _combine_and_backward(tokens, cols, k, dtype, pad)


# enough tokens for a thread to take several pieces of each row, by the number of experts a token
@pytest.mark.parametrize("tokens,cols,k", [(1901, 2056, 1), (1901, 2056, 2), (1901, 2056, 3), (1901, 2056, 4), (471, 8200, 2),
                                            (4801, 264, 4)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_combine_and_backward_of_many_tokens(tokens, cols, k, dtype):
    _combine_and_backward(tokens, cols, k, dtype, 0)


def _combine_and_backward(tokens, cols, k, dtype, pad):
    E = max(k, 3)
    _, slots, rows, offsets = _routing(tokens, E, k, 81, unused=tokens // 4)
    z, w = _normal((tokens * k, cols), dtype, 82), torch.rand((tokens, k), generator=_gen(83))
    z[offsets[-1]:] = float("nan")  # rows of no pair
    res, dy = _normal((tokens, cols), dtype, 84), _normal((tokens, cols), dtype, 85)
    sl = torch.from_numpy(slots).int().cuda()
    y, s = ox.combine(np.nan_to_num(_np(z)), slots, _np(w), _np(res))
    _close(experts.combine(_pad(z, pad), sl, w.cuda(), residual=_pad(res, pad)), y, s, dtype)
    y, s = ox.combine(np.nan_to_num(_np(z)), slots)
    _close(experts.combine(_pad(z, pad), sl), y, s, dtype)
    off = torch.from_numpy(offsets).int().cuda()
    dz, dw = experts.combine_backward(_pad(dy, pad), _pad(z, pad), sl, w.cuda(), off)
    wz, ww = ox.combine_grad(_np(dy), np.nan_to_num(_np(z)), slots, _np(w))
    _close(dz, wz, np.abs(wz), dtype)
    _close(dw, ww, ox.combine_grad(np.abs(_np(dy)), np.abs(np.nan_to_num(_np(z))), slots)[1], "f32")
    assert torch.all(dz[offsets[-1]:] == 0)
    acc = res.clone().cuda()
    experts.combine(_pad(z, 0), sl, w.cuda(), residual=acc, out=acc)
    y, s = ox.combine(np.nan_to_num(_np(z)), slots, _np(w), _np(res))
    _close(acc, y, s, dtype)


def test_combine_keeps_a_lost_tokens_nan():
    z = torch.ones(2, 8, device="cuda", dtype=torch.bfloat16)
    slots = torch.tensor([[0, -1], [-1, -1], [1, 99]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 0.0], [float("nan")] * 2, [1.0, 1.0]], device="cuda")
    y = experts.combine(z, slots, w).float().cpu()
    assert torch.all(y[0] == 0.5) and torch.isnan(y[1]).all() and torch.all(y[2] == 1)


# ---------------------------------------------------------------- streams, graphs, repeatability

def _block(x, res, wn, router, w1, w2, **kw):
    n = experts.rms_norm(x, wn, res, **kw)
    logits = gemm.matmul(n.y, router, **kw)
    r = experts.route(logits, 2, **kw)
    c = experts.expert_matmul(n.y, w1, r.offsets, r.rows, layout=1, activation="silu_gated", **kw)
    z = experts.expert_matmul(c, w2, r.offsets, layout=1, **kw)
    return experts.combine(z, r.slots, r.weights, residual=n.h, **kw), r, z, c


def _block_inputs(tokens=200, H=128, E=8, F=136):
    return [t.cuda() for t in (_normal((tokens, H), "bf16", 91), _normal((tokens, H), "bf16", 92), _normal((H,), "bf16", 93),
                               _normal((H, E), "bf16", 94, 0.1), _normal((E, 2 * F, H), "bf16", 95, 0.1),
                               _normal((E, H, F), "bf16", 96, 0.1))]


def test_block_repeats_bit_for_bit_on_any_stream():
    args = _block_inputs()
    y0, r0, *_ = _block(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y1, r1, *_ = _block(*args, stream=side)
    with torch.cuda.stream(side):
        y2, *_ = _block(*args)
    torch.cuda.synchronize()
    assert torch.equal(y0, y1) and torch.equal(y0, y2) and torch.equal(r0.slots, r1.slots)


def test_block_in_a_cuda_graph():
    args = _block_inputs(40)
    y0, *_ = _block(*args)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, *_ = _block(*args)
    fresh = _normal((40, 128), "bf16", 97).cuda()
    args[0].copy_(fresh)
    want, *_ = _block(*args)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and not torch.equal(y, y0)


def test_a_stalled_product_reports_a_timeout():
    """A producer that loads nothing: the kernel gives up within its limit and says so in the status word."""
    a, w = _normal((300, 64), "bf16", 98).cuda(), _normal((2, 64, 64), "bf16", 99).cuda()
    off = torch.tensor([0, 130, 300], dtype=torch.int32, device="cuda")
    try:
        for call in (lambda: experts.expert_matmul(a, w, off), lambda: experts.expert_weight_grad(a, a, off)):
            gemm.set_debug(1, 50_000_000)
            call()
            assert gemm.device_status() & 0xF == 1
            gemm.set_debug(0, 0)
            gemm.reset_device_status()
    finally:
        gemm.set_debug(0, 0)
        gemm.reset_device_status()
    C = experts.expert_matmul(a, w, off)
    c, s = ox.grouped(_np(a), _np(w), [0, 130, 300])
    _accept(C, c, s, "bf16")


@pytest.mark.parametrize("tokens", [20, 300])
def test_gather_without_a_workspace(tokens):
    """The C call without a workspace gathers the rows on their way: the same bits."""
    _, _, rows, offsets = _routing(tokens, 2, 1, 111)
    r, off = _dev_order(rows, offsets)
    a, w = _normal((tokens, 72), "bf16", 112).cuda(), _normal((2, 80, 72), "bf16", 113).cuda()
    C = torch.empty(tokens, 80, dtype=torch.bfloat16, device="cuda")
    lib, s = experts._load(), torch.cuda.current_stream().cuda_stream
    assert lib.gemm_bf16_grouped(2, off.data_ptr(), tokens, 80, 72, a.data_ptr(), tokens, 72, r.data_ptr(), w.data_ptr(),
                                 72, 80 * 72, C.data_ptr(), 80, 1, None, None, 0, s) == gemm.GEMM_OK
    assert torch.equal(C, experts.expert_matmul(a, w, off, r, layout=1))


def test_refusals_on_the_device():
    a, w = _normal((8, 64), "bf16", 101).cuda(), _normal((2, 64, 64), "bf16", 102).cuda()
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    with pytest.raises(gemm.GemmError):
        experts.expert_matmul(a[:, 1:], w[:, 1:], off)  # rows off 16-byte boundaries
    with pytest.raises(ValueError):
        experts.expert_matmul(a, w[:, :32], off)
    with pytest.raises(TypeError):
        experts.expert_matmul(a, w, off.long())
    with pytest.raises(ValueError):
        experts.expert_matmul(a, w, off[:2])
    with pytest.raises(ValueError):
        experts.expert_matmul(a.t(), w[:, :8], off)
    with pytest.raises(gemm.GemmError):
        experts.expert_matmul(a.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn), off)  # row-major 8-bit weights
    with pytest.raises(gemm.GemmError):
        experts.route(torch.zeros(2, 8, device="cuda"), 9)
    with pytest.raises(ValueError):
        experts.route(torch.zeros(2, 8, device="cuda"), 2, score="tanh")
    with pytest.raises(TypeError):
        experts.rms_norm(a, torch.ones(64, device="cuda"))
    with pytest.raises(ValueError):
        experts.rms_norm(a, torch.ones(63, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        experts.rms_norm(a, torch.ones(64, device="cuda", dtype=torch.bfloat16), out_dtype=torch.float16)
    with pytest.raises(ValueError):
        experts.combine(a, torch.zeros(8, dtype=torch.int32, device="cuda"))
    with pytest.raises(gemm.GemmError):
        experts.combine(a, torch.zeros(8, 33, dtype=torch.int32, device="cuda"))
    # host memory through the C call
    cfg = experts.RouteConfig(2, 0, 1, 1, 1, 1.0)
    host = torch.zeros(64)
    code = experts._load().gemm_route(2, 4, 8, host.data_ptr(), 8, None, cfg, off.data_ptr(), off.data_ptr(),
                                      off.data_ptr(), off.data_ptr(), off.data_ptr(), None, 0, None)
    assert code == gemm.GEMM_ERR_NOT_DEVICE_MEMORY
