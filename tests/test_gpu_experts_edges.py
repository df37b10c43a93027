"""The mixture-of-experts operators on the GPU at the edges of what they take:
values near the ends of the types' ranges, several host threads, no tokens,
operands of any width. Each case against the float64 oracle (oracle/experts.py);
tolerances as in test_gpu_experts.py where none is given.
"""

import threading

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


def test_rms_norm_backward_from_several_threads():
    """The C call from host threads at once, each on its own stream, with widths that take different shared memory."""
    lib = experts._load()
    widths = [4096, 8192, 6144, 2731]
    cases, errors = [], []
    for i, cols in enumerate(widths):
        t = [_normal((64, cols), "bf16", 10 * i + j).cuda() for j in range(3)]
        w = _normal((cols,), "bf16", 10 * i + 4).cuda()
        rstd = torch.rsqrt(t[1].float().square().mean(1) + 1e-6)
        cases.append((cols, *t, w, rstd, experts.rms_norm_backward(t[0], t[1], w, rstd, dh=t[2])))
    torch.cuda.synchronize()

    def work(case):
        cols, dy, h, dh, w, rstd, want = case
        try:
            torch.cuda.set_device(0)
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                dx, dw = torch.empty_like(h), torch.empty_like(w)
                need = lib.gemm_rmsnorm_backward_workspace(64, cols)
                ws = torch.empty(need, dtype=torch.uint8, device="cuda")
                args = (1, 64, cols, dy.data_ptr(), cols, h.data_ptr(), cols, w.data_ptr(), rstd.data_ptr(), dh.data_ptr(),
                        cols, dx.data_ptr(), cols, dw.data_ptr(), ws.data_ptr(), need, s.cuda_stream)
                codes = [lib.gemm_rmsnorm_backward(*args) for _ in range(400)]
            s.synchronize()
            assert codes == [gemm.GEMM_OK] * len(codes), (cols, [c for c in codes if c][:3])
            assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    for _ in range(3):
        threads = [threading.Thread(target=work, args=(c,)) for c in cases]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    assert not errors, errors


def test_rms_norm_of_no_columns():
    """Every output is written: the mean of no elements is not a number, and the 8-bit scale has its least value."""
    x, w = torch.zeros(5, 0, device="cuda"), torch.zeros(0, device="cuda")
    torch.full((64,), 7.0, device="cuda")  # (what freed memory would show)
    n = experts.rms_norm(x, w, x)
    assert n.y.shape == n.h.shape == (5, 0) and torch.isnan(n.rstd).all()
    n = experts.rms_norm(x, w, out_dtype=torch.float8_e4m3fn)
    assert n.y.shape == (5, 0) and torch.isnan(n.rstd).all() and torch.all(n.scale == 1e-12 / 448)


# ---------------------------------------------------------------- no tokens

def test_combine_backward_of_no_tokens():
    z = torch.ones(4, 16, device="cuda", dtype=torch.bfloat16)
    slots, w = torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    dz, dw = experts.combine_backward(z[:0], z, slots, w, off)
    assert torch.all(dz == 0) and dw.shape == (0, 2) and dw.dtype == torch.float32
    dz, dw = experts.combine_backward(z[:0], z, slots, None, off)
    assert torch.all(dz == 0) and dw is None


def test_block_of_no_tokens():
    from dense_gemm_tensor_gb300 import moe
    block = moe.MoeBlock.random(128, 64, 4, 2, torch.bfloat16)
    x = torch.zeros(0, 128, device="cuda", dtype=torch.bfloat16)
    assert block.serve(x, x).shape == (0, 128)
    y, saved = block.forward(x, x)
    assert y.shape == (0, 128)
    grads = block.backward(y, saved)
    assert grads.x.shape == (0, 128)
    for g, p in zip(grads[1:], (block.norm, block.router, block.up, block.down)):
        assert g.shape == p.shape and torch.all(g == 0)


# ---------------------------------------------------------------- operands of any width

def _routing(tokens, E, k, seed, empty=(), unused=0):
    rng = np.random.default_rng(seed)
    open_ = [e for e in range(E) if e not in empty]
    ids = np.stack([rng.permutation(open_)[:k] for _ in range(tokens)])
    if unused:
        ids[-unused:] = -1
    return (ids, *ox.order(ids, E))


def _dev_order(rows, offsets):
    return torch.from_numpy(rows).int().cuda(), torch.from_numpy(offsets).int().cuda()


def _pitch16(t):
    """A CUDA view whose rows sit a multiple of 16 bytes apart (NaN in the gaps)."""
    per = 16 // t.element_size()
    full = -(-t.shape[-1] // per) * per
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


KINDS = [("bf16", 0), ("bf16", 1), ("f16", 0), ("f16", 1), ("e4m3", 1)]


@pytest.mark.parametrize("K,N", [(67, 1), (1, 67), (1, 1)])
@pytest.mark.parametrize("dtype,layout", KINDS)
def test_weights_of_one_row(K, N, dtype, layout):
    """The pitch of a weight matrix of one row says nothing; the matrices start 16-byte multiples apart."""
    _, _, rows, offsets = _routing(20, 3, 2, 1)
    a, w = _normal((20, K), dtype, 2), _normal((3, N, K) if layout else (3, K, N), dtype, 3)
    r, off = _dev_order(rows, offsets)
    C = experts.expert_matmul(_pitch16(a), _pitch16(w), off, r, layout=layout)
    c, s = ox.grouped(_np(a.float()), _np(w.float()), offsets, rows, layout)
    _accept(C, c, s, dtype)


# one token; a few rows a group; groups of more than a tile; pairs of tiles
SIZES = [(1, 4, 2, 67, 41), (23, 5, 2, 133, 90), (300, 3, 2, 515, 131), (700, 2, 1, 90, 333)]


@pytest.mark.parametrize("tokens,E,k,K,N", SIZES)
@pytest.mark.parametrize("dtype,layout", KINDS)
@pytest.mark.parametrize("gather", [True, False])
def test_contiguous_rows_of_any_width(tokens, E, k, K, N, dtype, layout, gather):
    _, _, rows, offsets = _routing(tokens, E, k, 1, empty=(1,) if E > 3 else (), unused=tokens // 9)
    n = tokens if gather else tokens * k
    a, w = _normal((n, K), dtype, 2), _normal((E, N, K) if layout else (E, K, N), dtype, 3)
    if dtype != "e4m3":  # a row that no slot takes touches its neighbours' memory only
        a[list(set(range(n)) - set(rows[:offsets[-1]] if gather else range(offsets[-1])))] = float("nan")
    r, off = _dev_order(rows, offsets)
    C = experts.expert_matmul(a.cuda(), _pitch16(w), off, r if gather else None, layout=layout)
    c, s = ox.grouped(_np(a.float()), _np(w.float()), offsets, rows if gather else None, layout)
    _accept(C, c, s, dtype)


@pytest.mark.parametrize("tokens,E,k,K,N", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("which", ["A", "dC", "both"])
def test_weight_gradient_of_contiguous_rows_of_any_width(tokens, E, k, K, N, dtype, layout, gather, which):
    _, _, rows, offsets = _routing(tokens, E, k, 21, empty=(2,) if E > 3 else (), unused=tokens // 9)
    a, dc = _normal((tokens if gather else tokens * k, K), dtype, 22), _normal((tokens * k, N), dtype, 23)
    dc[offsets[-1]:] = float("nan")  # rows of no group
    r, off = _dev_order(rows, offsets)
    dw = experts.expert_weight_grad(a.cuda() if which != "dC" else _pitch16(a), dc.cuda() if which != "A" else _pitch16(dc),
                                    off, r if gather else None, layout=layout)
    want, s = ox.grouped_wgrad(_np(a), np.nan_to_num(_np(dc)), offsets, rows if gather else None, layout)
    _accept(dw, want, s, dtype)


@pytest.mark.parametrize("tokens,E,k,K,N", SIZES)
@pytest.mark.parametrize("dtype,layout", KINDS)
@pytest.mark.parametrize("gather", [True, False])
def test_contiguous_weights_of_any_width(tokens, E, k, K, N, dtype, layout, gather):
    _, _, rows, offsets = _routing(tokens, E, k, 31, empty=(1,) if E > 3 else (), unused=tokens // 9)
    n = tokens if gather else tokens * k
    a, w = _normal((n, K), dtype, 32), _normal((E, N, K) if layout else (E, K, N), dtype, 33)
    if E > 3 and dtype != "e4m3":
        w[1] = float("nan")  # no row goes there
    r, off = _dev_order(rows, offsets)
    for rows_of_a in (a.cuda(), _pitch16(a)):
        C = experts.expert_matmul(rows_of_a, w.cuda(), off, r if gather else None, layout=layout)
        c, s = ox.grouped(_np(a.float()), np.nan_to_num(_np(w.float())), offsets, rows if gather else None, layout)
        _accept(C, c, s, dtype)


def test_rows_longer_than_two_gigabytes():
    """Sixteen named rows of 2^30 + 64 columns, put in slot order first."""
    K = (1 << 30) + 64
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("takes 40 GB")
    a, w = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((1, K), (1, 1, K)))
    at = torch.tensor([0, 5, (1 << 29) + 3, (1 << 30) - 1, 1 << 30, K - 1], device="cuda")
    a[0, at] = torch.tensor([1.0, 2, 4, 8, 16, 32], device="cuda").bfloat16()
    w[0, 0, at] = 1
    off = torch.tensor([0, 16], dtype=torch.int32, device="cuda")
    rows = torch.zeros(16, dtype=torch.int32, device="cuda")
    try:
        gemm.set_debug(0, 60_000_000_000)  # one CTA walks 16.8 million slabs, some seconds
        C = experts.expert_matmul(a, w, off, rows, layout=1)
        assert C.shape == (16, 1) and torch.all(C == 63)
    finally:
        gemm.set_debug(0, 0)


@pytest.mark.parametrize("tokens,E,k,K,F", [(1, 4, 2, 64, 37), (9, 5, 2, 200, 131), (400, 3, 2, 136, 197), (500, 2, 2, 67, 70)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("padded", [True, False])
def test_gated_row_major_halves_of_any_width(tokens, E, k, K, F, dtype, gather, padded):
    _, _, rows, offsets = _routing(tokens, E, k, 11, empty=(0,) if E > 3 else ())
    a, w = _normal((tokens if gather else tokens * k, K), dtype, 12), _normal((E, K, 2 * F), dtype, 13, 0.2)
    bias = _normal((E, 2 * F), dtype, 14)
    r, off = _dev_order(rows, offsets)
    C = experts.expert_matmul(_pitch16(a), _pitch16(w) if padded else w.cuda(), off, r if gather else None, layout=0,
                              bias=bias.cuda(), activation="silu_gated")
    c, s = ox.grouped(_np(a), _np(w), offsets, rows if gather else None, 0)
    e = np.searchsorted(offsets, np.arange(len(rows)), side="right") - 1
    c, s = c + _np(bias)[e], s + np.abs(_np(bias)[e])
    g, v = c[:, :F], c[:, F:]
    silu = g / (1 + np.exp(-g))
    _accept(C, silu * v, 1.1 * s[:, :F] * (np.abs(v) + 1e-3 * s[:, F:]) + np.abs(silu) * s[:, F:], dtype)


@pytest.mark.parametrize("hidden,inner", [(128, 100), (100, 72), (101, 33)])
def test_block_of_any_width(hidden, inner):
    """The operators take each other's outputs: the block against its own form with every width padded to whole pieces."""
    from dense_gemm_tensor_gb300 import moe
    block = moe.MoeBlock.random(hidden, inner, 4, 2, torch.bfloat16)
    x, residual, dy = (_normal((50, hidden), "bf16", 40 + i).cuda() for i in range(3))
    y, saved = block.forward(x, residual)
    served, grads = block.serve(x, residual), block.backward(dy, saved)
    assert block.quantize().serve(x, residual).shape == y.shape
    n = saved.norm
    ids, w = saved.routing.ids.long(), saved.routing.weights
    want = n.h.double()
    for j in range(2):
        gate, value = torch.einsum("tnh,th->tn", block.up.double()[ids[:, j]], n.y.double()).chunk(2, dim=1)
        z = torch.einsum("thf,tf->th", block.down.double()[ids[:, j]], torch.nn.functional.silu(gate) * value)
        want = want + w[:, j:j + 1].double() * z
    for got in (y, served):  # four roundings to bfloat16 on the way: up, inner, z, y
        assert (got.double() - want).norm() <= 4 * 2.0 ** -9 * want.norm()
    for g, p in zip(grads, (x, block.norm, block.router, block.up, block.down)):
        assert g.shape == p.shape and bool(torch.isfinite(g.float()).all())


# ---------------------------------------------------------------- numbers at the ends of their ranges

def test_numbers_that_do_not_fit_32_bits_are_refused():
    logits = torch.zeros(4, 8, device="cuda")
    with pytest.raises(ValueError):
        experts.route(logits, (1 << 32) + 2)
    with pytest.raises(ValueError):
        experts.route(logits, 2, groups=(1 << 32) + 1, kept_groups=(1 << 32) + 1)
    a, w = torch.zeros(4, 64, device="cuda").bfloat16(), torch.zeros(2, 64, 64, device="cuda").bfloat16()
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        experts.expert_matmul(a, w, off, layout=1 << 32)
    with pytest.raises(ValueError):
        experts.expert_weight_grad(a, a, off, layout=(1 << 32) + 1)


def test_routing_of_the_most_tokens():
    """tokens * k just below 2^31, whose last block of tokens ends past it."""
    tokens = (1 << 31) - 1
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("takes 60 GB")
    logits = torch.zeros(tokens, 1, dtype=torch.float16, device="cuda")
    logits[-1] = -float("inf")
    r = experts.route(logits, 1)
    assert r.offsets.tolist() == [0, tokens - 1]
    for lo in range(0, tokens, 1 << 28):
        hi = min(tokens, lo + (1 << 28))
        for got, last in ((r.slots[lo:hi, 0], -1), (r.rows[lo:hi], -1)):
            want = torch.arange(lo, hi, dtype=torch.int32, device="cuda")
            if hi == tokens:
                want[-1] = last
            assert torch.equal(got, want)
    assert int(r.ids[-1]) == -1 and not bool(r.ids[:-1].any()) and float(r.weights[-1]) == 0


# ---------------------------------------------------------------- activations over their range

@pytest.mark.parametrize("tokens", [182, 1500])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("act", ["silu_gated", "gelu_tanh"])
def test_activations_from_minus_90_to_90(tokens, dtype, act):
    """Pre-activations that the product gives exactly. The hardware's exponential of x is within 2 + 1.17 |x| units in the
    last place (2^-23), at most 1.3e-5 up to 88; GELU's argument adds |x| times four roundings (2^-24), 2.1e-5 there; the
    quotient's and the products' own are a few 2^-22: 4e-5 in all. Where the divisor passes 2^126 the quotient is 0:
    at most 91 * 2^-126 is lost."""
    F = 16
    v = torch.linspace(-90, 90, tokens).to(DT[dtype])
    a = torch.zeros(tokens, 8, dtype=DT[dtype])
    a[:, 0], a[:, 1] = v, 1
    w = torch.zeros(1, 2 * F if act == "silu_gated" else F, 8, dtype=DT[dtype])
    w[0, :F, 0] = 1
    w[0, F:, 1] = 1
    off = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    C = experts.expert_matmul(a.cuda(), w.cuda(), off, layout=1, activation=act)
    x = _np(v)
    t = x if act == "silu_gated" else 2 * np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3)
    with np.errstate(over="ignore"):
        want = np.repeat((x / (1 + np.exp(-t)))[:, None], F, axis=1)
    got = _np(C)
    allowed = 0.5 * oracle.ulp(want, dtype) + 4e-5 * np.abs(want) + 91 * 2.0 ** -126
    assert np.all(np.abs(got - want) <= allowed), np.argwhere(np.abs(got - want) > allowed)[:5]
