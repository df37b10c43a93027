"""The oracle of the mixture-of-experts operators (oracle/experts.py), pinned to
worked examples, and its gradients to central differences of its forward
definitions (the weights' sum against each logit, a norm's output against each
input, a product's sum against each weight)."""

import numpy as np
import pytest

from oracle import experts as ox


def _difference(f, x, h=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        g[i] = (f(up) - f(down)) / (2 * h)
    return g


def test_rms_norm_worked():
    # mean square of (3, 4) is 12.5; with eps 0 the norm divides by sqrt(12.5)
    y, r = ox.rms_norm([[3.0, 4.0]], [1.0, 2.0], 0.0)
    assert np.allclose(r, 1 / np.sqrt(12.5)) and np.allclose(y, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]])
    y, r = ox.rms_norm([[0.0, 0.0]], [1.0, 1.0], 0.25)
    assert r[0] == 2.0 and np.all(y == 0)


def test_rms_norm_gradient_by_differences():
    rng = np.random.default_rng(0)
    h, w, dy = rng.normal(size=(3, 5)), rng.normal(size=5), rng.normal(size=(3, 5))
    dx, dw = ox.rms_norm_grad(dy, h, w, ox.rms_norm(h, w, 1e-3)[1])
    assert np.allclose(dx, _difference(lambda x: (ox.rms_norm(x, w, 1e-3)[0] * dy).sum(), h), atol=1e-8)
    assert np.allclose(dw, _difference(lambda x: (ox.rms_norm(h, x, 1e-3)[0] * dy).sum(), w), atol=1e-8)


def test_choice_worked():
    l = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))
    assert np.allclose(ox.scores(l, "softmax"), [[1 / 8, 1 / 4, 1 / 2, 1 / 8]])
    assert ox.choose(ox.keys(l, "softmax"), 3).tolist() == [[2, 1, 0]]  # the tie goes to the lower index
    assert np.allclose(ox.route_weights(l, np.array([[2, 1]]), "softmax"), [[2 / 3, 1 / 3]])
    # groups {0, 1} and {2, 3}: sums 3/8 and 5/8
    assert ox.choose(ox.keys(l, "softmax", groups=2, kept=1), 2).tolist() == [[2, 3]]
    # a bias moves the choice and not the weights
    ids = ox.choose(ox.keys(l, "softmax", bias=[1, 0, 0, 0]), 1)
    assert ids.tolist() == [[0]] and ox.route_weights(l, ids, "softmax", renormalize=False)[0, 0] == pytest.approx(1 / 8)
    masked = np.array([[-np.inf, 0.0, -np.inf], [-np.inf] * 3])
    ids = ox.choose(ox.keys(masked, "softmax"), 2)
    assert ids.tolist() == [[1, -1], [-1, -1]]
    assert ox.route_weights(masked, ids, "softmax").tolist() == [[1.0, 0.0], [0.0, 0.0]]


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_by_differences(kind, renormalize):
    rng = np.random.default_rng(1)
    l, dw = rng.normal(size=(3, 6)), rng.normal(size=(3, 2))
    l[1, 2] = -np.inf
    ids = ox.choose(ox.keys(l, kind), 2)
    ids[2, 1] = -1
    f = lambda x: (ox.route_weights(x, ids, kind, renormalize, 1.5) * dw).sum()  # noqa: E731
    with np.errstate(invalid="ignore"):
        want = np.nan_to_num(_difference(f, l))
    assert np.allclose(ox.route_grad(dw, l, ids, kind, renormalize, 1.5), want, atol=1e-8)


def test_order_worked():
    slots, rows, offsets = ox.order(np.array([[1, 0], [-1, 1], [0, -1]]), 3)
    assert offsets.tolist() == [0, 2, 4, 4]
    assert rows.tolist() == [0, 2, 0, 1, -1, -1]
    assert slots.tolist() == [[2, 0], [-1, 3], [1, -1]]


@pytest.mark.parametrize("layout", [0, 1])
def test_grouped_and_its_gradients_by_differences(layout):
    rng = np.random.default_rng(2)
    a, rows, off = rng.normal(size=(3, 4)), np.array([0, 2, 2, 1, 0]), np.array([0, 2, 2, 4])  # the last slot is unused
    w = rng.normal(size=(3, 4, 3) if layout == 0 else (3, 3, 4))
    dc = rng.normal(size=(5, 3))
    dc[4] = 0
    c, s = ox.grouped(a, w, off, rows, layout)
    assert np.all(c[4] == 0) and np.all(s >= np.abs(c) - 1e-12)
    assert np.allclose(c[2], a[2] @ (w[2] if layout == 0 else w[2].T))
    dw, _ = ox.grouped_wgrad(a, dc, off, rows, layout)
    assert np.all(dw[1] == 0)
    assert np.allclose(dw, _difference(lambda x: (ox.grouped(a, x, off, rows, layout)[0] * dc).sum(), w), atol=1e-8)
    # the gradient of A: the product with the other layout flag, then the sum over a row's slots
    ds, _ = ox.grouped(dc, w, off, None, 1 - layout)
    da = np.zeros_like(a)
    np.add.at(da, rows, ds)
    assert np.allclose(da, _difference(lambda x: (ox.grouped(x, w, off, rows, layout)[0] * dc).sum(), a), atol=1e-8)


def test_combine_gradient_by_differences():
    rng = np.random.default_rng(3)
    z, w, slots, dy = rng.normal(size=(4, 3)), rng.normal(size=(2, 2)), np.array([[3, -1], [0, 2]]), rng.normal(size=(2, 3))
    y, s = ox.combine(z, slots, w, np.ones((2, 3)))
    assert np.allclose(y[0], 1 + w[0, 0] * z[3]) and np.all(s >= np.abs(y) - 1e-12)
    dz, dw = ox.combine_grad(dy, z, slots, w)
    assert np.allclose(dz, _difference(lambda x: (ox.combine(x, slots, w)[0] * dy).sum(), z), atol=1e-8)
    assert np.allclose(dw, _difference(lambda x: (ox.combine(z, slots, x)[0] * dy).sum(), w), atol=1e-8)
