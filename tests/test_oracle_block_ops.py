"""CPU pins of the fp64 definitions in oracle/block_ops.py: hand values,
gradients against differences, singular values against the polynomial."""
import numpy as np
import pytest

from oracle import block_ops as B


def test_layernorm_hand_row():
    y, v, mean, rstd = B.layernorm([[1.0, 3.0]], [2.0, 1.0], [0.5, 0.0], eps=0.0,
                                   residual=[[1.0, 1.0]])
    assert np.allclose(v, [[2, 4]]) and mean[0] == 3.0 and rstd[0] == 1.0
    assert np.allclose(y, [[-1.5, 1.0]])


@pytest.mark.parametrize("n,d", [(1, 2), (3, 5), (4, 16)])
def test_layernorm_gradients_against_differences(n, d):
    g = np.random.default_rng(n * 100 + d)
    x, w, b, dy = g.normal(size=(n, d)), g.normal(size=d), g.normal(size=d), g.normal(size=(n, d))
    dr = g.normal(size=(n, d))
    _, _, mean, rstd = B.layernorm(x, w, b)
    dx, dw, db = B.layernorm_backward(dy, x, mean, rstd, w, dr)
    h = 1e-6
    f = lambda x_, w_, b_: (B.layernorm(x_, w_, b_)[0] * dy).sum() + (x_ * dr).sum()
    for i in np.ndindex(n, d):
        e = np.zeros((n, d)); e[i] = h
        assert abs((f(x + e, w, b) - f(x - e, w, b)) / (2 * h) - dx[i]) < 1e-6
    for j in range(d):
        e = np.zeros(d); e[j] = h
        assert abs((f(x, w + e, b) - f(x, w - e, b)) / (2 * h) - dw[j]) < 1e-6
        assert abs((f(x, w, b + e) - f(x, w, b - e)) / (2 * h) - db[j]) < 1e-6


def test_grouped_gradients_against_differences():
    g = np.random.default_rng(3)
    off = [0, 2, 2, 5]
    x, w, dy = g.normal(size=(5, 4)), g.normal(size=(3, 6, 4)), g.normal(size=(5, 6))
    f = lambda x_, w_: (B.grouped(x_, w_, off) * dy).sum()
    dx, dw = B.grouped_dgrad(dy, w, off), B.grouped_wgrad(dy, x, off)
    assert (dw[1] == 0).all()
    h = 1e-6
    for i in np.ndindex(*x.shape):
        e = np.zeros_like(x); e[i] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[i]) < 1e-6
    for i in np.ndindex(*w.shape):
        e = np.zeros_like(w); e[i] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[i]) < 1e-6


def test_grouped_rows_outside_the_groups():
    y = B.grouped(np.ones((4, 2)), np.ones((1, 3, 2)), [1, 3])
    assert np.isnan(y[[0, 3]]).all() and (y[1:3] == 2).all()


@pytest.mark.parametrize("rows,cols", [(5, 9), (9, 5), (6, 6)])
def test_orthogonalize_maps_singular_values(rows, cols):
    g = np.random.default_rng(rows).normal(size=(rows, cols))
    out, _ = B.orthogonalize(g, steps=3)
    u, s, vt = np.linalg.svd(g, full_matrices=False)
    s = s / (np.sqrt((g ** 2).sum()) + B.NS_EPS)
    a, b, c = B.NS_COEFFS
    for _ in range(3):
        s = a * s + b * s ** 3 + c * s ** 5
    assert np.allclose(out, (u * s) @ vt, atol=1e-12)


def test_momentum_forms():
    g, m = np.ones((2, 3)), np.full((2, 3), 2.0)
    _, new = B.orthogonalize(g, m, momentum=0.5)
    assert (new == 2.0).all()
    rng = np.random.default_rng(0)
    g, m = rng.normal(size=(3, 4)), rng.normal(size=(3, 4))
    nest, new = B.orthogonalize(g, m, 0.9, True)
    assert np.allclose(nest, B.orthogonalize(g + 0.9 * new)[0])
    assert np.allclose(B.orthogonalize(g, m, 0.9, False)[0], B.orthogonalize(new)[0])
