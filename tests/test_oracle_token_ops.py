"""CPU pins of the definitions in oracle/token_ops.py: hand values, gradients
against differences, 4-bit codes against their own grid."""
import numpy as np
import pytest

from oracle import token_ops as B


def test_rmsnorm_hand_row():
    o, v, rstd = B.rmsnorm([[1.0, 3.0]], [2.0, 1.0], 0.0, [[2.0, 1.0]])
    assert np.allclose(v, [[3, 4]]) and np.allclose(rstd, 1 / np.sqrt(12.5))
    assert np.allclose(o, np.array([[6.0, 4.0]]) / np.sqrt(12.5))


@pytest.mark.parametrize("n,d", [(1, 2), (3, 5), (4, 16)])
def test_rmsnorm_gradients_against_differences(n, d):
    g = np.random.default_rng(n * 100 + d)
    x, w, dy, dr = g.normal(size=(n, d)), g.normal(size=d), g.normal(size=(n, d)), g.normal(size=(n, d))
    dx, dw = B.rmsnorm_backward(dy, x, B.rmsnorm(x, w)[2], w, dr)
    h = 1e-6
    f = lambda x_, w_: (B.rmsnorm(x_, w_)[0] * dy).sum() + (x_ * dr).sum()
    for i in np.ndindex(n, d):
        e = np.zeros((n, d)); e[i] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[i]) < 1e-6
    for j in range(d):
        e = np.zeros(d); e[j] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[j]) < 1e-6


def test_tiles_of_a_short_row():
    o = np.array([[448.0] + [1.0] * 127 + [3.5, -7.0], [0.0] * 130])
    codes, scale = B.tiles(o)
    assert codes.shape == (2, 130) and scale.shape == (2, 2)
    assert scale[0, 0] == 1.0 and np.isclose(scale[0, 1], 7.0 / 448) and (scale[1] == 1).all()
    v = B.tile_values(codes, scale)
    assert v[0, 0] == 448 and v[0, 1] == 1 and np.allclose(v[0, 128:], [3.5, -7.0]) and not v[1].any()


def test_dispatch_by_hand():
    idx = np.array([[1, 0], [-1, 1], [7, 1], [1, 1]])
    off, perm, inv = B.dispatch(idx, 3)
    assert off.tolist() == [0, 1, 6, 6] and perm.tolist() == [0, 0, 1, 2, 3, 3, -1, -1]
    assert inv.tolist() == [[1, 0], [-1, 2], [-1, 3], [4, 5]]
    off, perm, inv = B.dispatch(idx, 3, rows=4)
    assert off.tolist() == [0, 1, 4, 4] and perm.tolist() == [0, 0, 1, 2]
    assert inv.tolist() == [[1, 0], [-1, 2], [-1, 3], [-1, -1]]


def test_return_gradients_against_differences():
    g = np.random.default_rng(5)
    _, _, inv = B.dispatch(np.array([[1, 0], [-1, 1], [2, 1]]), 2)
    rows, w, dy = g.normal(size=(6, 4)), g.normal(size=(3, 2)), g.normal(size=(3, 4))
    drows, dw = B.combine_backward(dy, rows, inv, w)
    f = lambda r_, w_: (B.combine(r_, inv, w_) * dy).sum()
    h = 1e-6
    for i in np.ndindex(rows.shape):
        e = np.zeros(rows.shape); e[i] = h
        want = 0.0 if np.isnan(drows[i]) else drows[i]
        assert abs((f(rows + e, w) - f(rows - e, w)) / (2 * h) - want) < 1e-6
    for i in np.ndindex(w.shape):
        e = np.zeros(w.shape); e[i] = h
        assert abs((f(rows, w + e) - f(rows, w - e)) / (2 * h) - dw[i]) < 1e-6
    assert np.isnan(drows[4:]).all() and dw[1, 0] == 0 and dw[2, 0] == 0


def test_mx4_halves_go_to_even_codes():
    """One block scaled to 1 (its largest value 4 .. 8): every half between codes."""
    v = np.zeros((1, 32))
    v[0, :17] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, -0.25, -0.75, -5.0, 0.26, 0.74,
                 4.99, 5.01, -0.0]
    codes, byte = B.mx4_encode(v)
    assert byte.tolist() == [[127]]
    assert codes[0, :17].tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 7, 8, 10, 14, 1, 1, 6, 7, 8]
    assert B.mx4_decode(codes, byte, 17)[0, 7:9].tolist() == [6.0, 6.0]


def test_mx4_scales_and_layout():
    v = np.zeros((2, 200))
    v[0, 0], v[0, 32], v[0, 64], v[1, 199] = 1.0, 2.0 ** -140, np.inf, -3e38
    codes, byte = B.mx4_encode(v)
    assert codes.shape == (2, 224) and byte.shape == (2, 7)
    assert byte[0].tolist() == [125, 0, 255, 0, 0, 0, 0] and byte[1, 6] == 127 + 127 - 2
    assert codes[0, 0] == 6 and not codes[0, 64:96].any()
    w = B.mx4_words(byte)
    assert w.shape == (2, 2, 4) and w[0, 0].tolist() == [125, 0, 255, 0]
    assert w[1, 1].tolist() == [0, 0, 252, 0]
    assert np.isnan(B.mx4_decode(codes, byte, 200)[0, 64:96]).all()
    assert (B.mx4_unpack(B.mx4_pack(codes)) == codes).all()


def test_mx4_keeps_every_value_of_its_grid():
    g = np.random.default_rng(1)
    codes = g.integers(0, 16, size=(5, 96)).astype(np.uint8)
    codes[:, ::32] = 7  # the largest magnitude, so that the scale is the same one again
    byte = g.integers(0, 250, size=(5, 3)).astype(np.uint8)
    again, b2 = B.mx4_encode(B.mx4_decode(codes, byte, 96))
    assert (again == codes).all() and (b2 == byte).all()
