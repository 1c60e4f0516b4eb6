"""The float64 reference of the layer operators against closed forms and central differences."""

import numpy as np
import pytest

from oracle import layer as ol


@pytest.mark.parametrize("kind", ol.ACTS)
def test_activation_gradient_against_differences(kind):
    z = np.concatenate([np.linspace(-9, 9, 181) + 0.013, [-40.0, 40.0]])
    h = 1e-5
    diff = (ol.act(z + h, kind) - ol.act(z - h, kind)) / (2 * h)
    # central difference: h²/6·max|f'''| (below 3 here) and the rounding 2^-52·|f|/h
    assert np.all(np.abs(diff - ol.act_grad(z, kind)) <= 5e-10 + 2.0 ** -52 * (np.abs(z) + 1) / h * 2)


def test_activation_values():
    assert ol.act(np.array([0.0, 1.0, -1.0]), "gelu") == pytest.approx([0.0, 0.8413447460685429, -0.15865525393145707])
    assert ol.act(np.array([1.0]), "silu") == pytest.approx([0.7310585786300049])
    assert ol.act(np.array([-2.0, 3.0]), "relu").tolist() == [0.0, 3.0]
    z = np.linspace(-6, 6, 49)
    tanh_form = 0.5 * z * (1 + np.tanh(np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)))
    assert ol.act(z, "gelu_tanh") == pytest.approx(tanh_form, abs=1e-14)


@pytest.mark.parametrize("kind", ol.ACTS)
def test_product_gradients_against_differences(kind):
    rs = np.random.default_rng(3)
    A, B, bias = rs.normal(size=(3, 4)), rs.normal(size=(4, 5)), rs.normal(size=5)
    dY = rs.normal(size=(3, 5))

    def loss(A, B, bias):
        return float((dY * ol.product(A, B, kind, bias)[0]).sum())

    Z = ol.product(A, B, kind, bias)[1]
    dZ, _, dbias, _ = ol.act_backward(dY, Z, kind, "f32")
    h = 1e-6
    for x, grad in ((A, dZ @ B.T), (B, A.T @ dZ), (bias, dbias)):
        for i in np.ndindex(x.shape):
            keep = x[i]
            x[i] = keep + h
            up = loss(A, B, bias)
            x[i] = keep - h
            down = loss(A, B, bias)
            x[i] = keep
            assert abs((up - down) / (2 * h) - grad[i]) <= 1e-7 * (1 + abs(grad[i]))


def test_norm_gradients_against_differences():
    rs = np.random.default_rng(4)
    H, w, dY, dH = rs.normal(size=(3, 7)), rs.normal(size=7), rs.normal(size=(3, 7)), rs.normal(size=(3, 7))
    eps = 0.01

    def loss(H, w):
        return float((dY * ol.norm(H, w, eps)[0]).sum() + (dH * H).sum())

    dX, _, dw, _ = ol.norm_backward(dY, H, w, ol.norm(H, w, eps)[1], dH, "f32")
    h = 1e-6
    for x, grad in ((H, dX), (w, dw)):
        for i in np.ndindex(x.shape):
            keep = x[i]
            x[i] = keep + h
            up = loss(H, w)
            x[i] = keep - h
            down = loss(H, w)
            x[i] = keep
            assert abs((up - down) / (2 * h) - grad[i]) <= 1e-7 * (1 + abs(grad[i]))


@pytest.mark.parametrize("fmt", ("e4m3", "e5m2"))
def test_block_scale_is_the_smallest_power_that_fits(fmt):
    q = ol.QMAX[fmt]
    Y = np.zeros((1, 32 * 6))
    for b, top in enumerate((q, q * (1 + 2.0 ** -20), q / 2, 1.0, 0.0, q * 2.0 ** 30)):
        Y[0, 32 * b + 5] = -top
    e = ol.block_scale(Y, fmt)[0]
    assert e[:4].tolist() == [0, 1, -1, int(np.ceil(np.log2(1.0 / q)))] and e[5] == 30
    assert e[4] == int(np.ceil(np.log2(2.0 ** -100 / q)))
    tops = np.maximum(np.abs(Y).reshape(6, 32).max(axis=1), ol.AMAX_FLOOR)
    assert np.all(tops / 2.0 ** e <= q) and np.all(tops / 2.0 ** (e - 1.0) > q)
