"""Pins of the layer-step oracle (oracle/layer_steps.py) to facts outside it:
closed forms, sequence independence, and gradients against differences."""
import numpy as np
import pytest

from oracle import layer_steps as ol


def test_glr_constant_gate_closed_form():
    """Impulse at the first token under a constant gate: h_t = a^t."""
    a, T = 0.75, 20
    x = np.zeros((1, T, 8))
    x[0, 0] = 1.0
    r = ol.glr_forward(x, np.full_like(x, np.log(a)))
    np.testing.assert_allclose(r["y"][0, :, 3], a ** np.arange(T), rtol=1e-13)
    np.testing.assert_allclose(r["hT"][0], a ** (T - 1), rtol=1e-13)


def test_glr_zero_gate_is_a_cumulative_sum_and_minus_infinity_resets():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((1, 9, 8))
    g = np.zeros_like(x)
    h0 = rng.standard_normal((1, 8))
    np.testing.assert_allclose(ol.glr_forward(x, g, h0)["y"][0], h0 + np.cumsum(x[0], 0), rtol=1e-12)
    g[0, 4] = -np.inf
    np.testing.assert_allclose(ol.glr_forward(x, g, h0)["y"][0, 4:], np.cumsum(x[0, 4:], 0), rtol=1e-12)


def test_glr_packed_sequences_are_independent():
    rng = np.random.default_rng(2)
    cu = np.cumsum([0, 5, 0, 1, 17])
    x, g = rng.standard_normal((1, 23, 8)), -np.abs(rng.standard_normal((1, 23, 8)))
    h0 = rng.standard_normal((4, 8))
    r = ol.glr_forward(x, g, h0, cu)
    for n in range(4):
        one = ol.glr_forward(x[:, cu[n]:cu[n + 1]], g[:, cu[n]:cu[n + 1]], h0[n:n + 1])
        np.testing.assert_array_equal(r["y"][:, cu[n]:cu[n + 1]], one["y"])
        np.testing.assert_array_equal(r["hT"][n], one["hT"][0])


def test_glr_gradients_equal_differences():
    rng = np.random.default_rng(3)
    cu = [0, 7, 7, 12]
    x, dy = rng.standard_normal((2, 1, 12, 8))
    g = -np.abs(rng.standard_normal((1, 12, 8)))
    h0, dhT = rng.standard_normal((2, 3, 8))
    r = ol.glr_backward(x, g, dy, h0, dhT, cu)

    def loss(x, g, h0):
        f = ol.glr_forward(x, g, h0, cu)
        return (f["y"] * dy).sum() + (f["hT"] * dhT).sum()

    for name, at, grad in (("x", x, r["dx"]), ("g", g, r["dg"]), ("h0", h0, r["dh0"])):
        for i in rng.choice(at.size, 12, replace=False):
            d = np.zeros(at.size)
            d[i] = 1e-5
            d = d.reshape(at.shape)
            args = {"x": x, "g": g, "h0": h0}
            hi, lo = dict(args), dict(args)
            hi[name], lo[name] = at + d, at - d
            num = (loss(**hi) - loss(**lo)) / 2e-5
            # central difference: truncation ~1e-10, cancellation ~1e-15 |loss| / 1e-5
            assert abs(num - grad.reshape(-1)[i]) <= 1e-7 * (1 + abs(num)), name


def test_rmsnorm_unit_rows_and_scale_invariance():
    x = np.array([[3.0, -3.0, 3.0, -3.0, 3.0, 3.0, 3.0, 3.0]])
    np.testing.assert_allclose(ol.rmsnorm_forward(x, np.ones(8), 0.0)["y"], np.sign(x), rtol=1e-14)
    rng = np.random.default_rng(4)
    x, w = rng.standard_normal((3, 16)), rng.standard_normal(16)
    np.testing.assert_allclose(ol.rmsnorm_forward(x, w, 0.0)["y"], ol.rmsnorm_forward(7 * x, w, 0.0)["y"], rtol=1e-12)
    np.testing.assert_allclose(ol.rmsnorm_forward(x - 1, w, 1e-6, residual=np.ones_like(x))["y"],
                               ol.rmsnorm_forward(x, w, 1e-6)["y"], rtol=1e-10)


@pytest.mark.parametrize("eps", [1e-6, 0.5])
def test_rmsnorm_gradients_equal_differences(eps):
    rng = np.random.default_rng(5)
    s, dy, dsum = rng.standard_normal((3, 4, 8))
    w = rng.standard_normal(8)
    r = ol.rmsnorm_backward(s, w, eps, dy, dsum)

    def loss(s, w):
        return (ol.rmsnorm_forward(s, w, eps)["y"] * dy).sum() + (s * dsum).sum()

    for i in range(s.size):
        d = np.zeros(s.size)
        d[i] = 1e-5
        d = d.reshape(s.shape)
        num = (loss(s + d, w) - loss(s - d, w)) / 2e-5
        assert abs(num - r["ds"].reshape(-1)[i]) <= 1e-7 * (1 + abs(num))
    for i in range(8):
        d = np.zeros(8)
        d[i] = 1e-5
        num = (loss(s, w + d) - loss(s, w - d)) / 2e-5
        assert abs(num - r["dweight"][i]) <= 1e-7 * (1 + abs(num))


def test_linear_is_the_sum_of_products():
    x = np.arange(6.0).reshape(2, 3)
    w = np.array([[1.0, 0, 0], [0, 2, 0], [1, 1, 1], [-1, 0, 1]])
    r = ol.linear_forward(x, w, bias=np.array([0.0, 1, 0, -1]), residual=np.ones((2, 4)),
                          x_scale=np.array([1.0, 2.0]), w_scale=np.array([1.0, 1, 10, 1]))
    np.testing.assert_allclose(r["y"], [[1, 4, 31, 2], [7, 18, 241, 4]])


def test_activations_closed_forms():
    z = np.array([0.0, 1.0, -1.0, 30.0, -30.0])
    np.testing.assert_allclose(ol.activation(z, "silu"), [0, 1 / (1 + np.exp(-1)), -1 / (1 + np.exp(1)), 30, -30 * np.exp(-30)],
                               rtol=1e-12)
    # Phi(1) = 0.8413447460685429
    np.testing.assert_allclose(ol.activation(z[:3], "gelu"), [0, 0.8413447460685429, -0.15865525393145707], rtol=1e-12)
    for act in ("silu", "gelu"):
        v = np.linspace(-6, 6, 41)
        num = (ol.activation(v + 1e-6, act) - ol.activation(v - 1e-6, act)) / 2e-6
        np.testing.assert_allclose(ol.activation_grad(v, act), num, atol=1e-8)
        assert np.abs(ol.activation_grad(v, act)).max() <= 1.13


@pytest.mark.parametrize("act", [None, "silu", "gelu"])
def test_linear_gradients_equal_differences(act):
    rng = np.random.default_rng(6)
    x, w, b, dy = (rng.standard_normal(s) for s in ((3, 5), (4, 5), (4,), (3, 4)))
    f = ol.linear_forward(x, w, bias=b, act=act)
    r = ol.linear_backward(x, w, dy, z=f["z"], act=act)

    def loss(x, w, b):
        return (ol.linear_forward(x, w, bias=b, act=act)["y"] * dy).sum()

    for name, at, grad in (("x", x, r["dx"]), ("w", w, r["dw"]), ("b", b, r["dbias"])):
        for i in range(at.size):
            d = np.zeros(at.size)
            d[i] = 1e-5
            d = d.reshape(at.shape)
            hi, lo = dict(x=x, w=w, b=b), dict(x=x, w=w, b=b)
            hi[name], lo[name] = at + d, at - d
            num = (loss(**hi) - loss(**lo)) / 2e-5
            assert abs(num - grad.reshape(-1)[i]) <= 1e-7 * (1 + abs(num)), name
