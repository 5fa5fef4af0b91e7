"""Pins of oracle/model_steps.py to facts outside it: the serial scan, the conv
over sequences, closed forms, and gradients against differences."""
import numpy as np
import pytest
import torch

import oracle
from oracle import conv as oconv
from oracle import model_steps as om


@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("G", [1, 3])
def test_delta_steps_are_the_serial_scan(gate, G):
    """Three sequences' tokens in mixed order over a pool, with rows of no slot among them."""
    rng = np.random.default_rng(4)
    T, H, d, lengths = 12, 2, 8, [5, 0, 7]
    cu = np.cumsum([0] + lengths)

    def rn(*s):
        return rng.standard_normal(s).astype(np.float32)

    q, k, v, beta = rn(1, T, H * G, d), rn(1, T, H, d) / 3, rn(1, T, H, d), rng.random((1, T, H)).astype(np.float32)
    g = -rng.random((1, T, H) if gate == "gdn" else (1, T, H, d)).astype(np.float32)
    h0 = rng.standard_normal((3, H, d, d))
    o, ht = oracle.Problem(q, k, v, beta, g, cu_seqlens=cu, scale=0.5).scan(h0=h0)
    slot_of = [6, 1, 3]
    order = [0, 5, 6, 1, 2, 7, 8, 3, 9, 10, 4, 11]      # tokens of both sequences, each in its own order
    slots = [slot_of[0 if t < 5 else 2] for t in order]
    rows = lambda a: np.insert(a[0][order], 3, 7.0, axis=0)   # noqa: E731
    pool = rng.standard_normal((8, H, d, d))
    pool[slot_of] = h0
    r = om.delta_steps(rows(q), rows(k), rows(v), rows(beta), rows(g), pool, slots[:3] + [-1] + slots[3:], 0.5)
    assert np.isnan(r["o"][3]).all()
    np.testing.assert_allclose(np.delete(r["o"], 3, 0), o[0][order], rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(r["state"][slot_of], ht, rtol=1e-12, atol=1e-13)
    others = [0, 2, 4, 5, 7]
    np.testing.assert_array_equal(r["state"][others], pool[others])


@pytest.mark.parametrize("W", [1, 2, 4, 8])
def test_conv_steps_are_the_conv_over_the_sequence(W):
    rng = np.random.default_rng(5)
    x, w, b = rng.standard_normal((1, 11, 3)), rng.standard_normal((3, W)), rng.standard_normal(3)
    want = oconv.causal_conv1d(x, w, b)[0]
    r = om.conv_steps(x[0], w, b, np.zeros((2, W - 1, 3)), [1] * 11)
    np.testing.assert_allclose(r["y"], want, rtol=1e-12)
    np.testing.assert_array_equal(r["state"][1], x[0, 11 - (W - 1):])
    np.testing.assert_array_equal(r["state"][0], 0)


def test_layernorm_is_torchs():
    gen = torch.Generator().manual_seed(6)
    x, r, dy, dsum = (torch.randn((5, 24), generator=gen, dtype=torch.float64) for _ in range(4))
    w, b = (torch.randn(24, generator=gen, dtype=torch.float64).requires_grad_() for _ in range(2))
    s = (x + r).requires_grad_()
    y = torch.nn.functional.layer_norm(s, (24,), w, b, 1e-5)
    ((y * dy).sum() + (s * dsum).sum()).backward()
    f = om.layernorm_forward(x, w, b, 1e-5, r)
    np.testing.assert_allclose(f["y"], y.detach().numpy(), rtol=1e-11)
    g = om.layernorm_backward(s, w, 1e-5, dy, dsum)
    for name, ref in (("ds", s.grad), ("dweight", w.grad), ("dbias", b.grad)):
        np.testing.assert_allclose(g[name], ref.numpy(), rtol=1e-10, atol=1e-12)


def test_layernorm_gradients_equal_differences():
    rng = np.random.default_rng(7)
    s, dy, dsum = rng.standard_normal((3, 2, 16))
    w, b = rng.standard_normal((2, 16))
    g = om.layernorm_backward(s, w, 1e-5, dy, dsum)

    def loss(s, w, b):
        return (om.layernorm_forward(s, w, b, 1e-5)["y"] * dy).sum() + (s * dsum).sum()

    for at, grad, put in ((s, g["ds"], lambda t: (t, w, b)), (w, g["dweight"], lambda t: (s, t, b)),
                          (b, g["dbias"], lambda t: (s, w, t))):
        for i in rng.choice(at.size, 8, replace=False):
            d = np.zeros(at.size)
            d[i] = 1e-5
            d = d.reshape(at.shape)
            diff = (loss(*put(at + d)) - loss(*put(at - d))) / 2e-5
            np.testing.assert_allclose(grad.reshape(-1)[i], diff, rtol=1e-5, atol=1e-7)


def test_embed_gradient_equals_differences_of_the_lookup():
    rng = np.random.default_rng(8)
    tokens, dy, table = [4, 0, -1, 4, 9, 4], rng.standard_normal((6, 8)), rng.standard_normal((5, 8))
    g = om.embed_backward(tokens, dy, 5, 1.5)["dtable"]

    def loss(t):
        return sum((1.5 * t[k] * dy[i]).sum() for i, k in enumerate(tokens) if 0 <= k < 5)

    for i in range(table.size):
        d = np.zeros(table.size)
        d[i] = 1.0
        np.testing.assert_allclose(g.reshape(-1)[i], loss(table + d.reshape(table.shape)) - loss(table), atol=1e-12)
    assert (g[[1, 2, 3]] == 0).all()
