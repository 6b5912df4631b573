"""Pins of the dense operators' fp64 oracle: closed forms, pure-Python loops
and central differences."""
import math

import numpy as np
import pytest

from oracle import dense_oracle as D


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def test_activation_values():
    z = np.array([-3.0, -1.0, -0.25, 0.0, 0.5, 2.0])
    for i, v in enumerate(z):
        sig = 1.0 / (1.0 + math.exp(-v))
        assert D.act(z, "silu")[i] == pytest.approx(v * sig, rel=1e-14, abs=1e-300)
        assert D.act(z, "gelu")[i] == pytest.approx(0.5 * v * (1 + math.erf(v / math.sqrt(2))), rel=1e-12, abs=1e-300)
        t = math.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
        assert D.act(z, "gelu_tanh")[i] == pytest.approx(0.5 * v * (1 + t), rel=1e-12, abs=1e-300)
        assert D.act(z, "relu")[i] == max(v, 0.0)
        assert D.act(z, "relu2")[i] == max(v, 0.0) ** 2
        assert D.act(z, "none")[i] == v


@pytest.mark.parametrize("name", D.ACTS)
def test_slope_is_the_difference_quotient(name):
    z = rng(1).standard_normal(200) * 2.0
    z = z[np.abs(z) > 1e-3]  # away from the kinks
    e = 1e-5
    num = (D.act(z + e, name) - D.act(z - e, name)) / (2 * e)
    # central difference: third derivative (below 3 here) times e^2 / 6, and rounding 1e-16 / e
    assert np.abs(num - D.act_slope(z, name)).max() < 1e-9


def test_kinks_have_slope_zero():
    assert D.act_slope(np.zeros(1), "relu")[0] == 0.0
    assert D.act_slope(np.zeros(1), "relu2")[0] == 0.0


def test_linear_by_loops():
    r = rng(2)
    x, w, b, res = (r.standard_normal(s) for s in ((3, 5), (4, 5), (4,), (3, 4)))
    out, pre = D.linear(x, w, b, res, "relu2")
    for t in range(3):
        for n in range(4):
            z = math.fsum(x[t, k] * w[n, k] for k in range(5)) + b[n]
            assert pre[t, n] == pytest.approx(z, rel=1e-12)
            assert out[t, n] == pytest.approx(max(z, 0.0) ** 2 + res[t, n], rel=1e-12)


def test_ffn_by_loops():
    r = rng(3)
    x, w13, w2, res = (r.standard_normal(s) for s in ((2, 3), (8, 3), (3, 4), (2, 3)))
    out, pre, h = D.ffn(x, w13, w2, "silu", res)
    for t in range(2):
        hs = []
        for f in range(4):
            g = math.fsum(x[t, k] * w13[f, k] for k in range(3))
            u = math.fsum(x[t, k] * w13[4 + f, k] for k in range(3))
            hs.append(g / (1 + math.exp(-g)) * u)
        for i in range(3):
            assert out[t, i] == pytest.approx(math.fsum(h_ * w2[i, f] for f, h_ in enumerate(hs)) + res[t, i], rel=1e-12)


def _numeric(f, a, e=1e-6):
    g = np.zeros_like(a)
    it = np.nditer(a, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        old = a[i]
        a[i] = old + e
        hi = f()
        a[i] = old - e
        lo = f()
        a[i] = old
        g[i] = (hi - lo) / (2 * e)
    return g


@pytest.mark.parametrize("name", D.ACTS)
def test_linear_gradients_by_differences(name):
    r = rng(4)
    x, w, b, dout = (r.standard_normal(s) for s in ((3, 4), (5, 4), (5,), (3, 5)))
    loss = lambda: float((D.linear(x, w, b, None, name)[0] * dout).sum())  # noqa: E731
    pre = D.linear(x, w, b, None, name)[1]
    dx, dw, db, _ = D.linear_backward(x, w, dout, name, pre)
    for a, g in ((x, dx), (w, dw), (b, db)):
        assert np.abs(_numeric(loss, a) - g).max() < 1e-7


@pytest.mark.parametrize("name", D.ACTS)
def test_ffn_gradients_by_differences(name):
    r = rng(5)
    x, w13, w2, dout = (r.standard_normal(s) for s in ((3, 4), (10, 4), (4, 5), (3, 4)))
    loss = lambda: float((D.ffn(x, w13, w2, name)[0] * dout).sum())  # noqa: E731
    pre = D.ffn(x, w13, w2, name)[1]
    dx, dw13, dw2, _, _ = D.ffn_backward(x, w13, w2, pre, dout, name)
    for a, g in ((x, dx), (w13, dw13), (w2, dw2)):
        assert np.abs(_numeric(loss, a) - g).max() < 1e-7


def test_clip():
    grads = [np.array([3.0, 0.0]), np.array([[4.0]]), np.zeros(0)]
    assert D.grad_norm(grads) == 5.0
    assert D.grad_norm(grads, "max") == 4.0
    n, out = D.clip(grads, 1.0)
    assert n == 5.0
    assert D.grad_norm(out) == pytest.approx(1.0, rel=1e-6)
    n, out = D.clip(grads, 100.0)
    assert all(np.array_equal(a, b) for a, b in zip(out, grads))
    n, out = D.clip([np.array([np.inf, 1.0])], 1.0)
    assert math.isinf(n) and out[0][1] == 1.0
