"""CPU fp64 oracle of the dense operators: linear layer, gated feed-forward
block, their gradients, and gradient clipping.

Plain numpy in float64, written from the formulas; nothing is rounded and no
code is shared with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

ACTS = ("none", "silu", "gelu", "gelu_tanh", "relu", "relu2")

_erf = np.vectorize(math.erf, otypes=[np.float64])
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def _sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def act(z: np.ndarray, name: str) -> np.ndarray:
    z = np.asarray(z, dtype=np.float64)
    if name == "none":
        return z
    if name == "silu":
        return z * _sigmoid(z)
    if name == "gelu":
        return 0.5 * z * _erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    p = np.maximum(z, 0.0)
    return p if name == "relu" else p * p


def act_slope(z: np.ndarray, name: str) -> np.ndarray:
    z = np.asarray(z, dtype=np.float64)
    if name == "none":
        return np.ones_like(z)
    if name == "silu":
        s = _sigmoid(z)
        return s + z * s * (1.0 - s)
    if name == "gelu":
        return 0.5 * _erfc(-z / math.sqrt(2.0)) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = np.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)
    if name == "relu":
        return (z > 0).astype(np.float64)
    return 2.0 * np.maximum(z, 0.0)


def linear(x, w, bias=None, residual=None, name="none"):
    """(out, pre): out = act(pre) + residual, pre = x w^T + bias."""
    pre = x @ w.T
    if bias is not None:
        pre = pre + bias
    out = act(pre, name)
    return (out if residual is None else out + residual), pre


def linear_backward(x, w, dout, name="none", pre=None, dx_residual=None):
    """(dx, dw, dbias, dz)."""
    dz = dout if name == "none" else dout * act_slope(pre, name)
    dx = dz @ w
    return (dx if dx_residual is None else dx + dx_residual), dz.T @ x, dz.sum(0), dz


def ffn(x, w13, w2, name="silu", residual=None):
    """(out, pre, h) of the gated block; w13 = [Wg; Wu]."""
    F = w2.shape[1]
    pre = x @ w13.T
    h = act(pre[:, :F], name) * pre[:, F:]
    out = h @ w2.T
    return (out if residual is None else out + residual), pre, h


def ffn_backward(x, w13, w2, pre, dout, name="silu", dx_residual=None):
    """(dx, dw13, dw2, da, h), da = [dg | du]."""
    F = w2.shape[1]
    g, u = pre[:, :F], pre[:, F:]
    a = act(g, name)
    dh = dout @ w2
    da = np.concatenate([dh * u * act_slope(g, name), dh * a], axis=1)
    dx = da @ w13
    return (dx if dx_residual is None else dx + dx_residual), da.T @ x, dout.T @ (a * u), da, a * u


def grad_norm(grads, norm_type="l2"):
    """Global norm; sums by math.fsum."""
    flat = [np.asarray(g, dtype=np.float64).ravel() for g in grads]
    if norm_type == "max":
        return max((float(np.abs(f).max()) for f in flat if f.size), default=0.0)
    return math.sqrt(math.fsum(float(np.dot(f, f)) for f in flat))


def clip(grads, max_norm, norm_type="l2"):
    """(norm, scaled gradients)."""
    n = grad_norm(grads, norm_type)
    c = min(1.0, max_norm / (n + 1e-6)) if math.isfinite(n) else 1.0
    return n, [np.asarray(g, dtype=np.float64) * c for g in grads]
