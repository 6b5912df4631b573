"""Inputs and tolerances of the dense operators' GPU tests.

Tolerances, derived before any run.  u is half a step of the output type
relative to the value: 2^-8 for bf16, 2^-11 for fp16, and `tiny` half its
smallest subnormal.
  - A product's sum over n terms in fp32: each addition may lose 2^-23 of the
    running magnitude (the tensor core's adder may truncate), so it is off by
    at most n 2^-23 S with S = sum |terms|.
  - An activation moves an error e of its argument by at most its steepest
    slope times e: 1.13 for silu and the gelus, 1 for relu and none, and
    2 |z| + e for relu^2; evaluating it in fp32 with the approximate exp and
    reciprocal adds at most 2^-18 |value| plus 2^-20 |z| (the argument of exp,
    up to 88, is rounded to fp32: 88 * 2^-24 relative in exp; gelu's normal
    distribution is a polynomial good to 7.5e-8 < 2^-23).
  - A value rounded to the 16-bit type on its way into the next product is off
    by u |value|.
  - The output's rounding: u |value| + tiny.
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import dense_oracle as D

ADD = 2.0 ** -23
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def np64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def act_error(z, e, name):
    """Bound on |act_fp32(z') - act(z)| for |z' - z| <= e."""
    if name == "none":
        return e
    if name == "relu":
        return e
    if name == "relu2":
        return 2 * np.abs(z) * e + e * e + 2.0 ** -22 * D.act(z, name)
    return 1.13 * e + 2.0 ** -18 * np.abs(D.act(z, name)) + 2.0 ** -20 * np.abs(z)


def slope_error(z, name):
    """Bound on the fp32 evaluation of act'(z)."""
    if name in ("none", "relu"):
        return 0.0 * z
    if name == "relu2":
        return 2.0 ** -22 * np.abs(D.act_slope(z, name))
    # terms of size up to 1.13 and z s (1 - s) <= |z| / 4, each within 2^-18
    return 2.0 ** -18 * (1.13 + np.abs(z))


def round_error(v, dtype):
    return U[dtype] * np.abs(v) + TINY[dtype]


def check(got, ref, bound, label, dtype):
    """Every element within its bound, its own rounding included."""
    got = np64(got)
    assert got.shape == ref.shape, (label, got.shape, ref.shape)
    allowed = bound + round_error(np.abs(ref) + bound, dtype)
    bad = ~(np.abs(got - ref) <= allowed)
    assert not bad.any(), (f"{label}: {bad.sum()} of {bad.size} off, worst "
                           f"{np.nanmax(np.abs(got - ref) / allowed)} of the bound at {np.argwhere(bad)[:3].tolist()}")


def sums(a, b):
    """S = |a| |b|^T of a product a b^T."""
    return np.abs(a) @ np.abs(b).T


def linear_bounds(x, w, pre, name):
    e = x.shape[1] * ADD * sums(x, w) + 2.0 ** -23 * np.abs(pre)
    return act_error(pre, e, name), e


def product_bound(a, b_t, a_err):
    """Bound of the product a b_t^T whose operand a is off by a_err."""
    return a.shape[1] * ADD * sums(a, b_t) + sums(a_err, b_t) * (1 + a.shape[1] * ADD)


class Draw:
    """Seeded device tensors; rows `pad` elements apart in a buffer whose
    gaps hold NaN."""

    def __init__(self, seed, dtype, pad=0):
        self.gen = torch.Generator().manual_seed(seed)
        self.dtype, self.pad = dtype, pad

    def whole(self, shape, std=1.0):
        return (torch.randn(shape, generator=self.gen) * std).to(self.dtype).cuda()

    def rows(self, T, n, std=1.0):
        buf = torch.full((T + 1, n + self.pad), float("nan"), dtype=self.dtype, device="cuda")
        buf[:T, :n] = self.whole((T, n), std)
        return buf[:T, :n]

    def out(self, T, n):
        """An output of T rows inside a larger buffer of sentinels."""
        buf = torch.full((T + 2, n + self.pad), 77.0, dtype=self.dtype, device="cuda")
        return buf, buf[1:T + 1, :n]


def untouched(buf, T, n):
    """The sentinels around an output's rows and columns are still there."""
    return bool((buf[0] == 77).all() and (buf[T + 1:] == 77).all() and (buf[:, n:] == 77).all())
