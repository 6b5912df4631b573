"""The dense operators' activations and slopes over their whole range, one
argument at a time: x is one-hot, so a pre-activation is exactly a chosen
value, through the forward epilogues, the dz kernel and the gate gradient.

Bounds, from the arithmetic of the evaluation in fp32 (the output's own
rounding comes on top, in check):
  silu, tanh-gelu: z s with s = 1 / (1 + 2^w).  w has an error of 2^-22 |w| at
    most (three roundings) and the hardware's 2^w and reciprocal 2^-22 each, so
    s is off by at most ln 2 |w| 2^-22 + 2^-21 relative; |w| <= 127 where s is
    not flushed to zero: below 2^-15.  What is flushed is below 2^-126 |z|, with
    |z| < 2^7 where s is that small and not zero itself.
  gelu: Phi(z) by a polynomial in t times E = e^(-z^2 / 2), within 7.5e-8 as
    published; value and approximation lie between 0 and E, so their difference
    does too; the polynomial's and E's roundings are below 2^-20 E, and 1 - tail
    rounds to 2^-25.  The hardware's 2^w returns 0 for results below 2^-126, so
    where E is that small (|z| > 13.2) the density z E / sqrt(2 pi) is lost
    whole: 0.4 |z| E, at most 0.4 x 13.3 x 2^-126 = 2^-123.
  slopes: the sums of their terms, each with the error of its factors; 1 - s is
    within 2^-22 (s rounds near 1) until 2^w < 2^-24, from where s is 1.
relu and none are exact, relu^2 rounds once.
"""
import math

import numpy as np
import pytest
import torch

from dense_testlib import check, np64
from grouped_gemm_gating_b200 import moe as M
from oracle import dense_oracle as D

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
EPI = {n: getattr(M, "EPI_" + n.upper()) for n in D.ACTS}
C = math.sqrt(2.0 / math.pi)
# two sizes of batch: the split kernel, and the pair kernel (asserted in
# test_dense_plan.py)
FORWARD = [(2, 8, 72), (5003, 8, 2552)]
BACKWARD = [(2, 8, 72), (4097, 520, 1256)]


def values(name, dtype, n):
    """n arguments: a grid through the steep part, the tails, and far beyond
    (as far as the result is finite)."""
    far = [1e-30, 1e-3, 20.0, 30.0, 60.0, 87.0, 90.0, 125.0, 200.0]
    if not (name == "relu2" and dtype is HF):
        far += [300.0, 1e4, 6e4]
    if dtype is BF:
        far += [1e10, 1e18]
    z = [0.0] + far + list(np.linspace(0.0625, 16.0, 24))
    z = torch.tensor(z + [-v for v in z], dtype=torch.float64).to(dtype)
    return z.repeat(n // len(z) + 1)[:n]


def sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def reference(z, name):
    """(value, its bound, slope, its bound)."""
    zero = 0.0 * z
    E = np.exp(-0.5 * np.minimum(z * z, 1e4))
    E = np.where(E < 1e-300, 0.0, E)
    if name == "none":
        return z, zero, zero + 1.0, zero
    if name == "relu":
        return np.maximum(z, 0.0), zero, (z > 0).astype(np.float64), zero
    if name == "relu2":
        p = np.maximum(z, 0.0)
        return p * p, 2.0 ** -24 * p * p, 2.0 * p, zero
    if name == "gelu":
        value, slope = D.act(z, name), D.act_slope(np.clip(z, -1e3, 1e3), name)
        phi = np.minimum(7.5e-8, E) + 2.0 ** -20 * E + (z > 0) * 2.0 ** -24
        zc = np.minimum(np.abs(z), 1e3)
        flushed = np.where(E < 2.0 ** -125, E, 0.0)  # E's own bound counts: a normal one may be computed below 2^-126
        density = 0.4 * zc * (E * (zc * zc * 2.0 ** -23 + 2.0 ** -21) + flushed)
        return value, np.abs(z) * phi + 2.0 ** -24 * np.abs(value), slope, phi + density + 2.0 ** -23 * np.abs(slope)
    if name == "silu":
        s, steep = sigmoid(z), zero + 1.0
    else:
        zc = np.clip(z, -1e3, 1e3)
        s = sigmoid(2.0 * C * (zc + 0.044715 * zc ** 3))
        steep = 2.0 * C * (1.0 + 3.0 * 0.044715 * zc * zc)
    value = z * s
    rest = sigmoid(-z) if name == "silu" else sigmoid(-2.0 * C * (zc + 0.044715 * zc ** 3))  # 1 - s
    hill = np.where(np.abs(z) < 800.0, z, 0.0) * s * rest * steep
    small = np.where(z < 0.0, 2.0 ** -126, 0.0) * np.minimum(np.abs(z), 128.0)
    ends = z > (17.0 if name == "silu" else 8.0)  # s is 1
    e_slope = np.where(z < 0.0, 2.0 ** -14 * (s + np.abs(hill)) + small * np.minimum(steep, 128.0),
                       np.where(ends, 2.0 ** -22, 2.0 ** -21 * (1.0 + z * np.where(ends, 0.0, steep))))
    return value, 2.0 ** -15 * np.abs(value) + small, s + hill, e_slope


def exact_ends(got, z, name):
    """Beyond the reach of an activation its value is z or 0, nothing between."""
    if name in ("none", "relu2"):
        return
    got, z = np64(got), np.broadcast_to(z, got.shape)
    assert np.array_equal(got[z >= 30.0], z[z >= 30.0])
    assert (got[z <= -125.0] == 0.0).all()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("name", D.ACTS)
@pytest.mark.parametrize("T,K,N", FORWARD)
def test_values(T, K, N, name, dtype):
    """moe_linear's activation, and the gate's in moe_ffn."""
    z = values(name, dtype, N)
    x = torch.zeros(T, K, dtype=dtype, device="cuda")
    x[:, 0] = 1.0
    w = torch.zeros(2 * N, K, dtype=dtype, device="cuda")
    w[:N, 0], w[N:, 0] = z.cuda(), 1.0
    out, h = (torch.full((T, N), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    y = torch.empty(T, K, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    M.moe_linear(x, w[:N], out, act=EPI[name], dev_status=status)
    M.moe_ffn(x, w, torch.zeros(K, N, dtype=dtype, device="cuda"), h, y, EPI[name], dev_status=status)
    torch.cuda.synchronize()
    assert M.moe_read_status(status) == 0
    z = np64(z)
    ref, bound, _, _ = reference(z, name)
    for got in (out, h):
        rows = got[[0, T // 2, T - 1]]
        check(rows, np.stack([ref] * 3), np.stack([bound] * 3), name, dtype)
        assert torch.equal(got, got[:1].expand_as(got))
        exact_ends(rows, z, name)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("name", D.ACTS)
@pytest.mark.parametrize("T,K,N", BACKWARD)
def test_slopes(T, K, N, name, dtype):
    """dbias of moe_linear_backward (one row's dout is 1, the others' 0), and
    [dg | du] and h of moe_ffn_backward, read from dw13 and dw2."""
    z = values(name, dtype, N).cuda()
    t0 = T // 2
    mk = lambda *s: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x, dout, pre, db = mk(T, K), mk(T, N), mk(T, N), mk(N) + 7
    dout[t0], pre[:] = 1.0, z
    if name != "none":
        ws = torch.empty(M.moe_linear_backward_workspace_size(T, K, N, EPI[name]), dtype=torch.uint8, device="cuda")
        M.moe_linear_backward(x, mk(N, K), dout, None, None, db, EPI[name], pre, ws, dev_status=status)
    x[:, 0] = 1.0
    dout, pre, w2 = mk(T, K), mk(T, 2 * N), mk(K, N)
    dout[t0, 0], w2[0] = 1.0, 1.0  # dh = 1 in one row
    pre[:, :N], pre[:, N:] = z, 1.0
    dw13, dw2 = mk(2 * N, K) + 7, mk(K, N) + 7
    ws = torch.empty(M.moe_ffn_backward_workspace_size(T, K, N), dtype=torch.uint8, device="cuda")
    M.moe_ffn_backward(x, mk(2 * N, K), w2, pre, dout, ws, None, dw13, dw2, EPI[name], dev_status=status)
    torch.cuda.synchronize()
    assert M.moe_read_status(status) == 0
    z = np64(z)
    ref, bound, slope, e_slope = reference(z, name)
    if name != "none":
        check(db, slope, e_slope, name + " dbias", dtype)
    check(dw13[:N, 0], slope, e_slope, name + " dg", dtype)
    check(dw13[N:, 0], ref, bound, name + " du", dtype)
    check(dw2[0], ref, bound, name + " h", dtype)
    exact_ends(dw2[0], z, name)
    assert not dw13[:, 1:].any() and not dw2[1:].any()
