"""GPU parity of the dense operators (linear layer, gated feed-forward block,
their gradients) against the fp64 oracle, through the C ABI."""
import numpy as np
import pytest
import torch

from dense_testlib import (ADD, U, Draw, act_error, check, linear_bounds, np64, product_bound, round_error,
                           slope_error, sums, untouched)
from grouped_gemm_gating_b200 import moe as M
from oracle import dense_oracle as D

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
EPI = {n: getattr(M, "EPI_" + n.upper()) for n in D.ACTS}


def ok(status):
    torch.cuda.synchronize()
    code = M.moe_read_status(status)
    assert code == 0, M.status_name(code)


# T, K, N, act, bias, residual, pre, dtype, pad: every tile edge (16, 64, 128,
# 256), one token, odd tokens, the narrowest and odd widths, long contractions
LINEAR = [
    (1, 8, 8, "none", False, False, False, BF, 0),
    (1, 2048, 2048, "none", False, True, False, BF, 0),
    (2, 72, 24, "silu", True, False, True, HF, 8),
    (3, 4096, 512, "gelu", True, True, True, BF, 0),
    (7, 1000, 1848, "relu2", True, True, True, HF, 24),
    (15, 64, 128, "relu", False, False, False, BF, 0),
    (16, 128, 136, "gelu_tanh", True, False, True, BF, 0),
    (17, 520, 264, "silu", False, True, False, HF, 40),
    (33, 264, 1000, "none", True, True, False, BF, 8),
    (64, 512, 640, "gelu", False, False, True, HF, 0),
    (65, 136, 72, "relu2", True, True, True, BF, 16),
    (127, 1024, 256, "silu", True, False, False, BF, 0),
    (128, 192, 384, "none", False, True, False, HF, 0),
    (129, 64, 8, "gelu_tanh", True, True, True, BF, 8),
    (255, 328, 264, "relu", True, True, True, HF, 0),
    (256, 256, 256, "none", False, False, False, BF, 0),
    (257, 1352, 680, "gelu", True, True, True, BF, 0),
    (300, 6152, 520, "silu", False, True, True, HF, 8),
    (777, 1000, 1848, "relu2", True, True, True, HF, 24),
    (1100, 520, 2312, "gelu_tanh", True, True, True, BF, 0),
    (2500, 72, 1032, "none", True, True, False, BF, 8),
    # several rounds of tiles: a whole last round, halves in it, and a last
    # column of tiles that lies half outside
    (5003, 136, 2552, "silu", True, True, False, BF, 8),
    (4700, 200, 2048, "none", False, True, True, HF, 0),
    (9700, 64, 1304, "gelu_tanh", True, False, True, BF, 0),
]


@pytest.mark.parametrize("T,K,N,name,bias,residual,keep,dtype,pad", LINEAR)
def test_linear(T, K, N, name, bias, residual, keep, dtype, pad):
    d = Draw(T * 7 + K, dtype, pad)
    x, w = d.rows(T, K), d.whole((N, K), K ** -0.5)
    b = d.whole((N,), 0.5) if bias else None
    r = d.rows(T, N) if residual else None
    buf, out = d.out(T, N)
    pre = torch.full((T, N), 77.0, dtype=dtype, device="cuda") if keep else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    M.moe_linear(x, w, out, b, r, EPI[name], pre, status)
    ok(status)
    ref, zref = D.linear(np64(x), np64(w), np64(b), np64(r), name)
    e_out, e_pre = linear_bounds(np64(x), np64(w), zref, name)
    check(out, ref, e_out + 2.0 ** -23 * np.abs(ref), "out", dtype)
    if keep:
        check(pre, zref, e_pre, "pre", dtype)
    assert untouched(buf, T, N)


def test_linear_in_place_residual():
    d = Draw(5, BF)
    x, w = d.whole((70, 128)), d.whole((264, 128), 0.1)
    r = d.whole((70, 264))
    want = torch.empty_like(r)
    M.moe_linear(x, w, want, None, r)
    M.moe_linear(x, w, r, None, r)
    torch.cuda.synchronize()
    assert torch.equal(r, want)


@pytest.mark.parametrize("T", [1, 5, 130, 300])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_linear_keeps_bad_rows_apart(T, bad):
    """A NaN or infinity in a token's row reaches that row alone, in a
    weight's row that column alone."""
    d = Draw(6, BF)
    x, w = d.whole((T, 200)), d.whole((136, 200), 0.1)
    clean = torch.empty(T, 136, dtype=BF, device="cuda")
    M.moe_linear(x, w, clean)
    x[T // 2, 3] = bad
    out = torch.empty_like(clean)
    M.moe_linear(x, w, out)
    x[T // 2, 3] = 0.0
    w[77, 5] = bad
    out2 = torch.empty_like(clean)
    M.moe_linear(x, w, out2)
    torch.cuda.synchronize()
    assert not torch.isfinite(out[T // 2]).any()
    keep = torch.arange(T, device="cuda") != T // 2
    assert torch.equal(out[keep], clean[keep])
    assert not torch.isfinite(out2[:, 77]).any()
    cols = torch.arange(136, device="cuda") != 77
    assert torch.equal(out2[keep][:, cols], clean[keep][:, cols])


@pytest.mark.parametrize("name", D.ACTS)
def test_activation_extremes(name):
    """Large and tiny arguments through the epilogue: x is one-hot, so the
    pre-activation is exactly w's value."""
    vals = [0.0, -0.0, 1e-30, -1e-30, 1e-3, -1e-3, 0.5, -0.5, 3.0, -3.0, 9.0, -9.0, 30.0, -30.0, 90.0, -90.0, 300.0,
            -300.0, 1e4, -1e4, 1e18, -1e18, 1.0, -1.0]
    w = torch.zeros(24, 8, dtype=BF)
    w[:, 0] = torch.tensor(vals).to(BF)
    x = torch.zeros(2, 8, dtype=BF)
    x[:, 0] = 1.0
    out = torch.empty(2, 24, dtype=BF, device="cuda")
    M.moe_linear(x.cuda(), w.cuda(), out, act=EPI[name])
    z = np64(w)[:, 0]
    ref = np.stack([D.act(z, name)] * 2)
    # below 2^-60 an activation's tail counts as zero
    check(out, ref, np.stack([act_error(z, 0.0 * z, name)] * 2) + 2.0 ** -60, name, BF)


# T, K, N, act, bias, dx_residual, dtype, pad
LINEAR_BWD = [
    (1, 8, 8, "silu", True, False, BF, 0),
    (5, 64, 72, "none", True, True, HF, 8),
    (64, 264, 128, "gelu", True, False, BF, 0),
    (127, 136, 520, "relu2", False, True, BF, 16),
    (129, 512, 264, "gelu_tanh", True, True, HF, 0),
    (413, 1352, 680, "none", True, False, HF, 8),
    (300, 72, 1032, "relu", True, True, BF, 0),
    (1030, 520, 264, "silu", True, False, BF, 40),
    (4700, 1024, 5112, "none", False, True, BF, 8),   # rounds of tiles, both products in one launch
]


@pytest.mark.parametrize("T,K,N,name,bias,res,dtype,pad", LINEAR_BWD)
def test_linear_backward(T, K, N, name, bias, res, dtype, pad):
    d = Draw(T * 3 + N, dtype, pad)
    x, w, dout = d.rows(T, K), d.whole((N, K), K ** -0.5), d.rows(T, N)
    pre = d.whole((T, N)) if name != "none" else None
    dxr = d.rows(T, K) if res else None
    buf, dx = d.out(T, K)
    dw = torch.full((N, K), 77.0, dtype=dtype, device="cuda")
    db = torch.full((N,), 77.0, dtype=dtype, device="cuda") if bias else None
    n = M.moe_linear_backward_workspace_size(T, K, N, EPI[name])
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    M.moe_linear_backward(x, w, dout, dx, dw, db, EPI[name], pre, ws, dxr, status)
    ok(status)
    X, W, G, P = np64(x), np64(w), np64(dout), np64(pre)
    rdx, rdw, rdb, dz = D.linear_backward(X, W, G, name, P, np64(dxr))
    fp32 = np.abs(G) * slope_error(P, name) + 2.0 ** -23 * np.abs(dz) if name != "none" else 0 * dz
    dz_err = fp32 + (round_error(np.abs(dz) + fp32, dtype) if name != "none" else 0)
    check(dx, rdx, product_bound(dz, W.T, dz_err) + 2.0 ** -23 * np.abs(rdx), "dx", dtype)
    check(dw, rdw, product_bound(dz.T, X.T, dz_err.T), "dw", dtype)
    if bias:
        check(db, rdb, (T * ADD * np.abs(dz) + fp32).sum(0), "dbias", dtype)
    assert untouched(buf, T, K)


def test_linear_backward_parts():
    """Each gradient alone equals the one of the whole call."""
    d = Draw(9, BF)
    x, w, dout, pre = d.whole((200, 136)), d.whole((72, 136), 0.1), d.whole((200, 72)), d.whole((200, 72))
    ws = torch.empty(M.moe_linear_backward_workspace_size(200, 136, 72, M.EPI_SILU), dtype=torch.uint8, device="cuda")
    mk = lambda: [torch.zeros(s, dtype=BF, device="cuda") for s in ((200, 136), (72, 136), (72,))]  # noqa: E731
    whole = mk()
    M.moe_linear_backward(x, w, dout, *whole, M.EPI_SILU, pre, ws)
    for i in range(3):
        part = [None, None, None]
        part[i] = mk()[i]
        M.moe_linear_backward(x, w, dout, *part, M.EPI_SILU, pre, ws)
        torch.cuda.synchronize()
        assert torch.equal(part[i], whole[i])


# T, d, F, act, residual, pre, dtype, pad
FFN = [
    (1, 8, 8, "silu", False, True, BF, 0),
    (1, 2048, 768, "silu", True, False, BF, 0),
    (3, 520, 1352, "gelu", True, True, HF, 8),
    (16, 64, 128, "relu", False, False, BF, 0),
    (33, 136, 72, "relu2", True, True, BF, 0),
    (64, 512, 264, "gelu_tanh", True, True, HF, 0),
    (130, 264, 520, "silu", True, True, BF, 16),
    (261, 672, 464, "gelu", False, True, BF, 0),
    (300, 1016, 1720, "none", True, True, HF, 0),
    (1290, 136, 328, "silu", True, False, BF, 8),
    (5003, 72, 1256, "silu", True, True, BF, 8),      # rounds of tiles
    (4900, 200, 1000, "gelu", False, False, HF, 0),
]


@pytest.mark.parametrize("T,d_,F,name,residual,keep,dtype,pad", FFN)
def test_ffn(T, d_, F, name, residual, keep, dtype, pad):
    d = Draw(T + d_ + F, dtype, pad)
    x, w13, w2 = d.rows(T, d_), d.whole((2 * F, d_), d_ ** -0.5), d.whole((d_, F), F ** -0.5)
    r = d.rows(T, d_) if residual else None
    buf, out = d.out(T, d_)
    h = torch.full((T + 1, F), 77.0, dtype=dtype, device="cuda")
    pre = torch.full((T + 1, 2 * F), 77.0, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    M.moe_ffn(x, w13, w2, h[:T], out, EPI[name], r, pre[:T] if keep else None, status)
    ok(status)
    X, A, B = np64(x), np64(w13), np64(w2)
    ref, zref, href = D.ffn(X, A, B, name, np64(r))
    e = d_ * ADD * sums(X, A)
    g, u, eg, eu = zref[:, :F], zref[:, F:], e[:, :F], e[:, F:]
    a, ea = D.act(g, name), act_error(g, eg, name)
    eh = ea * (np.abs(u) + eu) + np.abs(a) * eu + 2.0 ** -23 * np.abs(href)
    check(h[:T], href, eh, "h", dtype)
    eh = eh + round_error(np.abs(href) + eh, dtype)
    check(out, ref, product_bound(href, B, eh) + 2.0 ** -23 * np.abs(ref), "out", dtype)
    if keep:
        check(pre[:T], zref, e, "pre", dtype)
    assert untouched(buf, T, d_)
    assert bool((h[T] == 77).all() and (pre[T] == 77).all())
    # two roundings (h, out): relative L2 within u each
    err = np.linalg.norm(np64(out) - ref) / np.linalg.norm(ref)
    assert err <= 2 * U[dtype], err


def test_ffn_out_may_be_x():
    d = Draw(12, BF)
    x, w13, w2 = d.whole((40, 128)), d.whole((528, 128), 0.1), d.whole((128, 264), 0.1)
    h, want = torch.empty(40, 264, dtype=BF, device="cuda"), torch.empty(40, 128, dtype=BF, device="cuda")
    M.moe_ffn(x, w13, w2, h, want, residual=x)
    M.moe_ffn(x, w13, w2, h, x, residual=x)
    torch.cuda.synchronize()
    assert torch.equal(x, want)


# T, d, F, act, dx_residual, dtype, pad
FFN_BWD = [
    (1, 8, 8, "silu", False, BF, 0),
    (9, 64, 72, "gelu", True, HF, 8),
    (64, 136, 264, "relu2", False, BF, 0),
    (129, 512, 328, "silu", True, BF, 16),
    (333, 1016, 520, "gelu_tanh", False, HF, 16),
    (300, 72, 1032, "relu", True, BF, 0),
    (1030, 264, 136, "none", False, BF, 0),
    (3, 2040, 4096, "relu", True, BF, 0),     # dx in a launch of its own
]


@pytest.mark.parametrize("T,d_,F,name,res,dtype,pad", FFN_BWD)
def test_ffn_backward(T, d_, F, name, res, dtype, pad):
    d = Draw(T + 2 * d_ + F, dtype, pad)
    x, w13, w2 = d.rows(T, d_), d.whole((2 * F, d_), d_ ** -0.5), d.whole((d_, F), F ** -0.5)
    pre, dout = d.whole((T, 2 * F)), d.rows(T, d_)
    dxr = d.rows(T, d_) if res else None
    buf, dx = d.out(T, d_)
    dw13 = torch.full((2 * F, d_), 77.0, dtype=dtype, device="cuda")
    dw2 = torch.full((d_, F), 77.0, dtype=dtype, device="cuda")
    ws = torch.full((M.moe_ffn_backward_workspace_size(T, d_, F),), 255, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    M.moe_ffn_backward(x, w13, w2, pre, dout, ws, dx, dw13, dw2, EPI[name], dxr, status)
    ok(status)
    X, A, B, P, G = np64(x), np64(w13), np64(w2), np64(pre), np64(dout)
    rdx, rdw13, rdw2, da, h = D.ffn_backward(X, A, B, P, G, name, np64(dxr))
    g, u = P[:, :F], P[:, F:]
    dh = G @ B
    e_dh = d_ * ADD * sums(G, B.T)
    slope, a = D.act_slope(g, name), D.act(g, name)
    e_s, e_a = slope_error(g, name), act_error(g, 0.0, name)
    e_dg = e_dh * np.abs(u * slope) + (np.abs(dh) + e_dh) * np.abs(u) * e_s
    e_du = e_dh * np.abs(a) + (np.abs(dh) + e_dh) * e_a
    e_da = np.concatenate([e_dg, e_du], 1) + 2.0 ** -22 * np.abs(da)
    e_da = e_da + round_error(np.abs(da) + e_da, dtype)
    e_h = e_a * np.abs(u) + 2.0 ** -23 * np.abs(h)
    e_h = e_h + round_error(np.abs(h) + e_h, dtype)
    check(dx, rdx, product_bound(da, A.T, e_da) + 2.0 ** -23 * np.abs(rdx), "dx", dtype)
    check(dw13, rdw13, product_bound(da.T, X.T, e_da.T), "dw13", dtype)
    check(dw2, rdw2, product_bound(h.T, G.T, e_h.T).T, "dw2", dtype)
    assert untouched(buf, T, d_)
    for got, ref in ((dx, rdx), (dw13, rdw13), (dw2, rdw2)):
        norm = np.linalg.norm(ref)
        assert np.linalg.norm(np64(got) - ref) <= 2 * U[dtype] * norm + 1e-6


# The same tests at sizes of which every launch runs on CTA pairs (asserted
# without a GPU in test_dense_plan.py): odd token counts, widths that end inside
# a tile and inside 64 columns, a last round of whole tiles and of halves, rounds
# that reuse the epilogue's buffers, both types.
LINEAR_BWD_PAIRS = [
    (4700, 1032, 2056, "gelu", True, True, HF, 8),
    (3001, 1032, 2312, "relu2", True, False, BF, 0),
]
FFN_BWD_PAIRS = [
    (4097, 520, 1256, "silu", True, BF, 8),
    (4097, 264, 2312, "gelu", True, HF, 0),
    (3001, 520, 2312, "gelu_tanh", False, HF, 16),
    (2100, 1032, 1032, "relu2", True, BF, 0),
]


@pytest.mark.parametrize("case", LINEAR_BWD_PAIRS, ids=str)
def test_linear_backward_on_pairs(case):
    test_linear_backward(*case)


@pytest.mark.parametrize("case", FFN_BWD_PAIRS, ids=str)
def test_ffn_backward_on_pairs(case):
    test_ffn_backward(*case)


@pytest.mark.parametrize("name,g", [("relu", -1.0), ("relu2", -1.0), ("silu", -200.0), ("gelu", -40.0),
                                    ("gelu_tanh", -40.0)])
@pytest.mark.parametrize("T", [4, 9000])  # the split kernel and the pair kernel
def test_ffn_backward_of_a_closed_gate(T, name, g):
    """Where the gate's value and slope are 0, large finite dh and u (their
    product beyond fp32) give zero gradients, not 0 * infinity."""
    dd, F = 512, 1024
    e = lambda *s: torch.zeros(s, dtype=BF, device="cuda")  # noqa: E731
    x, dout, pre = e(T, dd), e(T, dd), e(T, 2 * F)
    w13, w2 = e(2 * F, dd) + 1, e(dd, F)
    x += 1
    dout[:, 0], w2[0] = 1e20, 1.0      # dh = 1e20
    pre[:, :F], pre[:, F:] = g, 1e20
    dx, dw13, dw2 = e(T, dd) + 7, e(2 * F, dd) + 7, e(dd, F) + 7
    ws = torch.empty(M.moe_ffn_backward_workspace_size(T, dd, F), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    M.moe_ffn_backward(x, w13, w2, pre, dout, ws, dx, dw13, dw2, EPI[name], dev_status=status)
    ok(status)
    assert not any(bool(t.any()) for t in (dx, dw13, dw2))


def test_ffn_gradients_against_differences():
    """The whole step's gradients against central differences of the oracle's
    forward in fp64, on the same values: directions drawn at random."""
    d = Draw(21, BF)
    T, dd, F = 48, 72, 40
    x, w13, w2, dout = d.whole((T, dd)), d.whole((2 * F, dd), 0.2), d.whole((dd, F), 0.2), d.whole((T, dd))
    b = M.FFNBuffers(T, dd, F, train=True)
    b.forward(x, w13, w2)
    b.backward(x, w13, w2, dout)
    ok(b.status)
    X, A, B, G = np64(x), np64(w13), np64(w2), np64(dout)
    loss = lambda X, A, B: float((D.ffn(X, A, B)[0] * G).sum())  # noqa: E731
    rng = np.random.Generator(np.random.PCG64(3))
    _, pre, _ = D.ffn(X, A, B)
    grads = D.ffn_backward(X, A, B, pre, G)
    for i, (got, ref) in enumerate(zip((b.dx, b.dw13, b.dw2), grads)):
        v = rng.standard_normal(ref.shape)
        args = [X, A, B]
        e = 1e-5
        hi, lo = list(args), list(args)
        hi[i], lo[i] = args[i] + e * v, args[i] - e * v
        num = (loss(*hi) - loss(*lo)) / (2 * e)
        # pre, then da and h, and the result are rounded: at most 4 u of each
        # term's size (a slope moves by at most 0.5 per unit of its argument)
        bound = 4 * U[BF] * float((np.abs(ref) * np.abs(v)).sum()) + 4 * U[BF] * np.linalg.norm(ref) * np.linalg.norm(v)
        assert abs(num - float((ref * v).sum())) <= 1e-5 * abs(num) + 1e-4
        assert abs(num - float((np64(got) * v).sum())) <= bound


def test_no_rows():
    """T = 0: outputs of T rows are no-ops, weight gradients become zero."""
    e = lambda *s: torch.empty(s, dtype=BF, device="cuda")  # noqa: E731
    dw, db = torch.ones(32, 64, dtype=BF, device="cuda"), torch.ones(32, dtype=BF, device="cuda")
    w = e(32, 64)
    M.moe_linear(e(0, 64), w, e(0, 32))
    M.moe_linear_backward(e(0, 64), w, e(0, 32), e(0, 64), dw, db)
    dw13, dw2 = torch.ones(64, 16, dtype=BF, device="cuda"), torch.ones(16, 32, dtype=BF, device="cuda")
    M.moe_ffn(e(0, 16), e(64, 16), e(16, 32), e(0, 32), e(0, 16))
    M.moe_ffn_backward(e(0, 16), e(64, 16), e(16, 32), e(0, 64), e(0, 16), None, e(0, 16), dw13, dw2)
    torch.cuda.synchronize()
    assert not any(bool(t.any()) for t in (dw, db, dw13, dw2))


def test_same_on_every_call_and_stream():
    """Results repeat bit for bit, on another stream and replayed from a graph."""
    d = Draw(31, BF)
    T, dd, F = 300, 264, 520
    x, w13, w2, dout = d.whole((T, dd)), d.whole((2 * F, dd), 0.1), d.whole((dd, F), 0.1), d.whole((T, dd))
    b = M.FFNBuffers(T, dd, F, train=True)
    names = ("out", "pre", "h", "dx", "dw13", "dw2")

    def step():
        b.forward(x, w13, w2, x)
        b.backward(x, w13, w2, dout, dx_residual=dout)

    def taken():
        torch.cuda.synchronize()
        got = [getattr(b, n).clone() for n in names]
        for n in names:
            getattr(b, n).zero_()
        torch.cuda.synchronize()
        return got

    step()
    want = taken()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    for a, c in zip(taken(), want):
        assert torch.equal(a, c)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        step()
    with torch.cuda.graph(g2):
        step()
    for g in (g1, g2, g1):
        g.replay()
        for a, c in zip(taken(), want):
            assert torch.equal(a, c)


@pytest.mark.parametrize("T", [1, 3, 5, 13])
def test_split_kernel_repeats(T):
    """Rows and shares of columns that leave the lanes of a warp a different
    number of items each, before the cluster's barrier; odd column sums."""
    d = Draw(33, BF)
    K, N = 1000, 1848
    x, w, r, dout = d.whole((T, K)), d.whole((N, K), K ** -0.5), d.whole((T, N)), d.whole((T, N))
    out, dx = torch.empty_like(r), torch.empty_like(x)
    dw, db = torch.empty_like(w), torch.empty(N, dtype=BF, device="cuda")
    want = None
    for _ in range(50):
        M.moe_linear(x, w, out, None, r)
        M.moe_linear_backward(x, w, dout, dx, dw, db)
        got = [t.clone() for t in (out, dx, dw, db)]
        want = want or got
        for a, c in zip(got, want):
            assert torch.equal(a, c)
    X, W = np64(x), np64(w)
    ref, zref = D.linear(X, W, None, np64(r))
    check(want[0], ref, linear_bounds(X, W, zref, "none")[0] + 2.0 ** -23 * np.abs(ref), "out", BF)
    G = np64(dout)
    check(want[3], G.sum(0), T * ADD * np.abs(G).sum(0), "dbias", BF)


def test_pair_kernel_repeats():
    """Large batches: what TMA brings for the epilogue (a residual, the kept
    g and u) is seen by every lane of a warp, call after call."""
    d = Draw(32, BF)
    T, K, N = 9001, 264, 2056
    x, w, r = d.whole((T, K)), d.whole((N, K), K ** -0.5), d.whole((T, N))
    b = M.FFNBuffers(T, K, 1032, train=True)
    w13, w2, dout = d.whole((2064, K), 0.05), d.whole((K, 1032), 0.05), d.whole((T, K))
    out = torch.empty_like(r)
    names = ("out", "pre", "dx", "dw13", "dw2")
    want = None
    for _ in range(20):
        M.moe_linear(x, w, out, None, r)
        b.forward(x, w13, w2, x)
        b.backward(x, w13, w2, dout, dx_residual=dout)
        got = [out.clone()] + [getattr(b, n).clone() for n in names]
        want = want or got
        for a, c in zip(got, want):
            assert torch.equal(a, c)
    ok(b.status)
    X, W = np64(x[-300:]), np64(w)
    ref, zref = D.linear(X, W, None, np64(r[-300:]))
    check(want[0][-300:], ref, linear_bounds(X, W, zref, "none")[0] + 2.0 ** -23 * np.abs(ref), "last rows", BF)


def test_offsets_past_32_bits():
    """An output of more than 2^31 elements, its last rows checked."""
    T, K, N = (1 << 18) + 100, 8, 8200
    x = torch.zeros(T, K, dtype=BF, device="cuda")
    x[:, 0] = 1.0
    x[-300:, 1] = torch.arange(300, device="cuda").to(BF)
    w = torch.zeros(N, K, dtype=BF, device="cuda")
    w[:, 0] = (torch.arange(N, device="cuda") % 128).to(BF)
    w[:, 1] = 1.0
    out = torch.empty(T, N, dtype=BF, device="cuda")
    M.moe_linear(x, w, out)
    torch.cuda.synchronize()
    want = (x[-400:].float() @ w.float().T).to(BF)  # small whole numbers: exact in fp32
    assert torch.equal(out[-400:], want)
    assert torch.equal(out[:5], (x[:5].float() @ w.float().T).to(BF))


def test_product_of_more_than_a_second():
    """1.9e15 operations in one launch, at least 1.2 s at the rate that a step
    of k takes: the kernel's waits run per tile, not per launch.  Values +-1:
    sums are whole numbers below 2^24, exact in fp32, then rounded once."""
    n = 98_816
    gen = torch.Generator(device="cuda").manual_seed(47)

    def signs():
        t = torch.empty(n, n, dtype=BF, device="cuda")
        for i in range(0, n, 8192):
            part = t[i:i + 8192]
            part.copy_(torch.randint(0, 2, part.shape, generator=gen, device="cuda", dtype=torch.int8) * 2 - 1)
        return t

    x, w = signs(), signs()
    out = torch.empty(n, n, dtype=BF, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    M.moe_linear(x, w, out, dev_status=status)
    ok(status)
    rows = torch.cat([torch.arange(0, n, 3001, device="cuda"), torch.arange(n - 3, n, device="cuda")])
    xs = x[rows].float()
    for i in range(0, n, 8192):
        want = (xs @ w[i:i + 8192].float().T).to(BF)
        assert torch.equal(out[rows, i:i + 8192], want)
    del x, w, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,N", [(4, 512), (300, 512), (9000, 2048)])
def test_timeout_is_reported(T, N):
    """A wait that runs out sets the status; the next call works.  Few rows,
    a medium batch, and the pair kernel with a residual on its way."""
    d = Draw(41, BF)
    x, w, r = d.whole((T, 512)), d.whole((N, 512), 0.05), d.whole((T, N))
    want, out = torch.empty(T, N, dtype=BF, device="cuda"), torch.empty(T, N, dtype=BF, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    M.moe_linear(x, w, want, None, r, dev_status=status)
    ok(status)
    try:
        M.moe_debug_timeouts(20_000_000, 1)
        M.moe_linear(x, w, out, None, r, dev_status=status)
        torch.cuda.synchronize()
    finally:
        M.moe_debug_timeouts(0, 0)
    assert M.status_name(M.moe_read_status(status)) == "MOE_ERR_DEVICE_TIMEOUT"
    status.zero_()
    M.moe_linear(x, w, out, None, r, dev_status=status)
    ok(status)
    assert torch.equal(out, want)


@pytest.mark.parametrize("T", [40, 9000])
def test_timeout_in_the_block(T):
    """The same through moe_ffn and moe_ffn_backward (gate, gate gradient and
    joint gradient kernels)."""
    d = Draw(42, BF)
    dd, F = 512, 1024
    x, w13, w2, dout = d.whole((T, dd)), d.whole((2 * F, dd), 0.05), d.whole((dd, F), 0.05), d.whole((T, dd))
    b = M.FFNBuffers(T, dd, F, train=True)

    def step():
        b.forward(x, w13, w2, x)
        b.backward(x, w13, w2, dout, dx_residual=dout)
        torch.cuda.synchronize()
        return [t.clone() for t in (b.out, b.dx, b.dw13, b.dw2)]

    want = step()
    ok(b.status)
    try:
        M.moe_debug_timeouts(10_000_000, 1)
        step()
    finally:
        M.moe_debug_timeouts(0, 0)
    assert M.status_name(M.moe_read_status(b.status)) == "MOE_ERR_DEVICE_TIMEOUT"
    b.status.zero_()
    for a, c in zip(step(), want):
        assert torch.equal(a, c)
    ok(b.status)


@pytest.mark.parametrize("T", [3, 700, 6000])
def test_slices_of_one_buffer(T):
    """x and out are neighbouring column slices of one buffer."""
    d = Draw(43, BF)
    buf = d.whole((T, 200 + 1000))
    keep = buf[:, :200].clone()
    w = d.whole((1000, 200), 0.1)
    want = torch.empty(T, 1000, dtype=BF, device="cuda")
    M.moe_linear(keep, w, want)
    M.moe_linear(buf[:, :200], w, buf[:, 200:])
    torch.cuda.synchronize()
    assert torch.equal(buf[:, 200:], want) and torch.equal(buf[:, :200], keep)


def test_two_calls_at_once():
    """Two streams run the block on buffers of their own at the same time."""
    d = Draw(44, BF)
    dd, F = 264, 520
    w13, w2 = d.whole((2 * F, dd), 0.1), d.whole((dd, F), 0.1)
    xs = [d.whole((T, dd)) for T in (5, 900)]
    bufs = [M.FFNBuffers(x.shape[0], dd, F, train=True) for x in xs]
    want = []
    for x, b in zip(xs, bufs):
        b.forward(x, w13, w2)
        b.backward(x, w13, w2, x)
        torch.cuda.synchronize()
        want.append([t.clone() for t in (b.out, b.dx, b.dw13, b.dw2)])
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(20):
        for x, b, s in zip(xs, bufs, streams):
            with torch.cuda.stream(s):
                b.forward(x, w13, w2)
                b.backward(x, w13, w2, x)
    torch.cuda.synchronize()
    for b, ref in zip(bufs, want):
        for t, r in zip((b.out, b.dx, b.dw13, b.dw2), ref):
            assert torch.equal(t, r)
        ok(b.status)


def test_refusals_leave_outputs_alone():
    x, w = torch.zeros(4, 64, dtype=BF, device="cuda"), torch.zeros(32, 64, dtype=BF, device="cuda")
    out = torch.ones(4, 32, dtype=BF, device="cuda")
    for kw in (dict(x=x.float()), dict(w=w[:, :60]), dict(w=w.to(HF)), dict(out=out.t().contiguous().t()),
               dict(bias=torch.zeros(31, dtype=BF, device="cuda")), dict(residual=out[:3]),
               dict(dev_status=torch.zeros(1, device="cuda")), dict(out=out.cpu())):
        a = dict(x=x, w=w, out=out) | kw
        with pytest.raises((ValueError, M.MoEError)):
            M.moe_linear(**a)
    with pytest.raises(M.MoEError):
        M.moe_linear(torch.zeros(4, 60, dtype=BF, device="cuda"), torch.zeros(32, 60, dtype=BF, device="cuda"), out)
    with pytest.raises(M.MoEError):
        M.moe_linear(x, w, out, act=17)
    torch.cuda.synchronize()
    assert bool((out == 1).all())


def test_training_step_together():
    """Expert layer and dense block, their backward passes, and one clip over
    all weight gradients: as a model runs them."""
    from moe_testlib import DeviceLayer, bf16_dev
    from grouped_gemm_gating_b200 import workloads as W
    cfg = W.MoEConfig("together", T=96, d=128, F=192, E=8, k=2, block_m=128, seed=1777)
    inp = W.make_inputs(cfg)
    layer = DeviceLayer(inp)
    d = Draw(51, BF)
    w13, w2 = d.whole((2 * 264, 128), 0.1), d.whole((128, 264), 0.1)
    dense = M.FFNBuffers(96, 128, 264, train=True)
    grads = M.MoEGradBuffers(96, 128, 192, 8, 2)
    clip = M.GradClip(grads.grads() + [dense.dw13, dense.dw2])
    mid = layer.run()
    out = dense.forward(mid, w13, w2, mid)
    dout = bf16_dev(W.grad_output(96, 128, seed=9))
    dx, _, _ = dense.backward(mid, w13, w2, dout, dx_residual=dout)
    grads.backward(layer.buf, layer.x, layer.w13, layer.w2, dx)
    torch.cuda.synchronize()
    before = [np64(t) for t in grads.grads() + [dense.dw13, dense.dw2]]
    norm = clip.clip(1.0)
    ok(clip.status)
    ok(dense.status)
    assert layer.status() == 0 and torch.isfinite(out).all()
    n, want = D.clip(before, 1.0)
    assert n > 1.0 and abs(float(norm) - n) <= 2.0 ** -22 * n
    for got, ref in zip(grads.grads() + [dense.dw13, dense.dw2], want):
        check(got, ref, 2.0 ** -22 * np.abs(ref), "clipped", BF)
    # the dense block's values, on the layer's own output
    X, A, B = np64(mid), np64(w13), np64(w2)
    ref, pre, h = D.ffn(X, A, B, "silu", X)
    assert np.linalg.norm(np64(out) - ref) <= 2 * U[BF] * np.linalg.norm(ref)
