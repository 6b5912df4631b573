"""Calls of the dense operators that their contract allows at its ends: in
place on large batches, the largest sizes, gradients in every combination,
weights written just before the call, fp16's range, stage profiling."""
import itertools

import numpy as np
import pytest
import torch

import test_gpu_dense as base
from dense_testlib import Draw, check, np64, product_bound, round_error
from grouped_gemm_gating_b200 import moe as M
from oracle import dense_oracle as D

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def ok(status):
    torch.cuda.synchronize()
    code = M.moe_read_status(status)
    assert code == 0, M.status_name(code)


def stat():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def scratch(n):
    return torch.full((n,), 255, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("T", [70, 2500, 9001])
@pytest.mark.parametrize("keep", [False, True])
def test_residual_in_place(T, keep):
    """out is the residual, a column slice of a larger buffer."""
    d = Draw(61, BF, 16)
    x, w, b = d.rows(T, 136), d.whole((2056, 136), 0.1), d.whole((2056,))
    r = d.rows(T, 2056)
    pre = [torch.empty(T, 2056, dtype=BF, device="cuda") if keep else None for _ in range(2)]
    want = torch.empty(T, 2056, dtype=BF, device="cuda")
    status = stat()
    M.moe_linear(x, w, want, b, r, M.EPI_SILU, pre[0], status)
    M.moe_linear(x, w, r, b, r, M.EPI_SILU, pre[1], status)
    ok(status)
    assert torch.equal(r, want) and (not keep or torch.equal(*pre))


@pytest.mark.parametrize("T", [40, 9001])
def test_block_in_place(T):
    """moe_ffn writes over x, which is its residual too; the backward passes
    add to dx what dx holds."""
    d = Draw(62, HF)
    dd, F = 264, 1032
    x, w13, w2 = d.whole((T, dd)), d.whole((2 * F, dd), 0.05), d.whole((dd, F), 0.05)
    h, pre = torch.empty(T, F, dtype=HF, device="cuda"), torch.empty(T, 2 * F, dtype=HF, device="cuda")
    want, status = torch.empty_like(x), stat()
    M.moe_ffn(x, w13, w2, h, want, residual=x, pre=pre, dev_status=status)
    y = x.clone()
    M.moe_ffn(y, w13, w2, h, y, residual=y, dev_status=status)
    ok(status)
    assert torch.equal(y, want)
    dout, r = d.whole((T, dd)), d.whole((T, dd))
    ws = scratch(M.moe_ffn_backward_workspace_size(T, dd, F))
    grads = [torch.empty_like(w13), torch.empty_like(w2)]
    M.moe_ffn_backward(x, w13, w2, pre, dout, ws, want, *grads, dx_residual=r, dev_status=status)
    dx = r.clone()
    M.moe_ffn_backward(x, w13, w2, pre, dout, ws, dx, *grads, dx_residual=dx, dev_status=status)
    ok(status)
    assert torch.equal(dx, want)
    wl, dl = d.whole((520, dd), 0.05), d.whole((T, 520))
    dw = torch.empty_like(wl)
    M.moe_linear_backward(x, wl, dl, want, dw, dx_residual=r, dev_status=status)
    dx = r.clone()
    M.moe_linear_backward(x, wl, dl, dx, dw, dx_residual=dx, dev_status=status)
    ok(status)
    assert torch.equal(dx, want)


@pytest.mark.parametrize("T", [33, 4097])
def test_block_gradients_in_every_combination(T):
    """Each subset of dx, dw13, dw2 against the oracle's values (launches, and
    with them the order of sums, depend on the subset)."""
    d = Draw(63, BF)
    dd, F = 136, 264
    x, w13, w2 = d.whole((T, dd)), d.whole((2 * F, dd), 0.1), d.whole((dd, F), 0.1)
    pre, dout = d.whole((T, 2 * F)), d.whole((T, dd))
    ws = scratch(M.moe_ffn_backward_workspace_size(T, dd, F))
    full = [torch.empty_like(t) for t in (x, w13, w2)]
    status = stat()
    M.moe_ffn_backward(x, w13, w2, pre, dout, ws, *full, dev_status=status)
    ok(status)
    X, A, B, P, G = (np64(t) for t in (x, w13, w2, pre, dout))
    *_, da, h = D.ffn_backward(X, A, B, P, G)
    # two orders of the same fp32 sums, each rounded once
    order = (product_bound(da, A.T, 0 * da), product_bound(da.T, X.T, 0 * da.T), product_bound(h.T, G.T, 0 * h.T).T)
    for which in itertools.product([False, True], repeat=3):
        if not any(which) or all(which):
            continue
        part = [torch.full_like(t, 77.0) if k else None for t, k in zip(full, which)]
        M.moe_ffn_backward(x, w13, w2, pre, dout, ws, *part, dev_status=status)
        ok(status)
        for p, f, e in zip(part, full, order):
            if p is not None:
                ref = np64(f)
                check(p, ref, 2.1 * e + round_error(np.abs(ref) + e, BF), "part", BF)


# T, K, N: the most columns on either side, next to the fewest
@pytest.mark.parametrize("T,K,N", [(1, 1 << 17, 8), (3, 8, 1 << 17), (130, 8, 1 << 17), (130, 1 << 17, 8)])
def test_most_columns(T, K, N):
    base.test_linear(T, K, N, "none", True, True, False, BF, 0)
    base.test_linear_backward(T, K, N, "none", True, True, BF, 0)


@pytest.mark.parametrize("T,dd,F", [(3, 8, 1 << 17), (3, 1 << 17, 8)])
def test_most_columns_of_a_block(T, dd, F):
    base.test_ffn(T, dd, F, "silu", True, True, BF, 0)
    base.test_ffn_backward(T, dd, F, "silu", True, BF, 0)


def test_most_rows():
    """2^24 tokens of 8 values: the ends of the rows, forward; weight gradients
    over all of them (ones in a few rows: exact)."""
    T = 1 << 24
    x = torch.zeros(T, 8, dtype=BF, device="cuda")
    rows = torch.tensor([0, 1, 255, 256, T // 2 - 1, T // 2, T - 257, T - 2, T - 1], device="cuda")
    x[rows, 0] = torch.arange(1.0, 10.0, device="cuda").to(BF)
    w = torch.zeros(16, 8, dtype=BF, device="cuda")
    w[:, 0] = torch.arange(16, device="cuda").to(BF)
    out = torch.full((T, 16), 7.0, dtype=BF, device="cuda")
    status = stat()
    M.moe_linear(x, w, out, dev_status=status)
    ok(status)
    want = (x[rows].float() @ w.float().T).to(BF)
    assert torch.equal(out[rows], want)
    assert int((out != 0).any(1).sum()) == len(rows)
    dout = torch.zeros_like(out)
    dout[rows] = 1.0
    dx, dw, db = torch.full_like(x, 7.0), torch.empty_like(w), torch.empty(16, dtype=BF, device="cuda")
    M.moe_linear_backward(x, w, dout, dx, dw, db, dev_status=status)
    ok(status)
    assert (db == 9).all() and (dw[:, 0] == 45).all() and not dw[:, 1:].any()
    assert (dx[rows, 0] == 120).all() and int((dx != 0).any(1).sum()) == len(rows)


@pytest.mark.parametrize("T", [1, 3, 300])
def test_weights_written_just_before(T):
    """The down projection's weights are fetched ahead of the kernel before it:
    never ahead of the kernels that wrote them, torch's or the library's own."""
    d = Draw(66, BF)
    dd, F = 1024, 2048
    x, w13 = d.whole((T, dd)), d.whole((2 * F, dd), 0.05)
    versions = [d.whole((dd, F), 0.05) for _ in range(4)]
    h, status = torch.empty(T, F, dtype=BF, device="cuda"), stat()
    want = []
    for v in versions:
        out = torch.empty(T, dd, dtype=BF, device="cuda")
        M.moe_ffn(x, w13, v, h, out, dev_status=status)
        torch.cuda.synchronize()
        want.append(out)
    w2 = torch.empty_like(versions[0])
    plans = [M.GradClip([v], [w2]) for v in versions]
    outs = [torch.empty_like(want[0]) for _ in range(80)]
    for i in range(40):
        w2.copy_(versions[i % 4])
        M.moe_ffn(x, w13, w2, h, outs[2 * i], dev_status=status)
        plans[(i + 1) % 4].clip(float("inf"))  # scales by 1 into w2
        M.moe_ffn(x, w13, w2, h, outs[2 * i + 1], dev_status=status)
    ok(status)
    for i in range(40):
        assert torch.equal(outs[2 * i], want[i % 4]) and torch.equal(outs[2 * i + 1], want[(i + 1) % 4])


@pytest.mark.parametrize("T", [2, 5003])
def test_range_of_h(T):
    """h is a value of dtype: beyond fp16's 65504 it is infinite, in bf16 not."""
    for dtype, finite in ((HF, False), (BF, True)):
        x = torch.zeros(T, 8, dtype=dtype, device="cuda")
        x[:, 0] = 1.0
        w13 = torch.zeros(2 * 2552, 8, dtype=dtype, device="cuda")
        w13[:, 0] = 300.0  # g = u = 300: h = 90000
        w2 = torch.zeros(8, 2552, dtype=dtype, device="cuda")
        w2[0] = 2.0 ** -10
        h, out, status = torch.empty(T, 2552, dtype=dtype, device="cuda"), torch.empty_like(x), stat()
        M.moe_ffn(x, w13, w2, h, out, M.EPI_RELU, dev_status=status)
        ok(status)
        if finite:  # 90000 in 8 bits; whole numbers below 2^24 in fp32
            assert (h == 90112).all() and (out[:, 0] == torch.tensor(2552 * 88.0).to(BF).cuda()).all()
        else:
            assert torch.isinf(h).all() and torch.isinf(out[:, 0]).all()


def test_stages_are_timed():
    d = Draw(67, BF)
    b = M.FFNBuffers(9, 64, 72, train=True)
    lin = M.LinearBuffers(9, 64, 72, M.EPI_SILU, train=True, bias=True)
    x, w13, w2, w, g = d.whole((9, 64)), d.whole((144, 64)), d.whole((64, 72)), d.whole((72, 64)), d.whole((9, 72))
    clip = M.GradClip([b.dw13, b.dw2, lin.dw, lin.dbias])

    def step():
        b.forward(x, w13, w2)
        b.backward(x, w13, w2, x)
        lin.forward(x, w)
        lin.backward(x, w, g)
        clip.norm()
        clip.clip(1.0)

    step()
    torch.cuda.synchronize()
    M.moe_profile_enable(True)
    step()
    M.moe_profile_enable(False)
    stages = M.moe_profile_collect()
    for name, calls in (("linear", 2), ("ffn_gate", 1), ("dense_backward", 2), ("grad_clip", 2)):
        assert stages[name][1] == calls and stages[name][0] > 0, (name, stages[name])
