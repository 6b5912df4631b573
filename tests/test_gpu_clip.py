"""GPU parity of the global gradient norm and clipping against the oracle."""
import math

import numpy as np
import pytest
import torch

from dense_testlib import TINY, U, np64
from grouped_gemm_gating_b200 import moe as M
from oracle import dense_oracle as D

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
U32 = {**U, FP: 2.0 ** -24}
TINY32 = {**TINY, FP: 2.0 ** -150}


def tensors(sizes, dtypes, seed=0, std=1.0, shift=0):
    """Tensors cut from one buffer per type, `shift` elements in (any
    alignment), NaN between them."""
    gen = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        dt = dtypes[i % len(dtypes)]
        buf = torch.full((n + shift + 9,), float("nan"), dtype=dt, device="cuda")
        buf[shift:shift + n] = (torch.randn(n, generator=gen) * std).to(dt).cuda()
        out.append(buf[shift:shift + n])
    return out


def check_clip(grads, outs, plan, max_norm, norm_type="l2"):
    before = [np64(g) for g in grads]
    n, want = D.clip(before, max_norm, norm_type)
    got = plan.clip(max_norm, M.NORM_L2 if norm_type == "l2" else M.NORM_MAX)
    torch.cuda.synchronize()
    assert M.moe_read_status(plan.status) == 0
    # squares to 2^-21 in groups of eight, the rest in 64 bits, one rounding
    # to fp32 (a subnormal norm's step is 2^-149)
    assert abs(float(got) - n) <= 2.0 ** -21 * n + 2.0 ** -149
    for o, ref, g in zip(outs, want, before):
        a = np64(o)
        dt = o.dtype
        # c within 2^-20 (the norm's error and its own rounding), a product's
        # rounding in fp32, the output's rounding
        tol = (2.0 ** -20 + 2.0 ** -24) * np.abs(ref) + U32[dt] * np.abs(ref) * 1.0001 + TINY32[dt] + 2.0 ** -149
        assert (np.abs(a - ref) <= tol).all()
        if n + 1e-6 <= max_norm * (1 - 2.0 ** -19):
            assert np.array_equal(a, g)


SIZES = [[1], [7], [8, 3, 0, 5], [2048], [2049, 1], [4095, 4097, 0, 0], [100_003], [300_000, 17, 2047, 65_536, 1, 9],
         [1] * 300, [0, 0, 5, 0]]


@pytest.mark.parametrize("sizes", SIZES, ids=[str(len(s)) + "x" + str(max(s)) for s in SIZES])
@pytest.mark.parametrize("dtypes", [(BF,), (FP,), (HF, FP, BF)], ids=["bf16", "fp32", "mixed"])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_clip_to_other_buffers(sizes, dtypes, shift):
    grads = tensors(sizes, dtypes, 1, shift=shift)
    outs = tensors(sizes, dtypes, 2, shift=(shift * 2) % 5)
    keep = [g.clone() for g in grads]
    plan = M.GradClip(grads, outs)
    check_clip(grads, outs, plan, 0.5)
    check_clip(grads, outs, plan, 1e9)
    check_clip(grads, outs, plan, 0.25, "max")
    for g, k in zip(grads, keep):
        assert torch.equal(g, k)
    for o in outs:  # what lies around the targets is as it was
        b = o._base
        assert int(torch.isnan(b).sum()) == b.numel() - o.numel()


@pytest.mark.parametrize("shift", [0, 1])
def test_clip_in_place(shift):
    grads = tensors([5000, 33, 70_000], (BF, FP), 3, shift=shift)
    plan = M.GradClip(grads)
    check_clip(grads, grads, plan, 1e9)      # nothing to do
    check_clip(grads, grads, plan, 2.0)
    again = float(plan.norm())
    # each value is off by u of itself at most, so is the norm
    assert abs(again - 2.0) <= 2.0 * 2.0 ** -8 + 1e-5


@pytest.mark.parametrize("std", [1e-38, 1e-30, 1e-22, 1e-15, 1e15, 1e18, 1e30])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_norm_of_tiny_and_large_gradients(std, dtype):
    grads = tensors([10_000, 3], (dtype,), 4, std)
    plan = M.GradClip(grads, [torch.empty_like(g) for g in grads])
    n = D.grad_norm([np64(g) for g in grads])
    assert abs(float(plan.norm()) - n) <= 2.0 ** -21 * n + 2.0 ** -149
    check_clip(grads, plan._held[1], plan, 1.0)


def test_no_elements():
    grads = [torch.empty(0, dtype=BF, device="cuda"), torch.empty((3, 0), device="cuda")]
    plan = M.GradClip(grads)
    assert float(plan.clip(1.0)) == 0.0 and float(plan.norm()) == 0.0
    assert M.moe_read_status(plan.status) == 0


def test_one_source_for_two_targets():
    g = tensors([3000], (FP,), 8)[0]
    a, b = torch.empty_like(g), torch.empty_like(g)
    check_clip([g, g], [a, b], M.GradClip([g, g], [a, b]), 1.0)


def test_more_elements_than_32_bits_count():
    """2^31 + 5 bf16 values: the last ones are counted and scaled."""
    g = torch.zeros((1 << 31) + 5, dtype=BF, device="cuda")
    g[-3:] = 2.0
    g[0] = 2.0
    plan = M.GradClip([g])
    assert abs(float(plan.clip(1.0)) - 4.0) <= 1e-6
    assert g[-3:].tolist() == [0.5] * 3 and float(g[0]) == 0.5 and float(g[1 << 30]) == 0.0


def test_zero_gradients():
    grads = [torch.zeros(5000, dtype=BF, device="cuda"), torch.zeros(3, device="cuda")]
    plan = M.GradClip(grads)
    assert float(plan.clip(1.0)) == 0.0
    assert float(plan.norm(M.NORM_MAX)) == 0.0
    assert not any(bool(g.any()) for g in grads)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("kind", [M.NORM_L2, M.NORM_MAX])
@pytest.mark.parametrize("where", [0, 4999])
def test_nonfinite_norm_is_flagged_and_scales_nothing(bad, kind, where):
    grads = tensors([5000, 40], (FP, BF), 5)
    grads[0][where] = bad
    keep = [g.clone() for g in grads]
    plan = M.GradClip(grads)
    norm = float(plan.clip(1.0, kind))
    assert math.isnan(norm) if math.isnan(bad) else math.isinf(norm)
    assert M.status_name(M.moe_read_status(plan.status)) == "MOE_ERR_NONFINITE"
    for g, k in zip(grads, keep):
        assert torch.equal(torch.nan_to_num(g), torch.nan_to_num(k))


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("value,n,finite", [(3e38, 2, False), (3e38, 1, True), (3e38, 5000, False), (2e38, 2, True)])
def test_norm_beyond_fp32(dtype, value, n, finite):
    """Finite gradients whose L2 norm fp32 cannot hold: reported as infinite,
    flagged and not scaled.  The largest norms that it can hold still scale."""
    g = torch.zeros(6000, dtype=dtype, device="cuda")
    g[100:100 + n] = value
    keep = g.clone()
    v = float(g[100])
    for call in ("norm", "clip"):
        plan = M.GradClip([g])
        norm = float(plan.norm() if call == "norm" else plan.clip(1e38))
        if finite:
            assert M.moe_read_status(plan.status) == 0
            assert abs(norm - v * math.sqrt(n)) <= 2.0 ** -21 * norm
        else:
            assert norm == math.inf
            assert M.status_name(M.moe_read_status(plan.status)) == "MOE_ERR_NONFINITE"
        if call == "clip" and finite:
            want = keep.double() * (1e38 / (v * math.sqrt(n)))
            # c, its product and the output's rounding
            assert bool(((g.double() - want).abs() <= (2.0 ** -20 + U32[dtype] * 1.0001) * want).all())
        else:
            assert torch.equal(g, keep)
    assert float(M.GradClip([keep]).norm(M.NORM_MAX)) == v


def test_same_on_every_call_and_in_a_graph():
    grads = tensors([200_001, 3000, 5], (BF, FP), 6)
    outs = [torch.empty_like(g) for g in grads]
    plan = M.GradClip(grads, outs)
    n = float(plan.clip(1.0))
    want = [o.clone() for o in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.clip(1.0)
    for _ in range(3):
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert float(plan.total_norm) == n
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        plan.clip(1.0)
    torch.cuda.synchronize()
    assert float(plan.total_norm) == n and all(torch.equal(a, b) for a, b in zip(outs, want))


def test_refusals():
    a = torch.zeros(100, device="cuda")
    for grads, outs in (([a.to(torch.float64)], None), ([a[::2]], None), ([a], [a[:50]]), ([a], [a.to(BF)]),
                        ([a], [a.cpu()]), ([a[:50]], [a[1:51]]), ([a, a], None),
                        ([a[:60], a[50:]], None)):
        with pytest.raises((ValueError, M.MoEError)):
            M.GradClip(grads, outs)
    plan = M.GradClip([a])
    for m in (0.0, -1.0, float("nan")):
        with pytest.raises(M.MoEError):
            plan.clip(m)
