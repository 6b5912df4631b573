"""Host-side argument checks of the dense operators.  Every call fails a check
(or is a size query or a no-op), so nothing reaches a CUDA API and the file
runs without a GPU."""
import ctypes

import pytest
import torch

from grouped_gemm_gating_b200 import build as B
from grouped_gemm_gating_b200 import moe as M

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
GiB = 1 << 30


def at(n):
    """Pointer n GiB up, so that different arguments never overlap."""
    return ctypes.c_void_p(n * GiB)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return M.load_library()


def linear(lib, **kw):
    T, K, N = kw.get("T", 4), kw.get("K", 64), kw.get("N", 32)
    return lib.moe_linear(kw.get("x", at(1)), kw.get("ldx", K), T, K, kw.get("w", at(2)), N, kw.get("bias"),
                          kw.get("res"), kw.get("ldr", N), kw.get("act", 0), kw.get("dtype", 0), kw.get("pre"),
                          kw.get("out", at(3)), kw.get("ldo", N), None, None)


def test_linear_checks(lib):
    assert linear(lib, T=-1) == INVALID
    assert linear(lib, K=0) == INVALID
    assert linear(lib, N=0) == INVALID
    assert linear(lib, K=60) == UNSUPPORTED
    assert linear(lib, N=36) == UNSUPPORTED
    assert linear(lib, K=1 << 18) == UNSUPPORTED
    assert linear(lib, T=(1 << 24) + 1) == UNSUPPORTED
    assert linear(lib, act=6) == INVALID
    assert linear(lib, act=-1) == INVALID
    assert linear(lib, dtype=2) == INVALID                       # fp32 matrices
    assert linear(lib, x=None) == INVALID
    assert linear(lib, w=None) == INVALID
    assert linear(lib, out=None) == INVALID
    assert linear(lib, x=ctypes.c_void_p(GiB + 8)) == INVALID    # 16-byte alignment
    assert linear(lib, bias=ctypes.c_void_p(4 * GiB + 2)) == INVALID
    assert linear(lib, ldx=56) == INVALID                        # rows overlap
    assert linear(lib, ldx=68) == UNSUPPORTED                    # stride not a multiple of 8
    assert linear(lib, res=at(4), ldr=24) == INVALID
    assert linear(lib, T=0, x=None, w=None, out=None) == OK


def test_linear_overlap(lib):
    assert linear(lib, out=at(1)) == INVALID                                  # out on x
    assert linear(lib, out=at(2)) == INVALID                                  # out on w
    assert linear(lib, out=ctypes.c_void_p(GiB + 64), ldo=32) == INVALID      # out inside x
    assert linear(lib, pre=at(3)) == INVALID                                  # pre on out
    assert linear(lib, pre=at(1)) == INVALID
    assert linear(lib, res=at(5), pre=at(5)) == INVALID
    assert linear(lib, bias=at(3)) == INVALID                                 # bias inside out
    assert linear(lib, res=at(3), ldr=40) == INVALID                          # same start, other stride
    assert linear(lib, res=ctypes.c_void_p(3 * GiB + 32)) == INVALID          # shifted
    # column slices of one buffer that run into each other
    assert linear(lib, ldx=96, out=ctypes.c_void_p(GiB + 2 * 56), ldo=96) == INVALID
    assert linear(lib, ldx=88, out=ctypes.c_void_p(GiB + 2 * 64), ldo=88) == INVALID   # wraps into the next row


def linear_bwd(lib, **kw):
    T, K, N = kw.get("T", 4), kw.get("K", 64), kw.get("N", 32)
    return lib.moe_linear_backward(kw.get("x", at(1)), kw.get("ldx", K), T, K, kw.get("w", at(2)), N,
                                   kw.get("act", 1), kw.get("dtype", 0), kw.get("pre", at(3)), kw.get("dout", at(4)),
                                   kw.get("ldd", N), kw.get("dxr"), kw.get("lddr", K), kw.get("dx", at(5)),
                                   kw.get("lddx", K), kw.get("dw", at(6)), kw.get("dbias"), kw.get("ws", at(7)),
                                   kw.get("wsb", 1 << 20), None, None)


def test_linear_backward_checks(lib):
    assert linear_bwd(lib, K=60) == UNSUPPORTED
    assert linear_bwd(lib, act=9) == INVALID
    assert linear_bwd(lib, dtype=2) == INVALID
    assert linear_bwd(lib, pre=None) == INVALID                  # an activation needs it
    assert linear_bwd(lib, dout=None) == INVALID
    assert linear_bwd(lib, x=None) == INVALID
    assert linear_bwd(lib, w=None) == INVALID
    assert linear_bwd(lib, dx=None, dw=None) == INVALID          # nothing to compute
    assert linear_bwd(lib, ws=None) == WORKSPACE
    assert linear_bwd(lib, wsb=64) == WORKSPACE
    assert linear_bwd(lib, dx=at(4)) == INVALID                  # dx on dout
    assert linear_bwd(lib, dw=at(2)) == INVALID                  # dw on w
    assert linear_bwd(lib, ws=at(1)) == INVALID                  # workspace on x
    assert linear_bwd(lib, dbias=at(6)) == INVALID               # dbias on dw
    assert linear_bwd(lib, dxr=ctypes.c_void_p(5 * GiB + 16)) == INVALID
    assert linear_bwd(lib, dxr=at(7)) == INVALID                 # added rows inside the workspace
    assert linear_bwd(lib, lddx=60) == INVALID


def ffn(lib, **kw):
    T, d, F = kw.get("T", 4), kw.get("d", 64), kw.get("F", 32)
    return lib.moe_ffn(kw.get("x", at(1)), kw.get("ldx", d), T, d, kw.get("w13", at(2)), kw.get("w2", at(3)), F,
                       kw.get("act", 1), kw.get("dtype", 0), kw.get("res"), kw.get("ldr", d), kw.get("pre"),
                       kw.get("h", at(4)), kw.get("out", at(5)), kw.get("ldo", d), None, None)


def test_ffn_checks(lib):
    assert ffn(lib, d=60) == UNSUPPORTED
    assert ffn(lib, F=36) == UNSUPPORTED
    assert ffn(lib, T=-1) == INVALID
    assert ffn(lib, act=6) == INVALID
    assert ffn(lib, dtype=2) == INVALID
    assert ffn(lib, h=None) == INVALID
    assert ffn(lib, out=None) == INVALID
    assert ffn(lib, w13=None) == INVALID
    assert ffn(lib, h=at(1)) == INVALID                          # h on x
    assert ffn(lib, pre=at(4)) == INVALID                        # pre on h
    assert ffn(lib, out=at(3)) == INVALID                        # out on w2
    assert ffn(lib, out=at(1), ldo=72) == INVALID                # x with another stride
    assert ffn(lib, out=ctypes.c_void_p(GiB + 16)) == INVALID    # x, shifted
    assert ffn(lib, T=0, x=None, h=None) == OK


def ffn_bwd(lib, **kw):
    T, d, F = kw.get("T", 4), kw.get("d", 64), kw.get("F", 32)
    return lib.moe_ffn_backward(kw.get("x", at(1)), kw.get("ldx", d), T, d, kw.get("w13", at(2)), kw.get("w2", at(3)),
                                F, kw.get("act", 1), kw.get("dtype", 0), kw.get("pre", at(4)), kw.get("dout", at(5)),
                                kw.get("ldd", d), kw.get("dxr"), kw.get("lddr", d), kw.get("dx", at(6)),
                                kw.get("lddx", d), kw.get("dw13", at(7)), kw.get("dw2", at(8)), kw.get("ws", at(9)),
                                kw.get("wsb", 1 << 20), None, None)


def test_ffn_backward_checks(lib):
    assert ffn_bwd(lib, d=60) == UNSUPPORTED
    assert ffn_bwd(lib, act=6) == INVALID
    assert ffn_bwd(lib, pre=None) == INVALID
    assert ffn_bwd(lib, dout=None) == INVALID
    assert ffn_bwd(lib, w2=None) == INVALID
    assert ffn_bwd(lib, dx=None, dw13=None, dw2=None) == INVALID
    assert ffn_bwd(lib, ws=None) == WORKSPACE
    assert ffn_bwd(lib, wsb=64) == WORKSPACE
    assert ffn_bwd(lib, dw13=at(2)) == INVALID
    assert ffn_bwd(lib, dw2=at(7)) == INVALID
    assert ffn_bwd(lib, dx=at(5)) == INVALID
    assert ffn_bwd(lib, dxr=ctypes.c_void_p(6 * GiB + 16)) == INVALID


def test_workspace_sizes(lib):
    assert M.moe_linear_backward_workspace_size(100, 64, 32, M.EPI_NONE) == 0
    n = M.moe_linear_backward_workspace_size(100, 64, 32, M.EPI_SILU)
    assert 100 * 32 * 2 <= n <= 100 * 32 * 2 + 512
    assert M.moe_linear_backward_workspace_size(100, 60, 32, M.EPI_SILU) == 0
    n = M.moe_ffn_backward_workspace_size(100, 64, 32)
    assert 100 * 3 * 32 * 2 <= n <= 100 * 3 * 32 * 2 + 768
    assert M.moe_ffn_backward_workspace_size(100, 64, 30) == 0
    assert M.moe_ffn_backward_workspace_size(-1, 64, 32) == 0
    assert lib.moe_grad_plan_size(0) == 0
    assert lib.moe_grad_plan_size(10) == 10 * lib.moe_grad_plan_size(1)


def plan(lib, src, numel, dtype, dst=None, plan_p=at(50), plan_b=1 << 20):
    n = len(src)
    chunks = ctypes.c_int64(0)
    return lib.moe_grad_plan((ctypes.c_void_p * n)(*src), None if dst is None else (ctypes.c_void_p * n)(*dst),
                             (ctypes.c_int64 * n)(*numel), (ctypes.c_int32 * n)(*dtype), n, plan_p, plan_b,
                             ctypes.byref(chunks), None)


def test_grad_plan_checks(lib):
    assert plan(lib, [GiB], [8], [3]) == INVALID                          # dtype
    assert plan(lib, [GiB], [-1], [0]) == INVALID
    assert plan(lib, [None], [8], [0]) == INVALID
    assert plan(lib, [GiB + 1], [8], [0]) == INVALID                      # element alignment
    assert plan(lib, [GiB + 2], [8], [2]) == INVALID
    assert plan(lib, [GiB], [8], [0], dst=[GiB + 8]) == INVALID           # shifted onto itself
    assert plan(lib, [GiB], [8], [0], dst=[None]) == INVALID
    assert plan(lib, [GiB, GiB], [8, 8], [0, 0]) == INVALID               # the same tensor twice, in place
    assert plan(lib, [GiB, GiB + 8], [8, 8], [0, 0]) == INVALID           # views that overlap
    assert plan(lib, [GiB, 2 * GiB], [8, 8], [0, 0], dst=[3 * GiB, 3 * GiB + 14]) == INVALID
    assert plan(lib, [GiB, 2 * GiB], [8, 8], [0, 0], dst=[3 * GiB, GiB]) == INVALID   # a target on another's source
    assert plan(lib, [2 * GiB, GiB], [8, (1 << 28) + 4], [0, 2], dst=[3 * GiB, GiB]) == INVALID  # in another target
    assert plan(lib, [GiB], [8], [0], plan_p=None) == WORKSPACE
    assert plan(lib, [GiB], [8], [0], plan_b=16) == WORKSPACE
    assert plan(lib, [GiB], [8], [0], plan_p=ctypes.c_void_p(GiB + 8)) == WORKSPACE
    c = ctypes.c_int64(0)
    assert lib.moe_grad_plan(None, None, None, None, 0, at(1), 64, ctypes.byref(c), None) == INVALID


def test_grad_clip_checks(lib):
    def clip(plan=at(1), n=1, chunks=1, kind=0, m=1.0, norm=at(2), ws=at(3), wsb=1 << 20):
        return lib.moe_grad_clip(plan, n, chunks, kind, m, norm, ws, wsb, None, None)
    assert clip(plan=None) == INVALID
    assert clip(n=0) == INVALID
    assert clip(chunks=-1) == INVALID
    assert clip(kind=2) == INVALID
    assert clip(m=0.0) == INVALID
    assert clip(m=-1.0) == INVALID
    assert clip(m=float("nan")) == INVALID
    assert clip(norm=None) == INVALID
    assert clip(norm=ctypes.c_void_p(GiB + 2)) == INVALID
    assert clip(ws=None) == WORKSPACE
    assert clip(wsb=8) == WORKSPACE
    assert lib.moe_grad_norm(None, 1, 1, 0, at(2), at(3), 1 << 20, None, None) == INVALID


def test_binding_refuses_cpu_tensors():
    x, w, o = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.bfloat16), \
        torch.zeros(4, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        M.moe_linear(x, w, o)
    with pytest.raises(ValueError):
        M.moe_ffn(x, torch.zeros(64, 64, dtype=torch.bfloat16), torch.zeros(64, 32, dtype=torch.bfloat16),
                  torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros_like(x))
    with pytest.raises(ValueError):
        M.GradClip([x])
    with pytest.raises(ValueError):
        M.GradClip([])


@pytest.mark.parametrize("train", [False, True])
def test_buffers_refuse_what_no_call_takes(lib, train):
    """A shape or activation that every call would refuse is refused when the
    buffers are made, before anything is allocated for it."""
    for T, K, N, act in ((4, 60, 32, 0), (4, 64, 36, 1), (-1, 64, 32, 0), (4, 1 << 18, 32, 0), ((1 << 24) + 1, 8, 8, 2),
                         (4, 64, 32, 6), (4, 64, 32, -1)):
        with pytest.raises(ValueError):
            M.LinearBuffers(T, K, N, act, train=train, device="cpu")
        with pytest.raises(ValueError):
            M.FFNBuffers(T, K, N, act, train=train, device="cpu")
    for T in (0, 4):  # shapes that calls take
        b = M.LinearBuffers(T, 64, 32, train=train, device="cpu")
        assert b.out.shape == (T, 32) and b.ws is None
        assert M.FFNBuffers(T, 64, 32, train=train, device="cpu").h.shape == (T, 32)
