"""Which kernel the dense operators' launches run on (plan_of in
dense_split.cuh), asked on the host: the large cases of the GPU tests have to
reach the CTA-pair kernel, the small ones the split kernel, so that refitted
constants cannot take a kernel out of the tests unseen."""
import os
import subprocess

import pytest

from grouped_gemm_gating_b200 import build as B
from test_gpu_activations import BACKWARD, FORWARD
from test_gpu_dense import FFN, FFN_BWD, FFN_BWD_PAIRS, LINEAR, LINEAR_BWD, LINEAR_BWD_PAIRS

PROGRAM = r"""
#include <algorithm>
#include <cstdio>
#include <cstring>
#include "dense_split.cuh"
using namespace moe;

constexpr int kSms = 148;

DenseProblem product(int major, int64_t M, int64_t N, int64_t K, int residual = 0) {
  DenseProblem p{};
  p.residual = residual ? &p : nullptr;  // only compared with null
  p.major = major;
  p.M = M;
  p.N = N;
  p.K = K;
  return p;
}
const char* kernel(const dense::Plan& p) { return p.split ? "split" : "pair"; }

// the plan of all products in one launch, and those of the two launches that
// may take its place
void gradients(DenseProblem* p, int n) {
  std::sort(p, p + n, [](const DenseProblem& a, const DenseProblem& b) { return a.K > b.K; });
  printf(" %s %s %s\n", kernel(dense::plan_of<kDenseLinear, kMajorAny>(p, n, kSms)),
         kernel(dense::plan_of<kDenseLinear, kMajorAny>(p, 1, kSms)),
         kernel(dense::plan_of<kDenseLinear, kMajorAny>(p + 1, n - 1, kSms)));
}

int main() {
  char op[32];
  long T, K, N;
  int r;
  while (scanf("%31s %ld %ld %ld %d", op, &T, &K, &N, &r) == 5) {
    if (!strcmp(op, "linear")) {
      DenseProblem p = product(kMajorKK, T, N, K, r);
      printf("%s\n", kernel(dense::plan_of<kDenseLinear, kMajorKK>(&p, 1, kSms)));
    } else if (!strcmp(op, "ffn")) {
      DenseProblem p = product(kMajorKK, T, N, K), q = product(kMajorKK, T, K, N, r);
      printf("%s %s\n", kernel(dense::plan_of<kDenseGate, kMajorKK>(&p, 1, kSms)),
             kernel(dense::plan_of<kDenseLinear, kMajorKK>(&q, 1, kSms)));
    } else if (!strcmp(op, "linear_backward")) {
      DenseProblem p[2] = {product(kMajorKN, T, K, N, r), product(kMajorMN, N, K, T)};
      gradients(p, 2);
    } else {
      DenseProblem dh = product(kMajorKN, T, N, K);
      printf("%s", kernel(dense::plan_of<kDenseGateGrad, kMajorKN>(&dh, 1, kSms)));
      DenseProblem p[3] = {product(kMajorKN, T, K, 2 * N, r), product(kMajorMN, 2 * N, K, T),
                           product(kMajorMN, K, N, T)};
      gradients(p, 3);
    }
  }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """plan(op, case) -> the kernels of its launches, in order."""
    src = tmp_path_factory.mktemp("plan") / "plan.cu"
    src.write_text(PROGRAM)
    exe = str(src.with_suffix(""))
    subprocess.run([B.nvcc_path(), *B.ARCH_FLAGS, "-std=c++17", "--expt-relaxed-constexpr", "-I", B.CSRC, "-I",
                    os.path.join(B.REPO_DIR, "include"), str(src), "-o", exe], check=True, capture_output=True)

    def ask(op, case):
        (T, K, N), residual = case[:3], case[4 if op.startswith("ffn") else 5]
        line = f"{op} {T} {K} {N} {int(residual)}\n"
        return subprocess.run([exe], input=line, capture_output=True, text=True, check=True).stdout.split()

    return ask


@pytest.mark.parametrize("case", LINEAR_BWD_PAIRS, ids=str)
def test_linear_backward_cases_on_pairs(plan, case):
    assert plan("linear_backward", case) == ["pair"] * 3


@pytest.mark.parametrize("case", FFN_BWD_PAIRS, ids=str)
def test_ffn_backward_cases_on_pairs(plan, case):
    assert plan("ffn_backward", case) == ["pair"] * 4


def test_forward_cases_reach_both_kernels(plan):
    for op, cases in (("linear", LINEAR), ("ffn", FFN)):
        small = [plan(op, c) for c in cases if c[0] <= 300]
        large = [plan(op, c) for c in cases if c[0] >= 4700]
        assert small and all(k == "split" for p in small for k in p), (op, small)
        assert len(large) >= 2 and all(p[0] == "pair" for p in large), (op, large)


def test_small_gradients_run_on_the_split_kernel(plan):
    for op, cases in (("linear_backward", LINEAR_BWD), ("ffn_backward", FFN_BWD)):
        for c in cases:
            if c[0] <= 300 and max(c[1:3]) <= 1100:
                assert set(plan(op, c)) == {"split"}, c


def test_activation_cases_reach_both_kernels(plan):
    for op, (small, large) in (("linear", FORWARD), ("ffn", FORWARD), ("ffn_backward", BACKWARD)):
        no_residual = ("silu", False, False)
        assert plan(op, small + no_residual)[0] == "split" and plan(op, large + no_residual)[0] == "pair", op
