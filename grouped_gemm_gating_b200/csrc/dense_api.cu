// C ABI of the dense operators: the linear layer, the gated feed-forward
// block and gradient clipping.  Argument checks, workspace layout and launch
// sequences; include/moe.h holds the contract of every entry point.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdlib>
#include <initializer_list>

#include "../../include/moe.h"
#include "dense.h"
#include "host.h"

using moe::aligned16;
using moe::DenseProblem;
using moe::finish;
using moe::kWsAlign;
using moe::num_sms_current_device;
using moe::round_up;
using moe::StageScope;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 24;
constexpr int kMaxCols = 1 << 17;
constexpr int64_t kMaxStride = int64_t(1) << 31;

enum Stage { kStLinear = 14, kStFfnGate = 15, kStGrad = 16, kStClip = 17 };

bool valid_act(moe_epi_act act) { return act >= MOE_EPI_NONE && act <= MOE_EPI_RELU2; }
bool valid_16bit(moe_dtype t) { return t == MOE_BF16 || t == MOE_FP16; }

moe_status check_size(int64_t T, int64_t a, int64_t b) {
  if (T < 0 || a < 1 || b < 1) return MOE_ERR_INVALID_ARG;
  if (T > kMaxRows || a > kMaxCols || b > kMaxCols || a % 8 || b % 8) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// A matrix of 16-bit values: rows x cols, rows ld elements apart.
struct Mat {
  const void* p;
  int64_t rows, cols, ld;
};

moe_status check_mat(const Mat& m) {
  if (m.p == nullptr || !aligned16(m.p) || m.ld < m.cols) return MOE_ERR_INVALID_ARG;
  if (m.ld % 8 || m.ld > kMaxStride) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Whether two matrices share an element.  Column slices of one row-major
// buffer interleave without sharing any.
bool share(const Mat& a, const Mat& b) {
  if (a.p == nullptr || b.p == nullptr || a.rows == 0 || b.rows == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  const uintptr_t a1 = a0 + 2 * static_cast<uintptr_t>((a.rows - 1) * a.ld + a.cols);
  const uintptr_t b1 = b0 + 2 * static_cast<uintptr_t>((b.rows - 1) * b.ld + b.cols);
  if (a1 <= b0 || b1 <= a0) return false;
  if (a.ld != b.ld) return true;
  const int64_t ld = a.ld;
  int64_t c = static_cast<int64_t>(b0 - a0) / 2 % ld;  // b's first column, counted from a's
  if (c < 0) c += ld;
  return c < a.cols || c + b.cols > ld;
}

bool same(const Mat& a, const Mat& b) { return a.p == b.p && (a.ld == b.ld || a.rows <= 1); }

moe_status check_all(std::initializer_list<Mat> ms) {
  moe_status worst = MOE_OK;
  for (const Mat& m : ms) {
    const moe_status st = check_mat(m);
    if (st == MOE_ERR_INVALID_ARG) return st;
    if (st != MOE_OK) worst = st;
  }
  return worst;
}

// No output shares memory with an input or another output.
bool disjoint(std::initializer_list<Mat> outs, std::initializer_list<Mat> ins) {
  for (const Mat* o = outs.begin(); o != outs.end(); ++o) {
    for (const Mat& i : ins)
      if (share(*o, i)) return false;
    for (const Mat* p = o + 1; p != outs.end(); ++p)
      if (share(*o, *p)) return false;
  }
  return true;
}

size_t linear_ws(int64_t T, int64_t N, moe_epi_act act) {  // dz; ws is rounded up to kWsAlign
  return act == MOE_EPI_NONE ? 0 : round_up(static_cast<size_t>(T) * N * 2, kWsAlign) + kWsAlign;
}

uint8_t* ws_base(void* ws) {
  return reinterpret_cast<uint8_t*>(round_up(reinterpret_cast<uintptr_t>(ws), kWsAlign));
}

// A gradient product: out [M, N] = a b over a contraction of K, with a [M, K]
// and b [K, N] (kMajorKN) or a [K, M] and b [K, N] (kMajorMN).
DenseProblem gradient(int major, moe_dtype dtype, int64_t M, int64_t N, int64_t K, const uint16_t* a, int64_t lda,
                      const uint16_t* b, int64_t ldb, uint16_t* out, int64_t ldo, int32_t* status) {
  DenseProblem p{};
  p.epi = moe::kDenseLinear;
  p.major = major;
  p.fp16 = dtype == MOE_FP16;
  p.act = MOE_EPI_NONE;
  p.M = M;
  p.N = N;
  p.K = K;
  p.a = a;
  p.lda = lda;
  p.b = b;
  p.ldb = ldb;
  p.out = out;
  p.ldo = ldo;
  p.status = status;
  return p;
}

// Whether a target shares memory with another tensor's source or target, or
// its own source shifted.  Intervals sorted by their start; a failed
// allocation reports -1.
struct Interval {
  uintptr_t start, end;
  bool target;
};
int targets_overlap(const void* const* src, void* const* dst, const int64_t* numel, const int32_t* dtype, int n) {
  Interval* v = static_cast<Interval*>(std::malloc(2 * static_cast<size_t>(n) * sizeof(Interval)));
  if (v == nullptr) return -1;
  int m = 0;
  for (int i = 0; i < n; ++i) {
    if (numel[i] == 0) continue;
    const uintptr_t bytes = static_cast<uintptr_t>(numel[i]) * (dtype[i] == MOE_FP32 ? 4 : 2);
    const uintptr_t s = reinterpret_cast<uintptr_t>(src[i]);
    const uintptr_t d = dst != nullptr ? reinterpret_cast<uintptr_t>(dst[i]) : s;
    v[m++] = {d, d + bytes, true};
    if (s != d) v[m++] = {s, s + bytes, false};
  }
  std::sort(v, v + m, [](const Interval& a, const Interval& b) { return a.start < b.start; });
  uintptr_t target_end = 0, source_end = 0;
  int found = 0;
  for (int i = 0; i < m && !found; ++i) {
    found = v[i].start < target_end || (v[i].target && v[i].start < source_end);
    uintptr_t* end = v[i].target ? &target_end : &source_end;
    if (v[i].end > *end) *end = v[i].end;
  }
  std::free(v);
  return found;
}

// One launch for all of them, the longest contraction first.
moe_status launch_gradients(DenseProblem* jobs, int n, int sms, cudaStream_t s, int launches) {
  if (n == 0) return finish(cudaSuccess, launches);
  std::sort(jobs, jobs + n, [](const DenseProblem& a, const DenseProblem& b) { return a.K > b.K; });
  const cudaError_t err = moe::launch_dense_grads(jobs, n, sms, s, &launches);
  return finish(err, launches);
}

Mat ws_mat(void* ws, size_t bytes) {  // the workspace as one row, for the overlap checks
  return {ws, ws != nullptr && bytes >= 2 ? 1 : 0, static_cast<int64_t>(bytes / 2), static_cast<int64_t>(bytes / 2)};
}

}  // namespace

extern "C" {

moe_status moe_linear(const uint16_t* x, int64_t ldx, int64_t T, int K, const uint16_t* w, int N,
                      const uint16_t* bias, const uint16_t* residual, int64_t ldr, moe_epi_act act, moe_dtype dtype,
                      uint16_t* pre, uint16_t* out, int64_t ldo, int32_t* dev_status, moe_stream_t stream) {
  moe_status st = check_size(T, K, N);
  if (st != MOE_OK) return st;
  if (!valid_act(act) || !valid_16bit(dtype)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return finish(cudaSuccess, 0);
  const Mat mx{x, T, K, ldx}, mw{w, N, K, K}, mo{out, T, N, ldo};
  const Mat mb{bias, bias ? 1 : 0, N, N}, mr{residual, residual ? T : 0, N, ldr}, mp{pre, pre ? T : 0, N, N};
  if ((st = check_all({mx, mw, mo})) != MOE_OK) return st;
  if (bias && (st = check_mat(mb)) != MOE_OK) return st;
  if (residual && (st = check_mat(mr)) != MOE_OK) return st;
  if (pre && (st = check_mat(mp)) != MOE_OK) return st;
  // out may be the residual itself.  The pair kernel fetches the residual of a
  // chunk (a box of 128 rows x 64 columns) some chunks ahead and stores the
  // chunk's result later: a box is read before it is written, and no two chunks
  // share an element.  In the split kernel a thread reads an element before it
  // writes it.
  if (!disjoint({mo, mp}, {mx, mw, mb}) || share(mp, mr) || (share(mo, mr) && !same(mo, mr)))
    return MOE_ERR_INVALID_ARG;
  const int sms = num_sms_current_device();
  if (sms <= 0) return MOE_ERR_CUDA;
  DenseProblem p{};
  p.epi = moe::kDenseLinear;
  p.major = moe::kMajorKK;
  p.fp16 = dtype == MOE_FP16;
  p.act = act;
  p.M = T;
  p.N = N;
  p.K = K;
  p.a = x;
  p.lda = ldx;
  p.b = w;
  p.ldb = K;
  p.bias = bias;
  p.residual = residual;
  p.ldr = ldr;
  p.out = out;
  p.ldo = ldo;
  p.pre = pre;
  p.ldp = N;
  p.status = dev_status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  StageScope scope(kStLinear, s);
  int launches = 0;
  const cudaError_t err = moe::launch_dense_linear(p, sms, s, &launches);
  return finish(err, launches);
}

size_t moe_linear_backward_workspace_size(int64_t T, int K, int N, moe_epi_act act) {
  if (check_size(T, K, N) != MOE_OK || !valid_act(act)) return 0;
  return linear_ws(T, N, act);
}

moe_status moe_linear_backward(const uint16_t* x, int64_t ldx, int64_t T, int K, const uint16_t* w, int N,
                               moe_epi_act act, moe_dtype dtype, const uint16_t* pre, const uint16_t* dout,
                               int64_t ldd, const uint16_t* dx_residual, int64_t lddr, uint16_t* dx, int64_t lddx,
                               uint16_t* dw, uint16_t* dbias, void* ws, size_t ws_bytes, int32_t* dev_status,
                               moe_stream_t stream) {
  moe_status st = check_size(T, K, N);
  if (st != MOE_OK) return st;
  if (!valid_act(act) || !valid_16bit(dtype)) return MOE_ERR_INVALID_ARG;
  if (dx == nullptr && dw == nullptr && dbias == nullptr) return MOE_ERR_INVALID_ARG;
  const bool has_act = act != MOE_EPI_NONE;
  const Mat mx{x, T, K, ldx}, mw{w, N, K, K}, md{dout, T, N, ldd}, mp{pre, has_act ? T : 0, N, N};
  const Mat mdx{dx, dx ? T : 0, K, lddx}, mdw{dw, dw ? N : 0, K, K}, mdb{dbias, dbias ? 1 : 0, N, N};
  const Mat mr{dx_residual, dx_residual && dx ? T : 0, K, lddr};
  if (T > 0) {
    if ((st = check_mat(md)) != MOE_OK) return st;
    if (dw && (st = check_mat(mx)) != MOE_OK) return st;
    if (dx && (st = check_all({mw, mdx})) != MOE_OK) return st;
    if (has_act && (st = check_mat(mp)) != MOE_OK) return st;
    if (dx && dx_residual && (st = check_mat(mr)) != MOE_OK) return st;
  }
  if (dw && (st = check_mat(mdw)) != MOE_OK) return st;
  if (dbias && (st = check_mat(mdb)) != MOE_OK) return st;
  const size_t need = linear_ws(T, N, act);
  if (T > 0 && need > 0 && (ws == nullptr || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  const Mat mws = ws_mat(T > 0 && need > 0 ? ws : nullptr, ws_bytes);
  if (!disjoint({mdx, mdw, mdb, mws}, {mx, mw, md, mp}) || share(mr, mdw) || share(mr, mdb) || share(mr, mws) ||
      (share(mr, mdx) && !same(mr, mdx)))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  StageScope scope(kStGrad, s);
  cudaError_t err = cudaSuccess;
  int launches = 0;
  if (T == 0) {  // a sum over no rows
    if (dw) err = cudaMemsetAsync(dw, 0, static_cast<size_t>(N) * K * 2, s);
    if (err == cudaSuccess && dbias) err = cudaMemsetAsync(dbias, 0, static_cast<size_t>(N) * 2, s);
    return finish(err, 0);
  }
  const int sms = num_sms_current_device();
  if (sms <= 0) return MOE_ERR_CUDA;
  const uint16_t* dz = dout;
  int64_t ldz = ldd;
  if (has_act || dbias) {
    moe::DzArgs a{};
    a.dout = dout;
    a.ldd = ldd;
    a.pre = has_act ? pre : nullptr;
    a.ldp = N;
    a.T = T;
    a.N = N;
    a.act = act;
    a.fp16 = dtype == MOE_FP16;
    a.dz = has_act ? reinterpret_cast<uint16_t*>(ws_base(ws)) : nullptr;
    a.dbias = dbias;
    err = moe::launch_dz(a, s, &launches);
    if (err != cudaSuccess) return MOE_ERR_CUDA;
    if (has_act) {
      dz = a.dz;
      ldz = N;
    }
  }
  DenseProblem jobs[2];
  int n = 0;
  auto job = [&](int major, int64_t M, int64_t K2, const uint16_t* b, int64_t ldb, uint16_t* out, int64_t ldo) {
    jobs[n++] = gradient(major, dtype, M, K, K2, dz, ldz, b, ldb, out, ldo, dev_status);
  };
  if (dx) {
    job(moe::kMajorKN, T, N, w, K, dx, lddx);
    jobs[0].residual = dx_residual;
    jobs[0].ldr = lddr;
  }
  if (dw) job(moe::kMajorMN, N, T, x, ldx, dw, K);
  return launch_gradients(jobs, n, sms, s, launches);
}

moe_status moe_ffn(const uint16_t* x, int64_t ldx, int64_t T, int d, const uint16_t* w13, const uint16_t* w2, int F,
                   moe_epi_act act, moe_dtype dtype, const uint16_t* residual, int64_t ldr, uint16_t* pre,
                   uint16_t* h, uint16_t* out, int64_t ldo, int32_t* dev_status, moe_stream_t stream) {
  moe_status st = check_size(T, d, F);
  if (st != MOE_OK) return st;
  if (!valid_act(act) || !valid_16bit(dtype)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return finish(cudaSuccess, 0);
  const int64_t F2 = 2 * static_cast<int64_t>(F);
  const Mat mx{x, T, d, ldx}, m13{w13, F2, d, d}, m2{w2, d, F, F}, mh{h, T, F, F}, mo{out, T, d, ldo};
  const Mat mr{residual, residual ? T : 0, d, ldr}, mp{pre, pre ? T : 0, F2, F2};
  if ((st = check_all({mx, m13, m2, mh, mo})) != MOE_OK) return st;
  if (residual && (st = check_mat(mr)) != MOE_OK) return st;
  if (pre && (st = check_mat(mp)) != MOE_OK) return st;
  // The second kernel reads the residual (which may be x) and writes out
  // while no tile of the first is left: out may be the residual or x itself.
  if (!disjoint({mh, mp, mo}, {m13, m2}) || !disjoint({mh, mp}, {mx, mr}) || (share(mo, mr) && !same(mo, mr)) ||
      (share(mo, mx) && !same(mo, mx)))
    return MOE_ERR_INVALID_ARG;
  const int sms = num_sms_current_device();
  if (sms <= 0) return MOE_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DenseProblem p{};
  p.epi = moe::kDenseGate;
  p.major = moe::kMajorKK;
  p.fp16 = dtype == MOE_FP16;
  p.act = act;
  p.M = T;
  p.N = F;
  p.K = d;
  p.a = x;
  p.lda = ldx;
  p.b = w13;
  p.ldb = d;
  p.out = h;
  p.ldo = F;
  p.pre = pre;
  p.ldp = F2;
  p.status = dev_status;
  cudaError_t err;
  int launches = 0;
  {
    StageScope scope(kStFfnGate, s);
    err = moe::launch_dense_gate(p, sms, s, &launches);
  }
  if (err != cudaSuccess) return MOE_ERR_CUDA;
  p.epi = moe::kDenseLinear;
  p.act = MOE_EPI_NONE;
  p.b_ready = 1;  // the gate/up kernel, which waited for all work before it, does not write w2
  p.N = d;
  p.K = F;
  p.a = h;
  p.lda = F;
  p.b = w2;
  p.ldb = F;
  p.residual = residual;
  p.ldr = ldr;
  p.out = out;
  p.ldo = ldo;
  p.pre = nullptr;
  {
    StageScope scope(kStLinear, s);
    err = moe::launch_dense_linear(p, sms, s, &launches);
  }
  return finish(err, launches);
}

size_t moe_ffn_backward_workspace_size(int64_t T, int d, int F) {
  if (check_size(T, d, F) != MOE_OK) return 0;
  return round_up(static_cast<size_t>(T) * 2 * F * 2, kWsAlign) + round_up(static_cast<size_t>(T) * F * 2, kWsAlign) +
         kWsAlign;
}

moe_status moe_ffn_backward(const uint16_t* x, int64_t ldx, int64_t T, int d, const uint16_t* w13, const uint16_t* w2,
                            int F, moe_epi_act act, moe_dtype dtype, const uint16_t* pre, const uint16_t* dout,
                            int64_t ldd, const uint16_t* dx_residual, int64_t lddr, uint16_t* dx, int64_t lddx,
                            uint16_t* dw13, uint16_t* dw2, void* ws, size_t ws_bytes, int32_t* dev_status,
                            moe_stream_t stream) {
  moe_status st = check_size(T, d, F);
  if (st != MOE_OK) return st;
  if (!valid_act(act) || !valid_16bit(dtype)) return MOE_ERR_INVALID_ARG;
  if (dx == nullptr && dw13 == nullptr && dw2 == nullptr) return MOE_ERR_INVALID_ARG;
  const int64_t F2 = 2 * static_cast<int64_t>(F);
  const Mat mx{x, T, d, ldx}, m13{w13, F2, d, d}, m2{w2, d, F, F}, mp{pre, T, F2, F2}, md{dout, T, d, ldd};
  const Mat mdx{dx, dx ? T : 0, d, lddx}, md13{dw13, dw13 ? F2 : 0, d, d}, md2{dw2, dw2 ? d : 0, F, F};
  const Mat mr{dx_residual, dx_residual && dx ? T : 0, d, lddr};
  if (T > 0) {
    if ((st = check_all({m2, mp, md})) != MOE_OK) return st;
    if (dw13 && (st = check_mat(mx)) != MOE_OK) return st;
    if (dx && (st = check_all({m13, mdx})) != MOE_OK) return st;
    if (dx && dx_residual && (st = check_mat(mr)) != MOE_OK) return st;
  }
  if (dw13 && (st = check_mat(md13)) != MOE_OK) return st;
  if (dw2 && (st = check_mat(md2)) != MOE_OK) return st;
  const size_t need = moe_ffn_backward_workspace_size(T, d, F);
  if (T > 0 && (ws == nullptr || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  const Mat mws = ws_mat(T > 0 ? ws : nullptr, ws_bytes);
  if (!disjoint({mdx, md13, md2, mws}, {mx, m13, m2, mp, md}) || share(mr, md13) || share(mr, md2) || share(mr, mws) ||
      (share(mr, mdx) && !same(mr, mdx)))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  StageScope scope(kStGrad, s);
  cudaError_t err = cudaSuccess;
  if (T == 0) {
    if (dw13) err = cudaMemsetAsync(dw13, 0, static_cast<size_t>(F2) * d * 2, s);
    if (err == cudaSuccess && dw2) err = cudaMemsetAsync(dw2, 0, static_cast<size_t>(F) * d * 2, s);
    return finish(err, 0);
  }
  const int sms = num_sms_current_device();
  if (sms <= 0) return MOE_ERR_CUDA;
  uint8_t* base = ws_base(ws);
  uint16_t* da = reinterpret_cast<uint16_t*>(base);
  uint16_t* h = reinterpret_cast<uint16_t*>(base + round_up(static_cast<size_t>(T) * F2 * 2, kWsAlign));
  int launches = 0;
  DenseProblem p{};
  p.fp16 = dtype == MOE_FP16;
  p.status = dev_status;
  // dh = dout W2, turned into [dg | du] and h on its way out
  p.epi = moe::kDenseGateGrad;
  p.major = moe::kMajorKN;
  p.act = act;
  p.M = T;
  p.N = F;
  p.K = d;
  p.a = dout;
  p.lda = ldd;
  p.b = w2;
  p.ldb = F;
  p.out = da;
  p.ldo = F2;
  p.pre = const_cast<uint16_t*>(pre);
  p.ldp = F2;
  p.out2 = h;
  err = moe::launch_dense_gate_grad(p, sms, s, &launches);
  if (err != cudaSuccess) return MOE_ERR_CUDA;
  DenseProblem jobs[3];
  int n = 0;
  if (dx) {
    jobs[n] = gradient(moe::kMajorKN, dtype, T, d, F2, da, F2, w13, d, dx, lddx, dev_status);
    jobs[n].residual = dx_residual;
    jobs[n++].ldr = lddr;
  }
  if (dw13) jobs[n++] = gradient(moe::kMajorMN, dtype, F2, d, T, da, F2, x, ldx, dw13, d, dev_status);
  if (dw2) jobs[n++] = gradient(moe::kMajorMN, dtype, d, F, T, dout, ldd, h, F, dw2, F, dev_status);
  return launch_gradients(jobs, n, sms, s, launches);
}

size_t moe_grad_plan_size(int n) {
  return n < 1 || n > (1 << 24) ? 0 : static_cast<size_t>(n) * sizeof(moe::ClipEntry);
}

size_t moe_grad_workspace_size(void) { return moe::kClipMaxBlocks * sizeof(double); }

moe_status moe_grad_plan(const void* const* src, void* const* dst, const int64_t* numel, const int32_t* dtype, int n,
                         void* plan, size_t plan_bytes, int64_t* chunks, moe_stream_t stream) {
  if (n < 1 || src == nullptr || numel == nullptr || dtype == nullptr || chunks == nullptr) return MOE_ERR_INVALID_ARG;
  if (n > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  if (plan == nullptr || plan_bytes < moe_grad_plan_size(n) || !aligned16(plan)) return MOE_ERR_WORKSPACE;
  int64_t total = 0;
  for (int i = 0; i < n; ++i) {
    if (dtype[i] != MOE_BF16 && dtype[i] != MOE_FP16 && dtype[i] != MOE_FP32) return MOE_ERR_INVALID_ARG;
    if (numel[i] < 0 || numel[i] > (int64_t(1) << 40)) return MOE_ERR_INVALID_ARG;
    if (numel[i] == 0) continue;
    const uintptr_t size = dtype[i] == MOE_FP32 ? 4 : 2;
    const uintptr_t s = reinterpret_cast<uintptr_t>(src[i]);
    const uintptr_t d = dst != nullptr ? reinterpret_cast<uintptr_t>(dst[i]) : s;
    if (s == 0 || d == 0 || s % size || d % size) return MOE_ERR_INVALID_ARG;
    total += (numel[i] + moe::kClipChunk - 1) / moe::kClipChunk;
  }
  if (targets_overlap(src, dst, numel, dtype, n) != 0) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int launches = 0;
  int64_t first = 0;
  constexpr int kPart = 96;
  moe::ClipEntry part[kPart];
  for (int i = 0; i < n; i += kPart) {
    const int m = n - i < kPart ? n - i : kPart;
    for (int j = 0; j < m; ++j) {
      const int k = i + j;
      part[j] = {src[k], dst != nullptr ? dst[k] : const_cast<void*>(src[k]), numel[k], first, dtype[k]};
      first += (numel[k] + moe::kClipChunk - 1) / moe::kClipChunk;
    }
    if (moe::launch_clip_plan(part, m, static_cast<moe::ClipEntry*>(plan) + i, s, &launches) != cudaSuccess)
      return MOE_ERR_CUDA;
  }
  *chunks = total;
  return finish(cudaSuccess, launches);
}

}  // extern "C"

namespace {

moe_status check_grad(const void* plan, int n, int64_t chunks, moe_norm_type type, const float* norm, const void* ws,
                      size_t ws_bytes) {
  if (n < 1 || n > (1 << 24) || chunks < 0 || plan == nullptr || !aligned16(plan) || norm == nullptr ||
      (reinterpret_cast<uintptr_t>(norm) & 3u))
    return MOE_ERR_INVALID_ARG;
  if (type != MOE_NORM_L2 && type != MOE_NORM_MAX) return MOE_ERR_INVALID_ARG;
  if (ws == nullptr || ws_bytes < moe_grad_workspace_size() || !aligned16(ws)) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_grad_norm(const void* plan, int n, int64_t chunks, moe_norm_type type, float* norm, void* ws,
                         size_t ws_bytes, int32_t* dev_status, moe_stream_t stream) {
  moe_status st = check_grad(plan, n, chunks, type, norm, ws, ws_bytes);
  if (st != MOE_OK) return st;
  const int sms = num_sms_current_device();
  if (sms <= 0) return MOE_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  StageScope scope(kStClip, s);
  int launches = 0;
  cudaError_t err = moe::launch_clip_norm(static_cast<const moe::ClipEntry*>(plan), n, chunks, type,
                                          static_cast<double*>(ws), norm, true, dev_status, sms, s, &launches);
  return finish(err, launches);
}

moe_status moe_grad_clip(const void* plan, int n, int64_t chunks, moe_norm_type type, float max_norm, float* norm,
                         void* ws, size_t ws_bytes, int32_t* dev_status, moe_stream_t stream) {
  moe_status st = check_grad(plan, n, chunks, type, norm, ws, ws_bytes);
  if (st != MOE_OK) return st;
  if (!(max_norm > 0.0f)) return MOE_ERR_INVALID_ARG;
  const int sms = num_sms_current_device();
  if (sms <= 0) return MOE_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  StageScope scope(kStClip, s);
  int launches = 0;
  const moe::ClipEntry* p = static_cast<const moe::ClipEntry*>(plan);
  cudaError_t err = moe::launch_clip_norm(p, n, chunks, type, static_cast<double*>(ws), norm, false, dev_status, sms, s,
                                          &launches);
  if (err != cudaSuccess) return MOE_ERR_CUDA;
  err = moe::launch_clip_scale(p, n, chunks, type, static_cast<double>(max_norm), static_cast<const double*>(ws), norm,
                               dev_status, sms, s, &launches);
  return finish(err, launches);
}

}  // extern "C"
