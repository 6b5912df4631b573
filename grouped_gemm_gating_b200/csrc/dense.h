// Host-visible interface of the dense operators' kernels.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/moe.h"

namespace moe {

// What the epilogue of one dense GEMM does with its fp32 sums.
enum DenseEpi : int {
  kDenseLinear = 0,    // out = act(sum + bias) + residual; optionally pre = sum + bias
  kDenseGate = 1,      // sums [g | u]: out = act(g) * u; optionally pre = [g | u]
  kDenseGateGrad = 2   // sum = dh: out = [dh u act'(g) | dh act(g)], out2 = act(g) u, from pre = [g | u]
};

// How the two operands lie in memory: K contiguous (rows of the contraction)
// or their own index contiguous (MN-major).
enum DenseMajor : int {
  kMajorKK = 0,   // A K, B K
  kMajorKN = 1,   // A K, B MN
  kMajorMN = 2,   // A MN, B MN
  kMajorAny = 3   // kernels only: kMajorKN and kMajorMN problems together in one launch
};
constexpr int kMaxJobs = 3;  // problems of one launch

// One GEMM: sum[m, n] = sum_k A[m, k] B[n, k], m < M, n < N.  16-bit values
// (bf16, or fp16 with fp16 = 1), strides in elements.
struct DenseProblem {
  int epi, major;
  int fp16;
  int act;               // moe_epi_act
  int64_t M, N, K;       // kDenseGate: N is the width of h (B has 2 N rows)
  const void* a;
  int64_t lda;           // kMajorMN: A is [K, M], else [M, K]
  const void* b;
  int64_t ldb;           // kMajorKK: B is [N, K] (gate: [2 N, K]), else [K, N]
  const void* bias;      // [N] or null
  const void* residual;  // [M, N] or null
  int64_t ldr;
  void* out;
  int64_t ldo;
  void* pre;             // linear: [M, N]; gate, gate-grad: [M, 2 N]; row stride ldp; null: not kept
  int64_t ldp;
  void* out2;            // gate-grad: h [M, N], row stride N
  int b_ready;           // b is not written by the kernel before this one in the stream
  int32_t* status;
};
cudaError_t launch_dense_linear(const DenseProblem& p, int num_sms, cudaStream_t stream, int* launches);
cudaError_t launch_dense_gate(const DenseProblem& p, int num_sms, cudaStream_t stream, int* launches);
cudaError_t launch_dense_gate_grad(const DenseProblem& p, int num_sms, cudaStream_t stream, int* launches);
// Up to kMaxJobs independent kMajorKN / kMajorMN products (gradients: no
// bias, activation or pre), the longest contraction first, in one launch or
// two.
cudaError_t launch_dense_grads(const DenseProblem* p, int n, int num_sms, cudaStream_t stream, int* launches);

// dz = dout * act'(pre) (pre null: dz is dout and is not written) and, with
// dbias, dbias[n] = sum_t dz[t, n].
struct DzArgs {
  const uint16_t* dout;
  int64_t ldd;
  const uint16_t* pre;  // [T, N], row stride ldp
  int64_t ldp;
  int64_t T, N;
  int act, fp16;
  uint16_t* dz;         // [T, N]
  uint16_t* dbias;      // [N] or null
};
cudaError_t launch_dz(const DzArgs& a, cudaStream_t stream, int* launches);

// Global norm over many tensors and their scaling (clip.cu).  A plan holds
// one entry per tensor; tensors are cut into chunks of kClipChunk elements
// and numbered through.
constexpr int kClipChunk = 2048;
struct ClipEntry {
  const void* src;
  void* dst;
  int64_t numel;
  int64_t first;   // index of the tensor's first chunk
  int64_t dtype;   // moe_dtype
};
constexpr int kClipMaxBlocks = 1024;
cudaError_t launch_clip_plan(const ClipEntry* entries, int n, ClipEntry* plan, cudaStream_t stream, int* launches);
// partial: kClipMaxBlocks doubles; norm: one float.
cudaError_t launch_clip_norm(const ClipEntry* plan, int n, int64_t chunks, int norm_type, double* partial, float* norm,
                             bool finish, int32_t* status, int num_sms, cudaStream_t stream, int* launches);
cudaError_t launch_clip_scale(const ClipEntry* plan, int n, int64_t chunks, int norm_type, double max_norm,
                              const double* partial, float* norm, int32_t* status, int num_sms, cudaStream_t stream,
                              int* launches);

}  // namespace moe
