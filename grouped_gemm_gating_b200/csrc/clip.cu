// Global norm over many gradient tensors and clipping to it.
//
//   norm = sqrt(sum_i g_i^2)  or  max_i |g_i|   over all elements of all tensors
//   g_i <- c g_i,  c = min(1, max_norm / (norm + 1e-6))
//
// Bound by memory: the norm needs every gradient before the first one can be
// scaled, so the tensors are read twice and written once unless they stay in
// L2 between the two kernels.  Tensors are numbered through in chunks of
// kClipChunk elements; a block takes one contiguous run of chunks (finding
// its first tensor once, by binary search) and goes through it front to back
// for the norm, back to front for the scaling, so that what the first kernel
// read last is what the second reads first.
//
// Sums: eight squares in fp32 (their relative error is below 2^-21, and
// averages out), then 64 bits throughout.  A group whose fp32 sum leaves the
// range where its squares are normal numbers is summed again in 64 bits, so
// neither large nor tiny gradients overflow or vanish.  Every block's sum is
// one partial; both kernels add the partials in a fixed order: the norm is
// the same on every call.
#include "common.cuh"
#include "dense.h"
#include "epilogue.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 4;

__device__ __forceinline__ void unpack_vec(uint4 v, int dtype, float (&f)[8], int* n) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (dtype == MOE_FP32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(w[i]);
#pragma unroll
    for (int i = 4; i < 8; ++i) f[i] = 0.0f;
    *n = 4;
    return;
  }
  *n = 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = split(dtype == MOE_FP16 ? unpack2<true>(w[i]) : unpack2<false>(w[i]));
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

__device__ __forceinline__ float load_one(const void* p, int64_t i, int dtype) {
  if (dtype == MOE_FP32) return static_cast<const float*>(p)[i];
  const uint16_t b = static_cast<const uint16_t*>(p)[i];
  return split(dtype == MOE_FP16 ? unpack2<true>(b) : unpack2<false>(b)).x;
}

__device__ __forceinline__ void store_one(void* p, int64_t i, int dtype, float v) {
  if (dtype == MOE_FP32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] =
        static_cast<uint16_t>(dtype == MOE_FP16 ? pack2<true>(v, 0.0f) : pack2<false>(v, 0.0f));
}

// max that keeps NaN
__device__ __forceinline__ double max_nan(double a, double b) { return a != a ? a : (b != b ? b : (a > b ? a : b)); }

// A thread's running norm: sum of squares or largest magnitude.
struct NormAcc {
  double v = 0.0;
  bool l2;
  __device__ void add(const float (&f)[8]) {
    if (l2) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(f[i], f[i], s);
      if (s > 1e-28f && s < 1e38f) {
        v += static_cast<double>(s);
        return;
      }
      bool any = false;  // all zero: nothing to add
#pragma unroll
      for (int i = 0; i < 8; ++i) any |= f[i] != 0.0f;
      if (!any) return;
#pragma unroll
      for (int i = 0; i < 8; ++i) v += static_cast<double>(f[i]) * static_cast<double>(f[i]);
    } else {
      float m = 0.0f;
      bool nan = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        m = fmaxf(m, fabsf(f[i]));
        nan |= f[i] != f[i];
      }
      v = max_nan(v, nan ? static_cast<double>(__uint_as_float(0x7fc00000u)) : static_cast<double>(m));
    }
  }
  __device__ void add_one(float f) {
    if (l2)
      v += static_cast<double>(f) * static_cast<double>(f);
    else
      v = max_nan(v, fabs(static_cast<double>(f)));
  }
};

// Sum (or max) over the block, in a fixed order; valid in every thread.
__device__ double block_reduce(double v, bool l2, double* smem) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double w = __shfl_xor_sync(0xffffffffu, v, o);
    v = l2 ? v + w : max_nan(v, w);
  }
  if (threadIdx.x % kWarp == 0) smem[threadIdx.x / kWarp] = v;
  __syncthreads();
  v = smem[0];
#pragma unroll
  for (int i = 1; i < kThreads / kWarp; ++i) v = l2 ? v + smem[i] : max_nan(v, smem[i]);
  return v;
}

__device__ double reduce_partials(const double* partial, int n, bool l2, double* smem) {
  double v = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) v = l2 ? v + partial[i] : max_nan(v, partial[i]);
  return block_reduce(v, l2, smem);
}

// This block's run of chunks [lo, hi).
__device__ __forceinline__ void run_of(int64_t chunks, int64_t* lo, int64_t* hi) {
  *lo = chunks * blockIdx.x / gridDim.x;
  *hi = chunks * (blockIdx.x + 1) / gridDim.x;
}

// Index of the tensor that holds chunk c: the last with first <= c (tensors
// without elements have no chunk and are skipped).
__device__ __forceinline__ int find(const ClipEntry* plan, int n, int64_t c) {
  int a = 0, b = n - 1;
  while (a < b) {
    const int m = (a + b + 1) / 2;
    if (plan[m].first <= c)
      a = m;
    else
      b = m - 1;
  }
  return a;
}

__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    norm_kernel(const ClipEntry* plan, int n, int64_t chunks, int norm_type, double* partial) {
  __shared__ double smem[kThreads / kWarp];
  pdl_wait();
  pdl_launch_dependents();
  NormAcc acc;
  acc.l2 = norm_type == MOE_NORM_L2;
  int64_t lo, hi;
  run_of(chunks, &lo, &hi);
  if (lo < hi) {
    for (int t = find(plan, n, lo); t < n; ++t) {
      const ClipEntry e = plan[t];
      if (e.first >= hi) break;
      const int64_t a = (lo > e.first ? lo - e.first : 0) * kClipChunk;
      int64_t b = (hi - e.first) * kClipChunk;
      if (b > e.numel) b = e.numel;
      if (a >= b) continue;
      const int dtype = static_cast<int>(e.dtype);
      const int size = dtype == MOE_FP32 ? 4 : 2;
      const uintptr_t p0 = reinterpret_cast<uintptr_t>(e.src) + a * size;
      int64_t head = static_cast<int64_t>((16 - (p0 & 15)) & 15) / size;  // elements before 16-byte alignment
      if (head > b - a) head = b - a;
      const int per = 16 / size;
      const int64_t vecs = (b - a - head) / per;
      const uint4* pv = reinterpret_cast<const uint4*>(p0 + head * size);
      int64_t i = threadIdx.x;
      for (; i + 3 * kThreads < vecs; i += 4 * kThreads) {
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = pv[i + j * kThreads];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float f[8];
          int m;
          unpack_vec(v[j], dtype, f, &m);
          acc.add(f);
        }
      }
      for (; i < vecs; i += kThreads) {
        float f[8];
        int m;
        unpack_vec(pv[i], dtype, f, &m);
        acc.add(f);
      }
      if (threadIdx.x < head) acc.add_one(load_one(e.src, a + threadIdx.x, dtype));
      const int64_t tail = a + head + vecs * per;
      if (tail + threadIdx.x < b) acc.add_one(load_one(e.src, tail + threadIdx.x, dtype));
    }
  }
  const double s = block_reduce(acc.v, acc.l2, smem);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__global__ void __launch_bounds__(kThreads) norm_finish_kernel(const double* partial, int n,
                                                               int norm_type, float* norm, int32_t* status) {
  __shared__ double smem[kThreads / kWarp];
  pdl_wait();
  pdl_launch_dependents();
  const bool l2 = norm_type == MOE_NORM_L2;
  double v = reduce_partials(partial, n, l2, smem);
  if (l2) v = sqrt(v);
  if (threadIdx.x == 0) {
    *norm = static_cast<float>(v);
    if (!isfinite(v)) set_status(status, MOE_ERR_NONFINITE);
  }
}

__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    scale_kernel(const ClipEntry* plan, int n, int64_t chunks, int norm_type, double max_norm,
                 const double* partial, float* norm, int32_t* status) {
  __shared__ double smem[kThreads / kWarp];
  pdl_wait();
  pdl_launch_dependents();
  const bool l2 = norm_type == MOE_NORM_L2;
  double v = reduce_partials(partial, gridDim.x, l2, smem);
  if (l2) v = sqrt(v);
  const bool finite = isfinite(v);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *norm = static_cast<float>(v);
    if (!finite) set_status(status, MOE_ERR_NONFINITE);
  }
  const double cd = max_norm / (v + 1e-6);
  const float c = finite && cd < 1.0 ? static_cast<float>(cd) : 1.0f;
  int64_t lo, hi;
  run_of(chunks, &lo, &hi);
  if (lo >= hi) return;
  for (int t = find(plan, n, hi - 1); t >= 0; --t) {
    const ClipEntry e = plan[t];
    const int64_t a = (lo > e.first ? lo - e.first : 0) * kClipChunk;
    int64_t b = (hi - e.first) * kClipChunk;
    if (b > e.numel) b = e.numel;
    if (a < b && !(c == 1.0f && e.src == e.dst)) {
      const int dtype = static_cast<int>(e.dtype);
      const int size = dtype == MOE_FP32 ? 4 : 2;
      const int per = 16 / size;
      const uintptr_t p0 = reinterpret_cast<uintptr_t>(e.src) + a * size;
      const uintptr_t q0 = reinterpret_cast<uintptr_t>(e.dst) + a * size;
      int64_t head = static_cast<int64_t>((16 - (p0 & 15)) & 15) / size;
      if (head > b - a) head = b - a;
      // vectors only where source and target are aligned alike
      const int64_t vecs = ((p0 ^ q0) & 15) == 0 ? (b - a - head) / per : 0;
      const uint4* pv = reinterpret_cast<const uint4*>(p0 + head * size);
      uint4* qv = reinterpret_cast<uint4*>(q0 + head * size);
      auto scaled = [&](uint4 x) {
        float f[8];
        int m;
        unpack_vec(x, dtype, f, &m);
        if (dtype == MOE_FP32)
          return make_uint4(__float_as_uint(f[0] * c), __float_as_uint(f[1] * c), __float_as_uint(f[2] * c),
                            __float_as_uint(f[3] * c));
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          o[k] = dtype == MOE_FP16 ? pack2<true>(f[2 * k] * c, f[2 * k + 1] * c)
                                   : pack2<false>(f[2 * k] * c, f[2 * k + 1] * c);
        return make_uint4(o[0], o[1], o[2], o[3]);
      };
      const int64_t tail = a + head + vecs * per;
      for (int64_t i = b - 1 - threadIdx.x; i >= tail; i -= kThreads) store_one(e.dst, i, dtype, load_one(e.src, i, dtype) * c);
      int64_t i = vecs - 1 - threadIdx.x;
      for (; i - 3 * kThreads >= 0; i -= 4 * kThreads) {
        uint4 x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = pv[i - j * kThreads];
#pragma unroll
        for (int j = 0; j < 4; ++j) qv[i - j * kThreads] = scaled(x[j]);
      }
      for (; i >= 0; i -= kThreads) qv[i] = scaled(pv[i]);
      if (threadIdx.x < head) store_one(e.dst, a + threadIdx.x, dtype, load_one(e.src, a + threadIdx.x, dtype) * c);
    }
    if (e.first <= lo) break;
  }
}

// Plan entries travel as launch parameters, a batch at a time.
constexpr int kBatch = 96;
struct Batch {
  ClipEntry e[kBatch];
};
static_assert(sizeof(Batch) <= 4000, "launch parameters");

__global__ void plan_kernel(const __grid_constant__ Batch batch, int n, ClipEntry* plan) {
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x < n) plan[threadIdx.x] = batch.e[threadIdx.x];
}

int clip_blocks(int64_t chunks, int num_sms) {
  int64_t g = static_cast<int64_t>(num_sms) * kBlocksPerSm;
  if (g > kClipMaxBlocks) g = kClipMaxBlocks;
  if (g > chunks) g = chunks;
  return g < 1 ? 1 : static_cast<int>(g);
}

}  // namespace

cudaError_t launch_clip_plan(const ClipEntry* entries, int n, ClipEntry* plan, cudaStream_t stream, int* launches) {
  for (int i = 0; i < n; i += kBatch) {
    Batch b;
    const int m = n - i < kBatch ? n - i : kBatch;
    for (int j = 0; j < kBatch; ++j) b.e[j] = entries[i + (j < m ? j : 0)];
    cudaError_t err = launch_pdl(plan_kernel, dim3(1), dim3(kBatch), 0, stream, b, m, plan + i);
    if (err != cudaSuccess) return err;
    ++*launches;
  }
  return cudaSuccess;
}

cudaError_t launch_clip_norm(const ClipEntry* plan, int n, int64_t chunks, int norm_type, double* partial, float* norm,
                             bool finish, int32_t* status, int num_sms, cudaStream_t stream, int* launches) {
  const int g = clip_blocks(chunks, num_sms);
  cudaError_t err = launch_pdl(norm_kernel, dim3(g), dim3(kThreads), 0, stream, plan, n, chunks, norm_type, partial);
  if (err != cudaSuccess) return err;
  ++*launches;
  if (!finish) return cudaSuccess;
  err = launch_pdl(norm_finish_kernel, dim3(1), dim3(kThreads), 0, stream, static_cast<const double*>(partial), g,
                   norm_type, norm, status);
  if (err == cudaSuccess) ++*launches;
  return err;
}

cudaError_t launch_clip_scale(const ClipEntry* plan, int n, int64_t chunks, int norm_type, double max_norm,
                              const double* partial, float* norm, int32_t* status, int num_sms, cudaStream_t stream,
                              int* launches) {
  cudaError_t err = launch_pdl(scale_kernel, dim3(clip_blocks(chunks, num_sms)), dim3(kThreads), 0, stream, plan, n,
                               chunks, norm_type, max_norm, partial, norm, status);
  if (err == cudaSuccess) ++*launches;
  return err;
}

}  // namespace moe
