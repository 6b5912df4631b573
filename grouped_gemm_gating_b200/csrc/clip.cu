// Global norm over many gradient tensors and clipping to it.
//
//   norm = sqrt(sum_i g_i^2)  or  max_i |g_i|   over all elements of all tensors
//   g_i <- c g_i,  c = min(1, max_norm / (norm + 1e-6))
//
// Bound by memory: the norm needs every gradient before the first one can be
// scaled, so the tensors are read twice and written once unless they stay in
// L2 between the two kernels.  Tensors are numbered through in chunks of
// kClipChunk elements; runs of chunks (of up to 256 KB) are dealt round-robin
// to the blocks, so that all of them read and write near each other (604 M
// bf16 values out of place: 371 us, the speed of a copy, against 474 us with
// one long run a block).  The norm goes front to back, run by run, and the
// scaling back to front: what the first kernel read last is what the second
// reads first.
//
// Sums: eight squares in fp32 (their relative error is below 2^-21, and
// averages out), then 64 bits throughout.  A group whose fp32 sum leaves the
// range where its squares are normal numbers is summed again in 64 bits, so
// neither large nor tiny gradients overflow or vanish.  Every block's sum is
// one partial; both kernels add the partials in a fixed order: the norm is
// the same on every call.
//
// Targets that lie differently within 16 bytes than their sources are written
// one value at a time: 200 M bf16 values 785 us, aligned alike 207 us.
#include "common.cuh"
#include "dense.h"
#include "epilogue.cuh"
#include <type_traits>

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kNormBlocksPerSm = 3;   // reading alone: 185 us against 197 with two (1.2 GB)
constexpr int kScaleBlocksPerSm = 2;  // reading and writing: 406 us against 420 with three
constexpr int kMinRun = 1, kMaxRun = 64;  // chunks of a run

// Runs f with the type as a compile-time constant.
template <class F>
__device__ __forceinline__ void with_dtype(int dtype, F&& f) {
  if (dtype == MOE_FP32)
    f(std::integral_constant<int, MOE_FP32>{});
  else if (dtype == MOE_FP16)
    f(std::integral_constant<int, MOE_FP16>{});
  else
    f(std::integral_constant<int, MOE_BF16>{});
}

// The four or eight values of a 16-byte vector.
template <int DT>
__device__ __forceinline__ void unpack_vec(uint4 v, float (&f)[DT == MOE_FP32 ? 4 : 8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == MOE_FP32) {
      f[i] = __uint_as_float(w[i]);
    } else {
      const float2 p = split(unpack2<DT == MOE_FP16>(w[i]));
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
}

template <int DT>
__device__ __forceinline__ uint4 scale_vec(uint4 v, float c) {
  float f[DT == MOE_FP32 ? 4 : 8];
  unpack_vec<DT>(v, f);
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (DT == MOE_FP32)
      o[k] = __float_as_uint(f[k] * c);
    else
      o[k] = pack2<DT == MOE_FP16>(f[2 * k] * c, f[2 * k + 1] * c);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
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
  template <int N>
  __device__ __forceinline__ void add(const float (&f)[N]) {
    if (l2) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) s = fmaf(f[i], f[i], s);
      if (s > 1e-28f && s < 1e38f) {
        v += static_cast<double>(s);
        return;
      }
      bool any = false;  // all zero: nothing to add
#pragma unroll
      for (int i = 0; i < N; ++i) any |= f[i] != 0.0f;
      if (!any) return;
#pragma unroll
      for (int i = 0; i < N; ++i) v += static_cast<double>(f[i]) * static_cast<double>(f[i]);
    } else {
      float m = 0.0f;
      bool nan = false;
#pragma unroll
      for (int i = 0; i < N; ++i) {
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

// Index of the tensor that holds chunk c: the last with first <= c (tensors
// without elements have no chunk and are skipped), looked for near `t` first.
__device__ __forceinline__ int find(const ClipEntry* plan, int n, int64_t c, int t) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if (plan[t].first > c)
      --t;  // the first tensor starts at chunk 0
    else if (t + 1 < n && plan[t + 1].first <= c)
      ++t;
    else
      return t;
  }
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

// The part [a, b) of a tensor that lies in chunks [lo, hi): `head` elements
// before the source is 16-byte aligned, then `vecs` vectors of `per`, then
// the rest from `tail`.
struct Span {
  ClipEntry e;
  int64_t a, b, tail;
  int vecs, dtype, size, per, head;  // a run has at most kMaxRun chunks
};
__device__ __forceinline__ Span span_of(const ClipEntry* plan, int t, int64_t lo, int64_t hi) {
  Span s;
  s.e = plan[t];
  s.a = (lo > s.e.first ? lo - s.e.first : 0) * kClipChunk;
  s.b = (hi - s.e.first) * kClipChunk;
  if (s.b > s.e.numel) s.b = s.e.numel;
  s.dtype = static_cast<int>(s.e.dtype);
  s.size = s.dtype == MOE_FP32 ? 4 : 2;
  s.per = 16 / s.size;
  const int64_t len = s.b > s.a ? s.b - s.a : 0;
  const uintptr_t p = reinterpret_cast<uintptr_t>(s.e.src) + s.a * s.size;
  s.head = static_cast<int>((16 - (p & 15)) & 15) / s.size;
  if (s.head > len) s.head = static_cast<int>(len);
  s.vecs = static_cast<int>((len - s.head) / s.per);
  s.tail = s.a + s.head + static_cast<int64_t>(s.vecs) * s.per;
  return s;
}

__global__ void __launch_bounds__(kThreads, kNormBlocksPerSm)
    norm_kernel(const ClipEntry* plan, int n, int64_t chunks, int run, int norm_type, double* partial) {
  __shared__ double smem[kThreads / kWarp];
  pdl_wait();
  pdl_launch_dependents();
  NormAcc acc;
  acc.l2 = norm_type == MOE_NORM_L2;
  int near = 0;
  for (int64_t lo = static_cast<int64_t>(blockIdx.x) * run; lo < chunks; lo += static_cast<int64_t>(gridDim.x) * run) {
    const int64_t hi = lo + run < chunks ? lo + run : chunks;
    near = find(plan, n, lo, near);
    for (int t = near; t < n; ++t) {
      const Span s = span_of(plan, t, lo, hi);
      if (s.e.first >= hi) break;
      near = t;
      if (s.a >= s.b) continue;
      const uint4* pv = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(s.e.src) + (s.a + s.head) * s.size);
      with_dtype(s.dtype, [&](auto dt) {
        constexpr int kDt = decltype(dt)::value;
        float f[kDt == MOE_FP32 ? 4 : 8];
        int i = threadIdx.x;
        for (; i + 3 * kThreads < s.vecs; i += 4 * kThreads) {
          uint4 v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = pv[i + j * kThreads];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            unpack_vec<kDt>(v[j], f);
            acc.add(f);
          }
        }
        for (; i < s.vecs; i += kThreads) {
          unpack_vec<kDt>(pv[i], f);
          acc.add(f);
        }
      });
      if (threadIdx.x < s.head) acc.add_one(load_one(s.e.src, s.a + threadIdx.x, s.dtype));
      if (s.tail + threadIdx.x < s.b) acc.add_one(load_one(s.e.src, s.tail + threadIdx.x, s.dtype));
    }
  }
  const double s = block_reduce(acc.v, acc.l2, smem);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// The norm counts as finite when the fp32 value that the caller sees is: two
// values of 3e38 are finite, their norm is reported as infinity.
__device__ __forceinline__ bool norm_finite(double v) { return isfinite(static_cast<float>(v)); }

__device__ __forceinline__ void report_norm(double v, float* norm, int32_t* status) {
  *norm = static_cast<float>(v);
  if (!norm_finite(v)) set_status(status, MOE_ERR_NONFINITE);
}

__global__ void __launch_bounds__(kThreads) norm_finish_kernel(const double* partial, int n,
                                                               int norm_type, float* norm, int32_t* status) {
  __shared__ double smem[kThreads / kWarp];
  pdl_wait();
  pdl_launch_dependents();
  const bool l2 = norm_type == MOE_NORM_L2;
  double v = reduce_partials(partial, n, l2, smem);
  if (l2) v = sqrt(v);
  if (threadIdx.x == 0) report_norm(v, norm, status);
}

__global__ void __launch_bounds__(kThreads, kScaleBlocksPerSm)
    scale_kernel(const ClipEntry* plan, int n, int64_t chunks, int run, int norm_type, double max_norm,
                 const double* partial, int n_partial, float* norm, int32_t* status) {
  __shared__ double smem[kThreads / kWarp];
  pdl_wait();
  pdl_launch_dependents();
  const bool l2 = norm_type == MOE_NORM_L2;
  double v = reduce_partials(partial, n_partial, l2, smem);
  if (l2) v = sqrt(v);
  if (blockIdx.x == 0 && threadIdx.x == 0) report_norm(v, norm, status);
  const double cd = max_norm / (v + 1e-6);
  const float c = norm_finite(v) && cd < 1.0 ? static_cast<float>(cd) : 1.0f;
  int near = n - 1;
  const int64_t runs = (chunks + run - 1) / run;
  for (int64_t r = runs - 1 - blockIdx.x; r >= 0; r -= gridDim.x) {
    const int64_t lo = r * run, hi = lo + run < chunks ? lo + run : chunks;
    near = find(plan, n, hi - 1, near);
    for (int t = near; t >= 0; --t) {
      const Span s = span_of(plan, t, lo, hi);
      near = t;
      if (s.a < s.b && !(c == 1.0f && s.e.src == s.e.dst)) {
        const uint8_t* p = static_cast<const uint8_t*>(s.e.src) + (s.a + s.head) * s.size;
        uint8_t* q = static_cast<uint8_t*>(s.e.dst) + (s.a + s.head) * s.size;
        // vectors only where source and target are aligned alike
        const bool alike = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15) == 0;
        const int vecs = alike ? s.vecs : 0;
        const int64_t tail = alike ? s.tail : s.a + s.head;
        const uint4* pv = reinterpret_cast<const uint4*>(p);
        uint4* qv = reinterpret_cast<uint4*>(q);
        // read and written for the last time here: not kept in L2 for long
        with_dtype(s.dtype, [&](auto dt) {
          constexpr int kDt = decltype(dt)::value;
          int i = threadIdx.x;
          for (; i + kThreads < vecs; i += 2 * kThreads) {
            const uint4 x0 = __ldcs(pv + i), x1 = __ldcs(pv + i + kThreads);
            __stcs(qv + i, scale_vec<kDt>(x0, c));
            __stcs(qv + i + kThreads, scale_vec<kDt>(x1, c));
          }
          if (i < vecs) __stcs(qv + i, scale_vec<kDt>(__ldcs(pv + i), c));
        });
        if (threadIdx.x < s.head)
          store_one(s.e.dst, s.a + threadIdx.x, s.dtype, load_one(s.e.src, s.a + threadIdx.x, s.dtype) * c);
        for (int64_t k = tail + threadIdx.x; k < s.b; k += kThreads)
          store_one(s.e.dst, k, s.dtype, load_one(s.e.src, k, s.dtype) * c);
      }
      if (s.e.first <= lo) break;
    }
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

// Chunks of a run (several runs a block while there are enough) and blocks.
int clip_run(int64_t chunks, int num_sms) {
  const int64_t r = chunks / (static_cast<int64_t>(num_sms) * kScaleBlocksPerSm * 8);
  return r < kMinRun ? kMinRun : r > kMaxRun ? kMaxRun : static_cast<int>(r);
}

int clip_blocks(int64_t chunks, int num_sms, int per_sm) {
  const int64_t run = clip_run(chunks, num_sms);
  int64_t g = static_cast<int64_t>(num_sms) * per_sm;
  if (g > kClipMaxBlocks) g = kClipMaxBlocks;
  if (g > (chunks + run - 1) / run) g = (chunks + run - 1) / run;
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
  const int g = clip_blocks(chunks, num_sms, kNormBlocksPerSm);
  cudaError_t err = launch_pdl(norm_kernel, dim3(g), dim3(kThreads), 0, stream, plan, n, chunks,
                               clip_run(chunks, num_sms), norm_type, partial);
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
  const dim3 grid(clip_blocks(chunks, num_sms, kScaleBlocksPerSm));
  cudaError_t err = launch_pdl(scale_kernel, grid, dim3(kThreads), 0, stream, plan, n, chunks,
                               clip_run(chunks, num_sms), norm_type, max_norm, partial,
                               clip_blocks(chunks, num_sms, kNormBlocksPerSm), norm, status);
  if (err == cudaSuccess) ++*launches;
  return err;
}

}  // namespace moe
