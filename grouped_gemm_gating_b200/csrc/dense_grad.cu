// Linear layer, backward, elementwise part: dz = dout * act'(pre) and the
// bias gradient db[n] = sum_t dz[t, n].
//
// Bound by memory: dout and pre are read once, dz is written once (with no
// activation dz is dout itself and only the column sums are formed).  A warp
// covers 256 contiguous columns of a row (16 bytes a lane); a block of eight
// warps walks its share of the rows, every eighth row a warp, and adds its
// fp32 sums into one partial row per block of rows.  A second kernel adds
// the partial rows in a fixed order, so db is the same on every call.
#include "common.cuh"
#include "dense.h"
#include "epilogue.cuh"

namespace moe {
namespace {

constexpr int kCols = 256;   // columns of a block
constexpr int kLanes = 8;    // warps of a block

template <bool kFp16>
__global__ void __launch_bounds__(kCols) dz_kernel(const uint16_t* dout, int64_t ldd,
                                                   const uint16_t* pre, int64_t ldp, int64_t T,
                                                   int64_t N, int64_t rows_per_block, int act,
                                                   uint16_t* dz, float* partial) {
  __shared__ float sums[kLanes][kCols];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * kCols + lane * 8;
  const int64_t t0 = blockIdx.y * rows_per_block;
  const int64_t t1 = t0 + rows_per_block < T ? t0 + rows_per_block : T;
  float s[8] = {};
  if (col < N) {
    for (int64_t t = t0 + warp; t < t1; t += kLanes) {
      const uint4 dv = *reinterpret_cast<const uint4*>(dout + t * ldd + col);
      const uint32_t dw[4] = {dv.x, dv.y, dv.z, dv.w};
      float d[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 p = unpack2<kFp16>(dw[i]);
        d[2 * i] = p.x;
        d[2 * i + 1] = p.y;
      }
      if (pre != nullptr) {
        const uint4 zv = *reinterpret_cast<const uint4*>(pre + t * ldp + col);
        const uint32_t zw[4] = {zv.x, zv.y, zv.z, zv.w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 z = unpack2<kFp16>(zw[i]);
          float s0, s1;
          act_value_slope(z.x, act, &s0);
          act_value_slope(z.y, act, &s1);
          d[2 * i] *= s0;
          d[2 * i + 1] *= s1;
          o[i] = pack2<kFp16>(d[2 * i], d[2 * i + 1]);
        }
        *reinterpret_cast<uint4*>(dz + t * N + col) = make_uint4(o[0], o[1], o[2], o[3]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] += d[i];
    }
  }
  if (partial == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[warp][lane * 8 + i] = s[i];
  __syncthreads();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kCols + threadIdx.x;
  if (c < N) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kLanes; ++w) v += sums[w][threadIdx.x];
    partial[blockIdx.y * N + c] = v;
  }
}

template <bool kFp16>
__global__ void __launch_bounds__(kCols) dbias_kernel(const float* partial, int blocks, int64_t N,
                                                      uint16_t* dbias) {
  __shared__ float sums[kLanes][kWarp + 1];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kWarp + lane;
  float v = 0.0f;
  if (c < N)
    for (int b = warp; b < blocks; b += kLanes) v += partial[b * N + c];
  sums[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < N) {
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < kLanes; ++w) v += sums[w][lane];
    dbias[c] = static_cast<uint16_t>(pack2<kFp16>(v, 0.0f));
  }
}

}  // namespace

cudaError_t launch_dz(const DzArgs& a, int num_sms, cudaStream_t stream, int* launches) {
  const int64_t gx = (a.N + kCols - 1) / kCols;
  // blocks of rows: enough to fill the GPU a few times over, at least a row per warp each
  int64_t gy = (static_cast<int64_t>(num_sms) * 8 + gx - 1) / gx;
  if (gy > kDzMaxBlocks) gy = kDzMaxBlocks;
  if (gy > (a.T + kLanes - 1) / kLanes) gy = (a.T + kLanes - 1) / kLanes;
  if (gy < 1) gy = 1;
  const int64_t rows = (a.T + gy - 1) / gy;
  float* partial = a.dbias != nullptr ? a.partial : nullptr;
  auto kern = a.fp16 ? dz_kernel<true> : dz_kernel<false>;
  cudaError_t err = launch_pdl(kern, dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), dim3(kCols), 0, stream,
                               a.dout, a.ldd, a.pre, a.ldp, a.T, a.N, rows, a.act, a.dz, partial);
  if (err != cudaSuccess) return err;
  ++*launches;
  if (partial == nullptr) return cudaSuccess;
  auto fin = a.fp16 ? dbias_kernel<true> : dbias_kernel<false>;
  err = launch_pdl(fin, dim3(static_cast<unsigned>((a.N + kWarp - 1) / kWarp)), dim3(kCols), 0, stream,
                   static_cast<const float*>(partial), static_cast<int>(gy), a.N, a.dbias);
  if (err == cudaSuccess) ++*launches;
  return err;
}

}  // namespace moe
