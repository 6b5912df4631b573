// Linear layer, backward, elementwise part: dz = dout * act'(pre) and the
// bias gradient db[n] = sum_t dz[t, n].
//
// Bound by memory: dout and pre are read once, dz is written once (with no
// activation dz is dout itself and only the column sums are formed).  A block
// covers 64 columns (a lane eight of them, 16 bytes; a warp four rows) and
// one of kParts shares of the rows; the blocks of all shares form a cluster,
// and their fp32 column sums meet in distributed shared memory, added in a
// fixed order: one launch, no scratch, the same db on every call.
#include "common.cuh"
#include "dense.h"
#include "epilogue.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kCols = 64;
constexpr int kThreads = 256;
constexpr int kRows = kThreads / 8;  // rows of a block's step
constexpr int kParts = 8;
// Rows of a thread in flight, and four blocks an SM (64 registers): 8192 x 8192
// with silu 79 us, 5.1 TB/s; three blocks 88 us, two blocks with four rows 87.
// At 64 registers the activations' variants share 76 bytes of spills; the
// three-block form has none and is the slower one all the same.
constexpr int kUnroll = 2;

template <bool kFp16>
__global__ void __launch_bounds__(kThreads, 4)
    dz_kernel(const uint16_t* dout, int64_t ldd, const uint16_t* pre, int64_t ldp, int64_t T, int64_t N, int act,
              uint16_t* dz, uint16_t* dbias) {
  __shared__ float sums[kThreads / kWarp][kCols];
  __shared__ __align__(16) float part[kCols];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * kCols + (lane & 7) * 8;
  const int64_t t0 = T * blockIdx.y / kParts, t1 = T * (blockIdx.y + 1) / kParts;
  F2 s2[4] = {f2(0.0f), f2(0.0f), f2(0.0f), f2(0.0f)};
  auto rows = [&](auto act_c) {
    for (int64_t t = t0 + threadIdx.x / 8; t < t1; t += kUnroll * kRows) {
      uint4 d4[kUnroll], z4[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int64_t r = t + k * kRows;
        if (r >= t1) continue;
        d4[k] = *reinterpret_cast<const uint4*>(dout + r * ldd + col);
        if (pre != nullptr) z4[k] = *reinterpret_cast<const uint4*>(pre + r * ldp + col);
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int64_t r = t + k * kRows;
        if (r >= t1) continue;
        F2 d[4];
        unpack8<kFp16>(d4[k], d);
        if (pre != nullptr) {
          F2 z[4];
          unpack8<kFp16>(z4[k], z);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            F2 slope;
            act_value_slope<decltype(act_c)::value>(z[i], &slope);
            d[i] = d[i] * slope;
          }
          *reinterpret_cast<uint4*>(dz + r * N + col) = pack8<kFp16>(d);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s2[i] = s2[i] + d[i];
      }
    }
  };
  if (col < N) with_act(act, rows);
  if (dbias == nullptr) return;  // the same in every block of the cluster
  float s[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = split(s2[i]);
    s[2 * i] = p.x;
    s[2 * i + 1] = p.y;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    s[i] += __shfl_xor_sync(0xffffffffu, s[i], 8);
    s[i] += __shfl_xor_sync(0xffffffffu, s[i], 16);
  }
  if (lane < 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[warp][lane * 8 + i] = s[i];
  }
  __syncthreads();
  if (threadIdx.x < kCols) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kThreads / kWarp; ++w) v += sums[w][threadIdx.x];
    part[threadIdx.x] = v;
  }
  ptx::cluster_sync();
  // this block finishes kCols / kParts of the columns
  constexpr int kMine = kCols / kParts;
  if (threadIdx.x < kMine) {
    const int i = blockIdx.y * kMine + threadIdx.x;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kCols + i;
    const uint32_t at = ptx::smem_u32(&part[i]);
    float p[kParts];
#pragma unroll
    for (int r = 0; r < kParts; ++r) p[r] = ptx::ld_cluster_f32(ptx::map_rank(at, r));
    float v = 0.0f;
#pragma unroll
    for (int r = 0; r < kParts; ++r) v += p[r];
    if (c < N) dbias[c] = static_cast<uint16_t>(pack2<kFp16>(v, 0.0f));
  }
  ptx::cluster_sync();  // no block leaves while another reads its sums
}

}  // namespace

cudaError_t launch_dz(const DzArgs& a, cudaStream_t stream, int* launches) {
  auto kern = a.fp16 ? dz_kernel<true> : dz_kernel<false>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.N + kCols - 1) / kCols), kParts);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = kParts;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t err =
      cudaLaunchKernelEx(&cfg, kern, a.dout, a.ldd, a.pre, a.ldp, a.T, a.N, a.act, a.dz, a.dbias);
  if (err == cudaSuccess) ++*launches;
  return err;
}

}  // namespace moe
