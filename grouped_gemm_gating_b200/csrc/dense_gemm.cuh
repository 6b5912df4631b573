// Dense GEMMs of the linear layer and the gated feed-forward block, and of
// their backward passes, on CTA pairs (tcgen05 cta_group::2).
//
//   sum[m, n] = sum_k A[m, k] B[n, k]    (fp32, one pass over k)
//
// with the operation's elementwise part in the epilogue (DenseEpi), so that
// no fp32 sum and no second pass over the output touches global memory:
//   linear    out = act(sum + bias) + residual
//   gate      B's rows are Wg's and Wu's: out = act(g) * u
//   gate-grad sum = dh: [dg | du] and h from the kept [g | u]
// A cluster of two CTAs works on 256 rows of M and BN columns: each CTA
// loads its own 128 rows of A and half of B's BN rows by TMA (zero fill past
// M, N and K, so every size a multiple of the 16-byte rule works), the bytes
// of both complete on the even CTA's barrier, and its MMA thread issues
// M = 256, N = BN MMAs over both CTAs' shared memory.  The two halves of a
// gate tile are one CTA's gate rows and the other's matching up rows, so a
// thread finds g and u of its row BN / 2 columns apart in tensor memory.
// Operands whose contraction index is not contiguous (dx = dz W reads W by
// rows of the contraction; dW = dz^T x reads both so) are read MN-major.
//
// Two accumulators in tensor memory: the epilogue (eight warps, two per lane
// quadrant, each on half of the columns) drains one while the MMA fills the
// other.  Tiles go in groups of kGroupM row tiles, column by column, so the
// pairs at work share operand rows in L2.
//
// Every mbarrier wait is bounded; on expiry the CTA records
// MOE_ERR_DEVICE_TIMEOUT and its roles leave their loops; loads and MMAs in
// flight are waited for before shared and tensor memory are given up.
#pragma once
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "dense.h"
#include "epilogue.cuh"
#include "host.h"
#include "ptx.cuh"

namespace moe {
namespace dense {

// After an abort, the odd CTA's wait for its last loads to land (they
// complete on the even CTA's barriers): far above a TMA load's latency.
constexpr uint64_t kDrainGraceNs = 50000;
constexpr int kGroupM = 8;

struct Args {
  CUtensorMap tm_a, tm_b;
  int64_t M, N, ldr, ldo, ldp;
  int nk, n_mt, n_nt;
  const uint16_t* bias;
  const uint16_t* residual;
  uint16_t* out;
  uint16_t* pre;
  uint16_t* out2;
  int act;
  int32_t* status;
  uint64_t wait_ns;
  int tfull_surplus;
};

template <int EPI, int MAJOR, int BN>
struct Cfg {
  static constexpr bool kAMn = MAJOR == kMajorMN;
  static constexpr bool kBMn = MAJOR != kMajorKK;
  static constexpr int kOutCols = EPI == kDenseGate ? BN / 2 : BN;  // output columns of a tile
  static constexpr int kABytes = 128 * 128;                          // 128 M values x 64 K
  static constexpr int kBBytes = BN / 2 * 128;                       // this CTA's half of B
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = BN == 256 ? 6 : 8;
  static constexpr int kTmemCols = 2 * BN;
  static constexpr int kNumThreads = 320;  // producer, MMA, eight epilogue warps
  static constexpr int kBarrierBytes = 256;
  static constexpr int kSmemBytes = kStages * kStageBytes + kBarrierBytes + 1024;
  static_assert((2 * kStages + 5) * 8 + 16 <= kBarrierBytes, "barrier area");
  static_assert(kSmemBytes <= 232448, "shared memory per block");
};

// Runs f with the activation as a compile-time constant.
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case MOE_EPI_SILU: f(std::integral_constant<int, MOE_EPI_SILU>{}); break;
    case MOE_EPI_GELU: f(std::integral_constant<int, MOE_EPI_GELU>{}); break;
    case MOE_EPI_GELU_TANH: f(std::integral_constant<int, MOE_EPI_GELU_TANH>{}); break;
    case MOE_EPI_RELU: f(std::integral_constant<int, MOE_EPI_RELU>{}); break;
    case MOE_EPI_RELU2: f(std::integral_constant<int, MOE_EPI_RELU2>{}); break;
    default: f(std::integral_constant<int, MOE_EPI_NONE>{}); break;
  }
}

template <int COLS>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[COLS]) {
#pragma unroll
  for (int i = 0; i < COLS; i += 16) ptx::tmem_ld16(addr + i, *reinterpret_cast<uint32_t(*)[16]>(&r[i]));
}

template <int COLS>
__device__ __forceinline__ void pin(uint32_t (&r)[COLS]) {  // uses stay after the wait
#pragma unroll
  for (int j = 0; j < COLS; ++j) asm volatile("" : "+r"(r[j]));
}

template <bool kFp16>
__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack2<kFp16>(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

template <bool kFp16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2<kFp16>(f[0], f[1]), pack2<kFp16>(f[2], f[3]), pack2<kFp16>(f[4], f[5]),
                    pack2<kFp16>(f[6], f[7]));
}

template <int EPI, int MAJOR, int BN, bool kFp16>
__global__ void __launch_bounds__(Cfg<EPI, MAJOR, BN>::kNumThreads, 1)
    dense_gemm_kernel(const __grid_constant__ Args args) {
  using C = Cfg<EPI, MAJOR, BN>;
  constexpr uint32_t kIdesc = ptx::idesc_16bit_f32(256, BN, kFp16, C::kAMn, C::kBMn);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStageBytes);
  uint64_t* empty = full + C::kStages;
  uint64_t* tfull = empty + C::kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* mma_done = tempty + 2;  // the MMA issuer's last commit (drain before TMEM is freed)
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  volatile int* never = reinterpret_cast<volatile int*>(tmem_holder + 2);  // stays 0: drains ignore the abort

  const int warp = threadIdx.x / kWarp;
  const int lane = threadIdx.x % kWarp;
  const int rank = static_cast<int>(ptx::cluster_ctarank());  // 0: issues the pair's MMAs
  const int pair = blockIdx.x >> 1;
  const int n_pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(&full[s], 1);   // even CTA: its producer's arrive + both CTAs' bytes
      ptx::mbar_init(&empty[s], 1);  // one commit of the pair's MMA
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&tfull[b], 1 + args.tfull_surplus);
      ptx::mbar_init(&tempty[b], 16);  // even CTA: eight epilogue warps of each CTA
    }
    ptx::mbar_init(mma_done, 1);
    *abort_flag = 0;
    *never = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&args.tm_a);
    ptx::prefetch_tmap(&args.tm_b);
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(tmem_holder, C::kTmemCols);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();  // both CTAs' barriers exist before any remote arrival
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  pdl_wait();
  pdl_launch_dependents();

  const int n_mt = args.n_mt, n_nt = args.n_nt, nk = args.nk;
  const int total_tiles = n_mt * n_nt;
  auto tile_of = [&](int tile, int* mt, int* nt) {
    const int per_group = kGroupM * n_nt;
    const int g = tile / per_group;
    const int m0 = g * kGroupM;
    const int gm = n_mt - m0 < kGroupM ? n_mt - m0 : kGroupM;
    const int r = tile - g * per_group;
    *nt = r / gm;
    *mt = m0 + (r - *nt * gm);
  };
  auto fail = [&]() {
    *abort_flag = 1;
    set_status(args.status, MOE_ERR_DEVICE_TIMEOUT);
  };

  if (warp == 0) {
    // ------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int issued = 0;  // stages filled so far
      for (int tile = pair; ok && tile < total_tiles; tile += n_pairs) {
        int mt, nt;
        tile_of(tile, &mt, &nt);
        const int m0 = mt * 256 + rank * 128;
        const int n0 = EPI == kDenseGate ? nt * (BN / 2) : nt * BN + rank * (BN / 2);
        for (int kb = 0; kb < nk; ++kb) {
          if (!ptx::mbar_wait_cluster_bounded(&empty[stage], phase ^ 1u, abort_flag, args.wait_ns)) {
            fail();
            ok = false;
            break;
          }
          uint8_t* sA = smem + stage * C::kStageBytes;
          uint8_t* sB = sA + C::kABytes;
          if (rank == 0) ptx::mbar_arrive_expect_tx(&full[stage], 2 * C::kStageBytes);
          if constexpr (C::kAMn) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
              ptx::tma_load_2d_pair(sA + j * 8192, &args.tm_a, &full[stage], m0 + 64 * j, kb * 64);
          } else {
            ptx::tma_load_2d_pair(sA, &args.tm_a, &full[stage], kb * 64, m0);
          }
          if constexpr (EPI == kDenseGate) {
            ptx::tma_load_3d_pair(sB, &args.tm_b, &full[stage], kb * 64, n0, rank);
          } else if constexpr (C::kBMn) {
#pragma unroll
            for (int j = 0; j < BN / 128; ++j)
              ptx::tma_load_2d_pair(sB + j * 8192, &args.tm_b, &full[stage], n0 + 64 * j, kb * 64);
          } else {
            ptx::tma_load_2d_pair(sB, &args.tm_b, &full[stage], kb * 64, n0);
          }
          ++issued;
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // The even CTA waits for the last phase of every stage it filled (at
      // once after a normal run).  The odd CTA's loads complete only on the
      // even CTA's barriers; after an abort it may have filled a phase the
      // even CTA never did, so it then gives its last loads time to land.
      if (rank != 0 && !ok) {
        const uint64_t t0 = ptx::globaltimer_ns();
        while (ptx::globaltimer_ns() - t0 < kDrainGraceNs) __nanosleep(256);
      }
      if (rank == 0) {
        for (int j = 1; j <= C::kStages && j <= issued; ++j) {
          int st = stage - j;
          uint32_t ph = phase;
          if (st < 0) {
            st += C::kStages;
            ph ^= 1u;
          }
          ptx::mbar_wait_cluster_bounded(&full[st], ph, never, kDrainLimitNs);
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (even CTA)
    if (lane == 0 && rank == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int abuf = 0;
      uint32_t aphase = 0;
      bool ok = true;
      for (int tile = pair; ok && tile < total_tiles; tile += n_pairs) {
        if (!ptx::mbar_wait_cluster_bounded(&tempty[abuf], aphase ^ 1u, abort_flag, args.wait_ns)) {
          fail();
          break;
        }
        ptx::tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(abuf * BN);
        for (int kb = 0; kb < nk; ++kb) {
          if (!ptx::mbar_wait_cluster_bounded(&full[stage], phase, abort_flag, args.wait_ns)) {
            fail();
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t sA = ptx::smem_u32(smem + stage * C::kStageBytes);
          const uint32_t sB = sA + C::kABytes;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t da = C::kAMn ? ptx::sw128_mnmajor_desc(sA + kk * 2048, 8192)
                                        : ptx::sw128_kmajor_desc(sA + kk * 32);
            const uint64_t db = C::kBMn ? ptx::sw128_mnmajor_desc(sB + kk * 2048, 8192)
                                        : ptx::sw128_kmajor_desc(sB + kk * 32);
            ptx::mma_bf16_pair(d_tmem, da, db, kIdesc, (kb | kk) != 0 ? 1u : 0u);
          }
          ptx::mma_commit_pair(&empty[stage]);
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        ptx::mma_commit_pair(&tfull[abuf]);  // with nothing to contract: arrives at once
        if (++abuf == 2) {
          abuf = 0;
          aphase ^= 1u;
        }
      }
      // no MMA of the pair may still run when TMEM is freed: the last commit
      // arrives on both CTAs' mma_done
      ptx::mma_commit_pair(mma_done);
      if (!ptx::mbar_wait_bounded(mma_done, 0u, never, kDrainLimitNs)) fail();
    } else if (lane == 0) {
      if (!ptx::mbar_wait_cluster_bounded(mma_done, 0u, never, kDrainLimitNs)) fail();
    }
  } else {
    // ------------------------------------------------ epilogue (both CTAs, own TMEM half)
    const int q = warp & 3;
    const int half = (warp - 2) >> 2;
    int abuf = 0;
    uint32_t aphase = 0;
    for (int tile = pair; tile < total_tiles; tile += n_pairs) {
      int mt, nt;
      tile_of(tile, &mt, &nt);
      if (!ptx::mbar_wait_cluster_bounded(&tfull[abuf], aphase, abort_flag, args.wait_ns)) {
        fail();
        break;
      }
      ptx::tc_fence_after();
      const uint32_t t_acc = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(abuf * BN);
      const int64_t row = static_cast<int64_t>(mt) * 256 + rank * 128 + q * 32 + lane;
      const bool live = row < args.M;
      const int c_lo = half * (C::kOutCols / 2);
      const int64_t col0 = static_cast<int64_t>(nt) * C::kOutCols;
#pragma unroll 1
      for (int c0 = c_lo; c0 < c_lo + C::kOutCols / 2; c0 += 32) {
        const int64_t col = col0 + c0;
        if (col >= args.N) break;  // uniform across the warp
        const int groups = args.N - col >= 32 ? 4 : static_cast<int>((args.N - col) >> 3);
        if constexpr (EPI == kDenseLinear) {
          uint32_t a[32];
          uint4 res[4];
          const bool has_res = MAJOR != kMajorMN && args.residual != nullptr;
          if (has_res && live) {
            const uint4* src = reinterpret_cast<const uint4*>(args.residual + row * args.ldr + col);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (i < groups) res[i] = src[i];
          }
          if (nk > 0) {
            tmem_ld(t_acc + c0, a);
            ptx::tmem_wait_ld();
            pin(a);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) a[j] = 0u;
          }
          with_act(MAJOR == kMajorKK ? args.act : MOE_EPI_NONE, [&](auto act) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (live && i < groups) {
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(a[8 * i + j]);
                if constexpr (MAJOR == kMajorKK) {
                  if (args.bias != nullptr) {
                    float b[8];
                    unpack8<kFp16>(*reinterpret_cast<const uint4*>(args.bias + col + 8 * i), b);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] += b[j];
                  }
                  if (args.pre != nullptr)
                    *reinterpret_cast<uint4*>(args.pre + row * args.ldp + col + 8 * i) = pack8<kFp16>(v);
#pragma unroll
                  for (int j = 0; j < 8; ++j) v[j] = act_value(v[j], decltype(act)::value);
                }
                if (has_res) {
                  float r[8];
                  unpack8<kFp16>(res[i], r);
#pragma unroll
                  for (int j = 0; j < 8; ++j) v[j] += r[j];
                }
                *reinterpret_cast<uint4*>(args.out + row * args.ldo + col + 8 * i) = pack8<kFp16>(v);
              }
            }
          });
        } else if constexpr (EPI == kDenseGate) {
          uint32_t g[32], u[32];
          tmem_ld(t_acc + c0, g);
          tmem_ld(t_acc + BN / 2 + c0, u);
          ptx::tmem_wait_ld();
          pin(g);
          pin(u);
          with_act(args.act, [&](auto act) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (live && i < groups) {
                float gv[8], uv[8], h[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  gv[j] = __uint_as_float(g[8 * i + j]);
                  uv[j] = __uint_as_float(u[8 * i + j]);
                  h[j] = act_value(gv[j], decltype(act)::value) * uv[j];
                }
                if (args.pre != nullptr) {
                  uint16_t* p = args.pre + row * args.ldp + col + 8 * i;
                  *reinterpret_cast<uint4*>(p) = pack8<kFp16>(gv);
                  *reinterpret_cast<uint4*>(p + args.N) = pack8<kFp16>(uv);
                }
                *reinterpret_cast<uint4*>(args.out + row * args.ldo + col + 8 * i) = pack8<kFp16>(h);
              }
            }
          });
        } else {
          uint32_t a[32];
          uint4 pg[4], pu[4];
          if (live) {
            const uint16_t* p = args.pre + row * args.ldp + col;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (i < groups) {
                pg[i] = *reinterpret_cast<const uint4*>(p + 8 * i);
                pu[i] = *reinterpret_cast<const uint4*>(p + args.N + 8 * i);
              }
          }
          tmem_ld(t_acc + c0, a);
          ptx::tmem_wait_ld();
          pin(a);
          with_act(args.act, [&](auto act) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (live && i < groups) {
                float g[8], u[8], h[8], dg[8], du[8];
                unpack8<kFp16>(pg[i], g);
                unpack8<kFp16>(pu[i], u);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  const float dh = __uint_as_float(a[8 * i + j]);
                  float slope;
                  const float v = act_value_slope(g[j], decltype(act)::value, &slope);
                  h[j] = v * u[j];
                  dg[j] = dh * u[j] * slope;
                  du[j] = dh * v;
                }
                uint16_t* p = args.out + row * args.ldo + col + 8 * i;
                *reinterpret_cast<uint4*>(p) = pack8<kFp16>(dg);
                *reinterpret_cast<uint4*>(p + args.N) = pack8<kFp16>(du);
                *reinterpret_cast<uint4*>(args.out2 + row * args.N + col + 8 * i) = pack8<kFp16>(h);
              }
            }
          });
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_leader(&tempty[abuf]);
      if (++abuf == 2) {
        abuf = 0;
        aphase ^= 1u;
      }
    }
  }

  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();  // the peer's last arrivals and reads are done
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem_base, C::kTmemCols);
  }
}

// Bytes of dynamic shared memory opted into once per device and kernel;
// concurrent first calls may both set it (idempotent).
template <class Kernel>
cudaError_t allow_smem(Kernel kern, int bytes, std::atomic<bool>* done) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev].load(std::memory_order_acquire)) {
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err != cudaSuccess) return err;
    done[dev].store(true, std::memory_order_release);
  }
  return cudaSuccess;
}

template <int EPI, int MAJOR, int BN, bool kFp16>
cudaError_t launch_variant(const DenseProblem& p, int num_sms, cudaStream_t stream) {
  using C = Cfg<EPI, MAJOR, BN>;
  auto kern = dense_gemm_kernel<EPI, MAJOR, BN, kFp16>;
  static std::atomic<bool> attr_done[64];
  cudaError_t err = allow_smem(kern, C::kSmemBytes, attr_done);
  if (err != cudaSuccess) return err;
  Args a = {};
  const uint64_t M = p.M, N = p.N, K = p.K;
  // With nothing to contract no load is issued; the maps then describe one row.
  const uint64_t Kd = K > 0 ? K : 8;
  bool ok;
  if (C::kAMn) {
    const uint64_t dims[2] = {M, Kd}, st[1] = {static_cast<uint64_t>(p.lda) * 2};
    const uint32_t box[2] = {64, 64};
    ok = encode_16bit(&a.tm_a, kFp16, p.a, 2, dims, st, box);
  } else {
    const uint64_t dims[2] = {Kd, M}, st[1] = {static_cast<uint64_t>(p.lda) * 2};
    const uint32_t box[2] = {64, 128};
    ok = encode_16bit(&a.tm_a, kFp16, p.a, 2, dims, st, box);
  }
  if (EPI == kDenseGate) {
    const uint64_t dims[3] = {Kd, N, 2}, st[2] = {static_cast<uint64_t>(p.ldb) * 2, static_cast<uint64_t>(p.ldb) * 2 * N};
    const uint32_t box[3] = {64, BN / 2, 1};
    ok = ok && encode_16bit(&a.tm_b, kFp16, p.b, 3, dims, st, box);
  } else if (C::kBMn) {
    const uint64_t dims[2] = {N, Kd}, st[1] = {static_cast<uint64_t>(p.ldb) * 2};
    const uint32_t box[2] = {64, 64};
    ok = ok && encode_16bit(&a.tm_b, kFp16, p.b, 2, dims, st, box);
  } else {
    const uint64_t dims[2] = {Kd, N}, st[1] = {static_cast<uint64_t>(p.ldb) * 2};
    const uint32_t box[2] = {64, BN / 2};
    ok = ok && encode_16bit(&a.tm_b, kFp16, p.b, 2, dims, st, box);
  }
  if (!ok) return cudaErrorInvalidValue;
  a.M = p.M;
  a.N = p.N;
  a.ldr = p.ldr;
  a.ldo = p.ldo;
  a.ldp = p.ldp;
  a.nk = static_cast<int>((p.K + 63) / 64);
  a.n_mt = static_cast<int>((p.M + 255) / 256);
  a.n_nt = static_cast<int>((p.N + C::kOutCols - 1) / C::kOutCols);
  a.bias = static_cast<const uint16_t*>(p.bias);
  a.residual = static_cast<const uint16_t*>(p.residual);
  a.out = static_cast<uint16_t*>(p.out);
  a.pre = static_cast<uint16_t*>(p.pre);
  a.out2 = static_cast<uint16_t*>(p.out2);
  a.act = p.act;
  a.status = p.status;
  a.wait_ns = launch_wait_limit_ns();
  a.tfull_surplus = launch_unreachable_arrivals();
  const int64_t tiles = static_cast<int64_t>(a.n_mt) * a.n_nt;
  const int pairs = static_cast<int>(tiles < num_sms / 2 ? tiles : num_sms / 2);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(C::kNumThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace dense

// One translation unit per kind.
cudaError_t launch_dense_linear(const DenseProblem& p, int num_sms, cudaStream_t stream);
cudaError_t launch_dense_dx(const DenseProblem& p, int num_sms, cudaStream_t stream);
cudaError_t launch_dense_dw(const DenseProblem& p, int num_sms, cudaStream_t stream);
cudaError_t launch_dense_gate(const DenseProblem& p, int num_sms, cudaStream_t stream);
cudaError_t launch_dense_gate_grad(const DenseProblem& p, int num_sms, cudaStream_t stream);

}  // namespace moe
