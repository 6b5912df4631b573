// The dense GEMMs of dense_gemm.cuh for few rows or few tiles: small tiles,
// the contraction split over the CTAs of a cluster.
//
// Few tokens leave a 256 x 256 tile mostly empty and most SMs without one,
// while the weights still have to come from memory once: the call is bound
// by their bytes (or, small enough, by latency), and every SM has to pull.
// Here a tile is 128 output columns x BT rows, with the roles of the operands
// swapped: the columns' operand (the weights) is the MMA's M = 128 side, the
// rows its N = BT side (16 to 128).  A cluster of S CTAs shares one tile,
// each contracting its part of k; the fp32 parts meet in shared memory, every
// CTA adds the S parts of its share of the columns through distributed shared
// memory, always in the same order, and applies the epilogue to the sum.  No
// workspace, no atomics, the same result on every call.
//
// A gate tile's 128 columns are 64 rows of Wg and the matching 64 of Wu.
#pragma once
#include "dense_gemm.cuh"

namespace moe {
namespace dense {

struct SplitJob {
  CUtensorMap tm_c, tm_r;  // the columns' operand, the rows' operand
  int64_t M, N, ldr, ldo, ldp;
  int nk, n_ct;            // k-blocks; tiles along the columns
  int r_mn;                // kMajorAny: the rows' operand is MN-major too
  int parts;               // parts of k: the cluster's S CTAs, or 1 (each CTA a tile of its own)
  int n_tiles;
  const uint16_t* bias;
  const uint16_t* residual;
  uint16_t* out;
  uint16_t* pre;
  uint16_t* out2;
};

template <int NJ>
struct SplitArgs {
  SplitJob job[NJ];
  int cluster0[NJ];        // first cluster of each job
  int n_jobs;
  int S;                   // CTAs of a cluster
  int act;
  int early;               // columns' operand is not written by the previous kernel of the stream
  int32_t* status;
  uint64_t wait_ns;
  int surplus;
};

template <int EPI, int MAJOR, int BT>
struct SplitCfg {
  static constexpr bool kCMn = MAJOR != kMajorKK;
  static constexpr int kJobs = MAJOR == kMajorAny ? kMaxJobs : 1;
  static constexpr int kOutCols = EPI == kDenseGate ? 64 : 128;
  static constexpr int kCBytes = 128 * 128;
  static constexpr int kRBytes = BT * 128;
  static constexpr int kStageBytes = kCBytes + kRBytes;
  // two CTAs on an SM up to 64 rows, one beyond
  static constexpr int kStages = BT <= 16 ? 6 : BT <= 32 ? 5 : BT <= 64 ? 4 : 6;
  static constexpr int kTmemCols = BT < 32 ? 32 : BT;
  static constexpr int kThreads = 256;
  static constexpr int kPartStride = 132;  // floats between two rows' sums of the 128 columns
  static constexpr int kSmemBytes = kStages * kStageBytes + 256 + 1024;
  static_assert(BT * kPartStride * 4 <= kStages * kStageBytes, "sums reuse the stages");
  static_assert(MAJOR != kMajorAny || BT % 64 == 0, "row operand chunks");
  static_assert(kSmemBytes <= 232448, "shared memory per block");
};

template <bool kFp16>
__device__ __forceinline__ void unpack4(uint2 v, F2 (&f)[2]) {
  f[0] = unpack2<kFp16>(v.x);
  f[1] = unpack2<kFp16>(v.y);
}

template <bool kFp16>
__device__ __forceinline__ void store4(uint16_t* p, const F2 (&f)[2]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2<kFp16>(f[0]), pack2<kFp16>(f[1]));
}

template <int EPI, int MAJOR, int BT, bool kFp16>
__global__ void __launch_bounds__(SplitCfg<EPI, MAJOR, BT>::kThreads)
    dense_split_kernel(const __grid_constant__ SplitArgs<SplitCfg<EPI, MAJOR, BT>::kJobs> args) {
  using C = SplitCfg<EPI, MAJOR, BT>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStageBytes);
  uint64_t* empty = full + C::kStages;
  uint64_t* done = empty + C::kStages;  // every MMA of this CTA
  uint64_t* drain = done + 1;           // the same, without the test hook's surplus
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  volatile int* never = reinterpret_cast<volatile int*>(tmem_holder + 2);

  const int warp = threadIdx.x / kWarp;
  const int lane = threadIdx.x % kWarp;
  const int S = args.S;
  const int cta = static_cast<int>(blockIdx.x) % S;
  const int cluster = static_cast<int>(blockIdx.x) / S;
  int which = 0;
#pragma unroll
  for (int j = 1; j < C::kJobs; ++j)
    if (j < args.n_jobs && cluster >= args.cluster0[j]) which = j;
  const SplitJob& jb = args.job[which];
  const int at = cluster - (C::kJobs > 1 ? args.cluster0[which] : 0);
  const int parts = jb.parts;
  const int tile = parts > 1 ? at : at * S + cta;
  const int rank = parts > 1 ? cta : 0;  // this CTA's part of k
  const bool idle = tile >= jb.n_tiles;  // fills up a cluster
  const bool r_mn = MAJOR == kMajorAny && jb.r_mn;
  const int64_t col0 = static_cast<int64_t>(tile % jb.n_ct) * C::kOutCols;
  const int64_t row0 = static_cast<int64_t>(tile / jb.n_ct) * BT;
  const int kb0 = idle ? 0 : static_cast<int>(static_cast<int64_t>(jb.nk) * rank / parts);
  const int kb1 = idle ? 0 : static_cast<int>(static_cast<int64_t>(jb.nk) * (rank + 1) / parts);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    ptx::mbar_init(done, 1 + args.surplus);
    ptx::mbar_init(drain, 1);
    *abort_flag = 0;
    *never = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&jb.tm_c);
    ptx::prefetch_tmap(&jb.tm_r);
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_holder, C::kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  auto fail = [&]() {
    *abort_flag = 1;
    set_status(args.status, MOE_ERR_DEVICE_TIMEOUT);
  };

  if (warp == 0) {
    if (ptx::elect_one()) {
      // ---------------------------------------------- TMA producer
      auto load_c = [&](int stage, int kb) {
        uint8_t* sC = smem + stage * C::kStageBytes;
        if constexpr (EPI == kDenseGate) {
          ptx::tma_load_3d(sC, &jb.tm_c, &full[stage], kb * 64, static_cast<int>(col0), 0);
          ptx::tma_load_3d(sC + 8192, &jb.tm_c, &full[stage], kb * 64, static_cast<int>(col0), 1);
        } else if constexpr (C::kCMn) {
          ptx::tma_load_2d(sC, &jb.tm_c, &full[stage], static_cast<int>(col0), kb * 64);
          ptx::tma_load_2d(sC + 8192, &jb.tm_c, &full[stage], static_cast<int>(col0) + 64, kb * 64);
        } else {
          ptx::tma_load_2d(sC, &jb.tm_c, &full[stage], kb * 64, static_cast<int>(col0));
        }
      };
      auto load_r = [&](int stage, int kb) {
        uint8_t* sR = smem + stage * C::kStageBytes + C::kCBytes;
        if (MAJOR == kMajorAny && r_mn) {
#pragma unroll
          for (int j = 0; j < BT / 64; ++j)
            ptx::tma_load_2d(sR + j * 8192, &jb.tm_r, &full[stage], static_cast<int>(row0) + 64 * j, kb * 64);
        } else {
          ptx::tma_load_2d(sR, &jb.tm_r, &full[stage], kb * 64, static_cast<int>(row0));
        }
      };
      const int n = kb1 - kb0;
      const int pre = n < C::kStages ? n : C::kStages;
      // Weights that the previous kernel does not write are fetched while it
      // still runs.
      if (args.early)
        for (int i = 0; i < pre; ++i) {
          ptx::mbar_arrive_expect_tx(&full[i], C::kStageBytes);
          load_c(i, kb0 + i);
        }
      pdl_wait();
      pdl_launch_dependents();
      for (int i = 0; i < pre; ++i) {
        if (!args.early) {
          ptx::mbar_arrive_expect_tx(&full[i], C::kStageBytes);
          load_c(i, kb0 + i);
        }
        load_r(i, kb0 + i);
      }
      int issued = pre;
      for (int i = pre; i < n; ++i) {
        const int st = i % C::kStages;
        if (!ptx::mbar_wait_bounded(&empty[st], ((i / C::kStages) & 1) ^ 1u, abort_flag, args.wait_ns)) {
          fail();
          break;
        }
        ptx::mbar_arrive_expect_tx(&full[st], C::kStageBytes);
        load_c(st, kb0 + i);
        load_r(st, kb0 + i);
        ++issued;
      }
      // the last load into every stage lands before shared memory is reused
      for (int i = issued > C::kStages ? issued - C::kStages : 0; i < issued; ++i)
        ptx::mbar_wait_bounded(&full[i % C::kStages], (i / C::kStages) & 1, never, kDrainLimitNs);
    }
  } else if (warp == 1) {
    if (ptx::elect_one()) {
      // ---------------------------------------------- MMA issuer
      const uint32_t smem0 = ptx::smem_u32(smem);
      const uint64_t desc_c = C::kCMn ? ptx::sw128_mnmajor_desc(smem0, 8192) : ptx::sw128_kmajor_desc(smem0);
      const uint64_t desc_r = r_mn ? ptx::sw128_mnmajor_desc(smem0 + C::kCBytes, 8192)
                                   : ptx::sw128_kmajor_desc(smem0 + C::kCBytes);
      constexpr uint32_t kStepC = (C::kCMn ? 2048 : 32) >> 4;  // 16 K further
      const uint32_t step_r = (r_mn ? 2048 : 32) >> 4;
      const uint32_t idesc = ptx::idesc_16bit_f32(128, BT, kFp16, C::kCMn, r_mn);
      for (int i = 0; i < kb1 - kb0; ++i) {
        const int st = i % C::kStages;
        if (!ptx::mbar_wait_bounded(&full[st], (i / C::kStages) & 1, abort_flag, args.wait_ns)) {
          fail();
          break;
        }
        ptx::tc_fence_after();
        const uint32_t off = static_cast<uint32_t>(st * C::kStageBytes) >> 4;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          ptx::mma_bf16(tmem_base, desc_c + (off + kk * kStepC), desc_r + (off + kk * step_r), idesc,
                        (i | kk) != 0 ? 1u : 0u);
        ptx::mma_commit(&empty[st]);
      }
      ptx::mma_commit(done);
      ptx::mma_commit(drain);
      if (!ptx::mbar_wait_bounded(drain, 0u, never, kDrainLimitNs)) fail();
    }
  }
  __syncwarp();
  pdl_wait();  // the epilogue reads what earlier kernels wrote
  if (!ptx::mbar_wait_bounded(done, 0u, abort_flag, args.wait_ns)) fail();
  __syncthreads();  // the stages are free: every load landed, every MMA read them
  ptx::tc_fence_after();

  // ---- this CTA's sums, [row][128 columns], in place of the stages (a job
  // with fewer k-blocks than parts leaves some CTAs none)
  float* part = reinterpret_cast<float*>(smem);
  {
    const int q = warp & 3;
    constexpr int kHalf = BT >= 32 ? BT / 2 : BT;  // rows of a warp
    if (BT >= 32 || warp < 4) {
      const int t0 = (warp >> 2) * kHalf;
      const uint32_t addr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(t0);
      float* dst = part + t0 * C::kPartStride + q * 32 + lane;
#pragma unroll 1
      for (int c = 0; c < kHalf; c += 16) {
        uint32_t a[16];
        ptx::tmem_ld16(addr + c, a);
        ptx::tmem_wait_ld();
        pin(a);
#pragma unroll
        for (int j = 0; j < 16; ++j) dst[(c + j) * C::kPartStride] = kb1 > kb0 ? __uint_as_float(a[j]) : 0.0f;
      }
    }
  }
  ptx::tc_fence_before();
  ptx::cluster_sync();  // every part is there
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, C::kTmemCols);
  }

  // ---- sums over the parts and the epilogue, four columns at a time; this
  // CTA takes an S-th of the tile's columns.  Steps of four items a thread,
  // all their loads before their arithmetic.
  constexpr int kGroups = C::kOutCols / 4;
  const int ng = kGroups / parts;  // powers of two
  const int shift = __ffs(ng) - 1;
  const int live = static_cast<int>(jb.M - row0 < BT ? jb.M - row0 : BT);
  const int items = idle ? 0 : live * ng;
  if (*abort_flag == 0) {
    auto run = [&](auto parts) {
      constexpr int kS = decltype(parts)::value;
      const uint32_t part_addr = ptx::smem_u32(part);
      uint32_t base[kS];
#pragma unroll
      for (int s = 0; s < kS; ++s) base[s] = kS == 1 ? part_addr : ptx::map_rank(part_addr, s);
      auto sum_at = [&](int t, int c, F2 (&v)[2]) {
        const uint32_t off = static_cast<uint32_t>(t * C::kPartStride + c) * 4;
        float4 p[kS];
#pragma unroll
        for (int s = 0; s < kS; ++s)
          p[s] = kS == 1 ? *reinterpret_cast<const float4*>(part + t * C::kPartStride + c)
                         : ptx::ld_cluster_f4(base[s] + off);
        v[0] = f2(p[0].x, p[0].y);
        v[1] = f2(p[0].z, p[0].w);
#pragma unroll
        for (int s = 1; s < kS; ++s) {
          v[0] = v[0] + f2(p[s].x, p[s].y);
          v[1] = v[1] + f2(p[s].z, p[s].w);
        }
      };
      constexpr int kU = 4;
      for (int i0 = threadIdx.x; i0 < items; i0 += kU * C::kThreads) {
        F2 v[kU][2], w[kU][2];
        uint2 x0[kU], x1[kU];  // residual or g; bias or u
        bool on[kU];
        int64_t rows[kU], cols[kU];
#pragma unroll
        for (int k = 0; k < kU; ++k) {
          const int i = i0 + k * C::kThreads;
          const int t = i >> shift;
          const int c = (rank * ng + (i & (ng - 1))) * 4;
          rows[k] = row0 + t;
          cols[k] = col0 + c;
          on[k] = i < items && cols[k] < jb.N;
          if (!on[k]) continue;
          if constexpr (EPI == kDenseLinear) {
            if (jb.residual != nullptr)
              x0[k] = *reinterpret_cast<const uint2*>(jb.residual + rows[k] * jb.ldr + cols[k]);
            if (MAJOR == kMajorKK && jb.bias != nullptr)
              x1[k] = *reinterpret_cast<const uint2*>(jb.bias + cols[k]);
          } else if constexpr (EPI == kDenseGateGrad) {
            const uint16_t* p = jb.pre + rows[k] * jb.ldp + cols[k];
            x0[k] = *reinterpret_cast<const uint2*>(p);
            x1[k] = *reinterpret_cast<const uint2*>(p + jb.N);
          }
        }
#pragma unroll
        for (int k = 0; k < kU; ++k) {
          if (!on[k]) continue;
          const int t = static_cast<int>(rows[k] - row0), c = static_cast<int>(cols[k] - col0);
          sum_at(t, c, v[k]);
          if (EPI == kDenseGate) sum_at(t, c + 64, w[k]);
        }
        with_act(EPI == kDenseLinear && MAJOR != kMajorKK ? MOE_EPI_NONE : args.act, [&](auto act) {
          [[maybe_unused]] constexpr int kAct = decltype(act)::value;
#pragma unroll
          for (int k = 0; k < kU; ++k) {
            if (!on[k]) continue;
            const int64_t row = rows[k], col = cols[k];
            if constexpr (EPI == kDenseLinear) {
              if constexpr (MAJOR == kMajorKK) {
                if (jb.bias != nullptr) {
                  F2 b[2];
                  unpack4<kFp16>(x1[k], b);
#pragma unroll
                  for (int j = 0; j < 2; ++j) v[k][j] = v[k][j] + b[j];
                }
                if (jb.pre != nullptr) store4<kFp16>(jb.pre + row * jb.ldp + col, v[k]);
#pragma unroll
                for (int j = 0; j < 2; ++j) v[k][j] = act_value<kAct>(v[k][j]);
              }
              if (jb.residual != nullptr) {
                F2 r[2];
                unpack4<kFp16>(x0[k], r);
#pragma unroll
                for (int j = 0; j < 2; ++j) v[k][j] = v[k][j] + r[j];
              }
              store4<kFp16>(jb.out + row * jb.ldo + col, v[k]);
            } else if constexpr (EPI == kDenseGate) {
              if (jb.pre != nullptr) {
                store4<kFp16>(jb.pre + row * jb.ldp + col, v[k]);
                store4<kFp16>(jb.pre + row * jb.ldp + jb.N + col, w[k]);
              }
#pragma unroll
              for (int j = 0; j < 2; ++j) v[k][j] = act_value<kAct>(v[k][j]) * w[k][j];
              store4<kFp16>(jb.out + row * jb.ldo + col, v[k]);
            } else {
              F2 g[2], u[2], dg[2], du[2], h[2];
              unpack4<kFp16>(x0[k], g);
              unpack4<kFp16>(x1[k], u);
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                F2 slope;
                const F2 a = act_value_slope<kAct>(g[j], &slope);
                h[j] = a * u[j];
                dg[j] = v[k][j] * (u[j] * slope);  // dh u alone may overflow where the slope is 0
                du[j] = v[k][j] * a;
              }
              store4<kFp16>(jb.out + row * jb.ldo + col, dg);
              store4<kFp16>(jb.out + row * jb.ldo + jb.N + col, du);
              store4<kFp16>(jb.out2 + row * jb.N + col, h);
            }
          }
        });
      }
    };
    switch (parts) {
      case 1: run(std::integral_constant<int, 1>{}); break;
      case 2: run(std::integral_constant<int, 2>{}); break;
      case 4: run(std::integral_constant<int, 4>{}); break;
      default: run(std::integral_constant<int, 8>{}); break;
    }
  }
  if (S > 1) ptx::cluster_sync();  // no CTA leaves while another reads its sums
}

template <int EPI, int MAJOR, int BT, bool kFp16>
cudaError_t launch_split_variant(const DenseProblem* p, int n, int S, const int* parts, cudaStream_t stream) {
  using C = SplitCfg<EPI, MAJOR, BT>;
  auto kern = dense_split_kernel<EPI, MAJOR, BT, kFp16>;
  static std::atomic<bool> attr_done[64];
  cudaError_t err = allow_smem(kern, C::kSmemBytes, attr_done);
  if (err != cudaSuccess) return err;
  SplitArgs<C::kJobs> a = {};
  int64_t clusters = 0;
  for (int i = 0; i < n; ++i) {
    const DenseProblem& q = p[i];
    SplitJob& j = a.job[i];
    const uint64_t M = q.M, N = q.N, K = q.K;
    const bool r_mn = q.major == kMajorMN;
    bool ok = r_mn ? encode_rows(&j.tm_r, kFp16, q.a, K, M, q.lda, 64, 64)
                   : encode_rows(&j.tm_r, kFp16, q.a, M, K, q.lda, 64, BT);
    if (EPI == kDenseGate)
      ok = ok && encode_parts(&j.tm_c, kFp16, q.b, K, N, q.ldb, 64);
    else if (C::kCMn)
      ok = ok && encode_rows(&j.tm_c, kFp16, q.b, K, N, q.ldb, 64, 64);
    else
      ok = ok && encode_rows(&j.tm_c, kFp16, q.b, N, K, q.ldb, 64, 128);
    if (!ok) return cudaErrorInvalidValue;
    j.M = q.M;
    j.N = q.N;
    j.ldr = q.ldr;
    j.ldo = q.ldo;
    j.ldp = q.ldp;
    j.nk = static_cast<int>((q.K + 63) / 64);
    j.n_ct = static_cast<int>((q.N + C::kOutCols - 1) / C::kOutCols);
    j.r_mn = r_mn;
    j.bias = static_cast<const uint16_t*>(q.bias);
    j.residual = static_cast<const uint16_t*>(q.residual);
    j.out = static_cast<uint16_t*>(q.out);
    j.pre = static_cast<uint16_t*>(q.pre);
    j.out2 = static_cast<uint16_t*>(q.out2);
    const int64_t tiles = static_cast<int64_t>(j.n_ct) * ((q.M + BT - 1) / BT);
    j.n_tiles = static_cast<int>(tiles);
    j.parts = parts[i];
    a.cluster0[i] = static_cast<int>(clusters);
    clusters += j.parts > 1 ? tiles : (tiles + S - 1) / S;
  }
  a.n_jobs = n;
  a.S = S;
  a.act = p[0].act;
  a.early = p[0].b_ready;
  a.status = p[0].status;
  a.wait_ns = launch_wait_limit_ns();
  a.surplus = launch_unreachable_arrivals();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * S));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(S);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int EPI, int MAJOR, bool kFp16>
cudaError_t launch_split(const DenseProblem* p, int n, int BT, int S, const int* parts, cudaStream_t stream) {
  if constexpr (MAJOR != kMajorAny) {
    if (BT == 16) return launch_split_variant<EPI, MAJOR, 16, kFp16>(p, n, S, parts, stream);
    if (BT == 32) return launch_split_variant<EPI, MAJOR, 32, kFp16>(p, n, S, parts, stream);
  }
  if (BT == 64) return launch_split_variant<EPI, MAJOR, 64, kFp16>(p, n, S, parts, stream);
  return launch_split_variant<EPI, MAJOR, 128, kFp16>(p, n, S, parts, stream);
}

// Which kernel a launch's problems run on, and how they are cut: the plan of
// the least estimated time.  The estimate's constants (microseconds, bytes a
// microsecond) are fitted to 150 products of 1 to 8192 rows, columns and
// contractions, each timed on the pair kernel and with every BT and S here;
// the plan it picks is within 1.5 % of the fastest one on average, and at
// worst 1.4 times it.  At one row of 2048 x 2048 the pair kernel takes 14 us
// and 16 x 128 tiles in 8 parts 4.3 us; at 512 rows 11.5 and (64 x 128, whole)
// 9.9 us; at 2048 rows 19.5 and 27 us.
struct Plan {
  bool split;
  int bt, s;            // rows of a tile, CTAs of a cluster
  int parts[kMaxJobs];  // parts of k: s or 1
  double us;            // estimate
};

template <int EPI, int MAJOR>
Plan plan_of(const DenseProblem* p, int n, int num_sms) {
  // pair kernel: launch to last store, 64 of k of a tile and of half a tile, whole tiles' longer end
  constexpr double kPairStart = 5.5 + (EPI == kDenseGateGrad ? 1.9 : 0.0), kPairStep = 0.39, kHalfStep = 0.255;
  constexpr double kPairEnd = 1.1, kPairHbm = 3.65e6;
  // here: launch to last store, 64 of k, stages' bytes of all SMs, a row's and a part's epilogue, 128-row tiles
  // (one CTA an SM), a second round of CTAs
  constexpr double kStart = 4.07, kStep = 0.154, kFill = 12.2e6;
  // weights from memory, and what one CTA streams: 134 MB at three rows in
  // 26.4 us by 128 CTAs, 23.9 us by 256; 67 MB in 18.8 us by 64, 14.5 by 128
  constexpr double kHbmFew = 6.0e6, kHbm = 6.7e6, kHbmCta = 0.055e6;
  constexpr double kRow = 0.0081, kJoin = 0.154, kTall = 1.26, kRound = 3.2;
  const int oc = EPI == kDenseGate ? 128 : 256, so = EPI == kDenseGate ? 64 : 128;
  const int most = num_sms / 2;
  Plan best{};
  double best_t, bytes = 0.0;
  {
    int64_t tiles = 0;
    double work = 0.0, longest = 0.0;
    for (int i = 0; i < n; ++i) {
      const int64_t t = ((p[i].M + 255) / 256) * ((p[i].N + oc - 1) / oc);
      const double M = static_cast<double>(p[i].M), N = static_cast<double>(p[i].N), K = static_cast<double>(p[i].K);
      const double nk = static_cast<double>((p[i].K + 63) / 64);
      tiles += t;
      work += static_cast<double>(t) * nk;
      longest = nk > longest ? nk : longest;
      bytes += 2.0 * (M * K + N * K * (EPI == kDenseGate ? 2 : 1) +
                      M * N * (EPI == kDenseGateGrad ? 5 : p[i].residual != nullptr ? 2 : 1));
    }
    if (n == 1) {
      const int64_t rest = tiles % most;
      const bool cut = 2 * rest <= most;
      const int64_t rounds = cut ? tiles / most : (tiles + most - 1) / most;
      best_t = longest * (kPairStep * static_cast<double>(rounds) + (cut && rest ? kHalfStep : 0.0)) +
               (rounds ? kPairEnd : 0.0);
    } else {
      const double even = work / most + 0.5 * longest;
      best_t = kPairStep * (even > longest ? even : longest) + kPairEnd;
    }
    if (best_t < bytes / kPairHbm) best_t = bytes / kPairHbm;
    best_t += kPairStart;
    best.us = best_t;
    if (tiles > 4 * most) return best;  // large: the pair kernel's
  }
  for (int bt = MAJOR == kMajorAny ? 64 : 16; bt <= 128; bt *= 2) {
    const int64_t slots = static_cast<int64_t>(num_sms) * (bt <= 64 ? 2 : 1);
    bool more = false;  // a taller tile would save tiles
    for (int i = 0; i < n; ++i) more |= p[i].M > bt;
    for (int s = 1; s <= 8; s *= 2) {
      // the first m jobs (those of the longest contraction) in s parts
      for (int m = s == 1 ? 0 : 1; m <= (s == 1 ? 0 : n); ++m) {
        int64_t ctas = 0;
        double tiles[kMaxJobs];
        for (int i = 0; i < n; ++i) {
          const int64_t t = ((p[i].M + bt - 1) / bt) * ((p[i].N + so - 1) / so) * (i < m ? s : 1);
          ctas += t;
          tiles[i] = static_cast<double>(t);
        }
        if (ctas > 2 * slots) continue;  // many tiles: the pair kernel's
        double step = static_cast<double>(ctas < slots ? ctas : slots) * (16384 + bt * 128) / kFill;
        if (step < kStep) step = kStep;
        double total = 0.0, longest = 0.0;
        for (int i = 0; i < n; ++i) {
          const int k = i < m ? s : 1;
          const double rows = static_cast<double>(p[i].M < bt ? p[i].M : bt) * (EPI == kDenseGateGrad ? 2 : 1);
          const double t = static_cast<double>((p[i].K + 64 * k - 1) / (64 * k)) * step + kRow * rows / k +
                           (k > 1 ? kJoin * k : 0.0) + (bt == 128 ? kTall : 0.0);
          total += tiles[i] * t;
          longest = t > longest ? t : longest;
        }
        double t = total / static_cast<double>(slots);
        if (t < longest) t = longest;
        if (ctas > slots) t += kRound;
        double rate = ctas > num_sms ? kHbm : kHbmFew;
        if (rate > kHbmCta * static_cast<double>(ctas)) rate = kHbmCta * static_cast<double>(ctas);
        if (t < bytes / rate) t = bytes / rate;
        t += kStart;
        if (t < best_t) {
          best_t = t;
          best.split = true;
          best.bt = bt;
          best.s = s;
          for (int i = 0; i < n; ++i) best.parts[i] = i < m ? s : 1;
        }
      }
    }
    if (!more) break;
  }
  best.us = best_t;
  return best;
}

template <int EPI, int MAJOR>
cudaError_t launch_planned(const DenseProblem* p, int n, const Plan& plan, int num_sms, cudaStream_t stream) {
  if (plan.split)
    return p->fp16 ? launch_split<EPI, MAJOR, true>(p, n, plan.bt, plan.s, plan.parts, stream)
                   : launch_split<EPI, MAJOR, false>(p, n, plan.bt, plan.s, plan.parts, stream);
  return p->fp16 ? launch_pair<EPI, MAJOR, true>(p, n, num_sms, stream)
                 : launch_pair<EPI, MAJOR, false>(p, n, num_sms, stream);
}

// One launch, or two where that saves more than a launch costs the host: the
// first job alone is then better cut than beside the others.  It is the one
// of the longest contraction: dx for few tokens (its contraction is the layer's
// width, twice that of a gated block), a weight gradient where the tokens are
// more.  30 rows of a 2048 -> 6144 block: dx and the weight gradients 85 us in
// one launch, 45 us in two.
template <int EPI, int MAJOR>
cudaError_t launch_kind(const DenseProblem* p, int n, int num_sms, cudaStream_t stream, int* launches) {
  constexpr double kHostLaunch = 2.5;  // microseconds
  const Plan joint = plan_of<EPI, MAJOR>(p, n, num_sms);
  ++*launches;
  if (n > 1) {
    const Plan first = plan_of<EPI, MAJOR>(p, 1, num_sms), others = plan_of<EPI, MAJOR>(p + 1, n - 1, num_sms);
    if (first.us + others.us + kHostLaunch < joint.us) {
      ++*launches;
      cudaError_t err = launch_planned<EPI, MAJOR>(p, 1, first, num_sms, stream);
      if (err != cudaSuccess) return err;
      return launch_planned<EPI, MAJOR>(p + 1, n - 1, others, num_sms, stream);
    }
  }
  return launch_planned<EPI, MAJOR>(p, n, joint, num_sms, stream);
}

}  // namespace dense
}  // namespace moe
