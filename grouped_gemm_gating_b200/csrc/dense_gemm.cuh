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
// Two accumulators in tensor memory: the epilogue (two groups of four warps,
// each on half of the columns) drains one while the MMA fills the other, 64
// columns at a time.  Matrices move between shared and global memory by TMA
// only, a warp of each group moving them: it fetches what the next chunks add
// (a residual, or g and u) as soon as the buffers' last results have left,
// and stores what the group has written in their place.  A step of 64 of k
// brings each SM 32 KB for 512 clocks of products, so other traffic adds to
// the products' time instead of hiding under it: 8192 x 6144 x 2048 takes
// 134 us as a plain product; dh with [dg | du] and h, 0.5 GB more, 206 us
// (timing-only builds without its loads 173 us, without its stores 154 us,
// without both 126 us; a thread per row instead of TMA 220 us).
//
// Tiles go in groups of row tiles (group_rows), so the pairs at work share
// operand rows in L2.  The tiles that do not fill a last round of
// all pairs are cut into halves of BN / 2 columns when that shortens it.
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

// Row tiles of a group: tiles go column by column within it.  The shorter
// side of the grid of tiles is kept whole, so that its operand stays in L2
// and the other one passes once (measured with groups of 2, 8 and 16: 64 x 8
// tiles at K = 8192 352, 359 and 368 us, a gate of 16 x 96 at K = 4096 585,
// 514 and 502 us, 32 x 32 at K = 8192 763, 693 and 720 us).  Three grids at
// long contractions: the rule goes by tiles alone, not by the bytes that K
// makes of them, and short contractions were not measured.
inline int group_rows(int n_mt, int n_nt) { return n_nt <= 8 ? 2 : n_mt <= 16 ? 16 : 8; }

struct Job {
  CUtensorMap tm_a, tm_b;
  CUtensorMap tm_bh;             // B in boxes of half the rows (half tiles; K-major operands only)
  CUtensorMap tm_out, tm_pre;    // out and pre; gate-grad: da and h
  CUtensorMap tm_res;            // residual; gate-grad: [g | u]
  int64_t M, N;
  int nk, n_mt, n_nt, group;
  int a_mn, b_mn;                // kMajorAny
  const uint16_t* bias;
  int residual, keep_pre;        // tm_res, tm_pre are wanted
};

template <int NJ>
struct Args {
  Job job[NJ];
  int tile0[NJ];                 // first tile of each job; the jobs' tiles are numbered through
  int n_jobs, n_tiles;
  int n_full;                    // whole tiles; the others, the last ones, are cut in two
  int act;
  int32_t* status;
  uint64_t wait_ns;
  int tfull_surplus;
};

template <int EPI, int MAJOR>
struct Cfg {
  static constexpr int BN = 256;
  static constexpr int kJobs = MAJOR == kMajorAny ? kMaxJobs : 1;
  static constexpr int kOutCols = EPI == kDenseGate ? BN / 2 : BN;  // output columns of a tile
  static constexpr int kABytes = 128 * 128;                          // 128 M values x 64 K
  static constexpr int kBBytes = BN / 2 * 128;                       // this CTA's half of B
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kSets = EPI == kDenseGateGrad ? 1 : 2;        // sets of buffers of an epilogue group
  static constexpr int kPerSet = EPI == kDenseGateGrad ? 3 : 1;
  static constexpr int kBufs = kSets * kPerSet;
  static constexpr int kBufBytes = 128 * 128;                        // 128 rows x 64 columns
  static constexpr int kStages = EPI == kDenseGateGrad ? 4 : 5;
  static constexpr int kTmemCols = 2 * BN;
  static constexpr int kNumThreads = 384;  // producer, MMA, eight epilogue warps, two that move their data
  static constexpr int kBarrierBytes = 256;
  static constexpr int kSmemBytes = kStages * kStageBytes + 2 * kBufs * kBufBytes + kBarrierBytes + 1024;
  static_assert((2 * kStages + 13) * 8 + 16 <= kBarrierBytes, "barrier area");
  static_assert(kSmemBytes <= 232448, "shared memory per block");
};

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

template <int EPI, int MAJOR, bool kFp16>
__global__ void __launch_bounds__(Cfg<EPI, MAJOR>::kNumThreads, 1)
    dense_gemm_kernel(const __grid_constant__ Args<Cfg<EPI, MAJOR>::kJobs> args) {
  using C = Cfg<EPI, MAJOR>;
  constexpr int BN = C::BN;
  auto a_mn = [&](const Job& j) { return MAJOR == kMajorAny ? j.a_mn != 0 : MAJOR == kMajorMN; };
  auto b_mn = [&](const Job& j) { return MAJOR == kMajorAny ? j.b_mn != 0 : MAJOR != kMajorKK; };
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* bufs = smem + C::kStages * C::kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(bufs + 2 * C::kBufs * C::kBufBytes);
  uint64_t* empty = full + C::kStages;
  uint64_t* tfull = empty + C::kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* ready = tempty + 2;       // [group][set]: buffers are free, and hold what was to be fetched
  uint64_t* written = ready + 4;      // [group][set]: the group's four warps wrote their results
  uint64_t* mma_done = written + 4;   // the MMA issuer's last commit (drain before TMEM is freed)
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
    for (int i = 0; i < 4; ++i) {
      ptx::mbar_init(&ready[i], 1);
      ptx::mbar_init(&written[i], 4);
    }
    ptx::mbar_init(mma_done, 1);
    *abort_flag = 0;
    *never = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&args.job[0].tm_a);
    ptx::prefetch_tmap(&args.job[0].tm_b);
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

  const int units = args.n_full + 2 * (args.n_tiles - args.n_full);
  // Unit u of work: a whole tile (part < 0) or one of a tile's halves.  The
  // last round, which may be short, is dealt in the opposite order: the first
  // pairs then had the larger units of the rounds before.
  const int last = units - units % n_pairs;
  struct Unit {
    int job, mt, nt, part;
  };
  auto unit_of = [&](int u) {
    Unit r;
    int tile = u;
    r.part = -1;
    if (u >= args.n_full) {
      tile = args.n_full + ((u - args.n_full) >> 1);
      r.part = (u - args.n_full) & 1;
    }
    r.job = 0;
#pragma unroll
    for (int j = 1; j < C::kJobs; ++j)
      if (j < args.n_jobs && tile >= args.tile0[j]) r.job = j;
    const Job& jb = args.job[r.job];
    if (C::kJobs > 1) tile -= args.tile0[r.job];
    const int per_group = jb.group * jb.n_nt;
    const int g = tile / per_group;
    const int m0 = g * jb.group;
    const int gm = jb.n_mt - m0 < jb.group ? jb.n_mt - m0 : jb.group;
    const int i = tile - g * per_group;
    r.nt = i / gm;
    r.mt = m0 + (i - r.nt * gm);
    return r;
  };
  // This pair's i-th unit, or -1.
  auto unit_at = [&](int i) {
    const int u = i * n_pairs + pair;
    if (u < last) return u;
    const int v = i * n_pairs + (n_pairs - 1 - pair);
    return i * n_pairs == last && v < units ? v : -1;
  };
  // Where an epilogue group's share of a unit lies: `chunks` times 64 columns
  // from `col` of the output, from `acc` of the accumulator.  (Half a gate
  // tile has 64 columns: the first group's.)
  struct Place {
    int m0, col, acc, chunks;
  };
  auto place_of = [&](const Unit& t, int group) {
    Place p;
    const bool whole = t.part < 0;
    const int cols = EPI == kDenseGate ? 64 : whole ? 128 : 64;
    p.m0 = t.mt * 256 + rank * 128;
    p.acc = group * cols;
    p.col = t.nt * C::kOutCols + (t.part > 0 ? C::kOutCols / 2 : 0) + p.acc;
    const int64_t left = p.m0 < args.job[t.job].M ? args.job[t.job].N - p.col : 0;
    p.chunks = left <= 0 ? 0 : left >= cols ? cols / 64 : static_cast<int>((left + 63) / 64);
    if (EPI == kDenseGate && !whole && group == 1) p.chunks = 0;
    return p;
  };
  // A chunk is made in passes, one buffer each: pre first when it is kept
  // (gate: g, then u), the output last.  Gate-grad: one pass, three buffers.
  auto passes_of = [&](const Job& jb) {
    return EPI == kDenseGateGrad || !jb.keep_pre ? 1 : EPI == kDenseGate ? 3 : 2;
  };
  auto set_of = [&](int pass) { return C::kSets == 1 ? 0 : pass & 1; };
  auto phase_of = [&](int pass) { return static_cast<uint32_t>((C::kSets == 1 ? pass : pass >> 1) & 1); };
  auto fail = [&]() {
    *abort_flag = 1;
    set_status(args.status, MOE_ERR_DEVICE_TIMEOUT);
  };

  if (warp == 0) {
    // ------------------------------------------------ TMA producer (both CTAs)
    if (ptx::elect_one()) {
      const uint32_t smem0 = ptx::smem_u32(smem);
      const uint32_t full0 = ptx::leader_addr(full);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int issued = 0;  // stages filled so far
      for (int it = 0, u; ok && (u = unit_at(it)) >= 0; ++it) {
        const Unit t = unit_of(u);
        const Job& jb = args.job[t.job];
        const int nk = jb.nk;
        const bool whole = t.part < 0;
        const int width = whole ? BN / 2 : BN / 4;  // B rows of this CTA
        const int m0 = t.mt * 256 + rank * 128;
        const int n0 = EPI == kDenseGate ? t.nt * (BN / 2) + (t.part > 0 ? width : 0)
                                         : t.nt * BN + (t.part > 0 ? BN / 2 : 0) + rank * width;
        const CUtensorMap* tm_b = whole ? &jb.tm_b : &jb.tm_bh;
        const uint32_t bytes = 2u * (C::kABytes + (whole ? C::kBBytes : C::kBBytes / 2));
        for (int kb = 0; kb < nk; ++kb) {
          if (!ptx::mbar_wait_cluster_bounded(&empty[stage], phase ^ 1u, abort_flag, args.wait_ns)) {
            fail();
            ok = false;
            break;
          }
          const uint32_t sA = smem0 + stage * C::kStageBytes;
          const uint32_t sB = sA + C::kABytes;
          const uint32_t bar = full0 + stage * 8;
          if (rank == 0) ptx::mbar_arrive_expect_tx(&full[stage], bytes);
          if (a_mn(jb)) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
              ptx::tma_load_2d_pair_at(sA + j * 8192, &jb.tm_a, bar, m0 + 64 * j, kb * 64);
          } else {
            ptx::tma_load_2d_pair_at(sA, &jb.tm_a, bar, kb * 64, m0);
          }
          if constexpr (EPI == kDenseGate) {
            ptx::tma_load_3d_pair_at(sB, tm_b, bar, kb * 64, n0, rank);
          } else if (b_mn(jb)) {
            ptx::tma_load_2d_pair_at(sB, &jb.tm_b, bar, n0, kb * 64);
            if (whole) ptx::tma_load_2d_pair_at(sB + 8192, &jb.tm_b, bar, n0 + 64, kb * 64);
          } else {
            ptx::tma_load_2d_pair_at(sB, tm_b, bar, kb * 64, n0);
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
    if (rank == 0 && ptx::elect_one()) {
      const uint32_t smem0 = ptx::smem_u32(smem);
      int stage = 0;
      uint32_t phase = 0;
      int abuf = 0;
      uint32_t aphase = 0;
      bool ok = true;
      for (int it = 0, u; ok && (u = unit_at(it)) >= 0; ++it) {
        const Job& jb = args.job[unit_of(u).job];
        const int nk = jb.nk;
        const bool am = a_mn(jb), bm = b_mn(jb);
        const uint32_t idesc = ptx::idesc_16bit_f32(256, u < args.n_full ? BN : BN / 2, kFp16, am, bm);
        const uint64_t desc_a = am ? ptx::sw128_mnmajor_desc(smem0, 8192) : ptx::sw128_kmajor_desc(smem0);
        const uint64_t desc_b = bm ? ptx::sw128_mnmajor_desc(smem0 + C::kABytes, 8192)
                                   : ptx::sw128_kmajor_desc(smem0 + C::kABytes);
        const uint32_t step_a = (am ? 2048 : 32) >> 4, step_b = (bm ? 2048 : 32) >> 4;  // 16 K further
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
          const uint32_t st = static_cast<uint32_t>(stage * C::kStageBytes) >> 4;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            ptx::mma_bf16_pair(d_tmem, desc_a + (st + kk * step_a), desc_b + (st + kk * step_b), idesc,
                               (kb | kk) != 0 ? 1u : 0u);
          ptx::mma_commit_pair(&empty[stage]);
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        ptx::mma_commit_pair(&tfull[abuf]);
        if (++abuf == 2) {
          abuf = 0;
          aphase ^= 1u;
        }
      }
      // no MMA of the pair may still run when TMEM is freed: the last commit
      // arrives on both CTAs' mma_done
      ptx::mma_commit_pair(mma_done);
      if (!ptx::mbar_wait_bounded(mma_done, 0u, never, kDrainLimitNs)) fail();
    }
  } else if (warp >= 10) {
    // ------------------------------------------------ mover of one epilogue group's data
    if (ptx::elect_one()) {
      const int group = warp - 10;
      uint8_t* my_bufs = bufs + group * C::kBufs * C::kBufBytes;
      uint64_t* my_ready = ready + group * 2;
      uint64_t* my_written = written + group * 2;
      int it_f = 0, c_f = 0, s_f = 0, u_f = unit_at(0);  // next pass to make ready
      int asked = 0, stored = 0;                         // passes made ready, passes stored
      auto make_ready = [&]() {
        while (u_f >= 0) {
          const Unit t = unit_of(u_f);
          const Place p = place_of(t, group);
          if (c_f < p.chunks) {
            const Job& jb = args.job[t.job];
            const int set = set_of(asked);
            uint8_t* b = my_bufs + set * C::kPerSet * C::kBufBytes;
            const int col = p.col + c_f * 64;
            const bool last_pass = s_f + 1 == passes_of(jb);
            if constexpr (EPI == kDenseGateGrad) {
              ptx::mbar_arrive_expect_tx(&my_ready[set], 2 * C::kBufBytes);
              ptx::tma_load_3d(b, &jb.tm_res, &my_ready[set], col, 0, p.m0);
              ptx::tma_load_3d(b + C::kBufBytes, &jb.tm_res, &my_ready[set], col, 1, p.m0);
            } else if (EPI == kDenseLinear && jb.residual && last_pass) {
              ptx::mbar_arrive_expect_tx(&my_ready[set], C::kBufBytes);
              ptx::tma_load_2d(b, &jb.tm_res, &my_ready[set], col, p.m0);
            } else {
              ptx::mbar_arrive(&my_ready[set]);
            }
            ++asked;
            if (last_pass) {
              s_f = 0;
              ++c_f;
            } else {
              ++s_f;
            }
            return;
          }
          c_f = 0;
          u_f = unit_at(++it_f);
        }
      };
      for (int i = 0; i < C::kSets; ++i) make_ready();
      bool ok = true;
      for (int it = 0, u; ok && (u = unit_at(it)) >= 0; ++it) {
        const Unit t = unit_of(u);
        const Job& jb = args.job[t.job];
        const Place p = place_of(t, group);
        const int passes = passes_of(jb);
        for (int c = 0; ok && c < p.chunks; ++c) {
          const int col = p.col + c * 64;
          for (int s = 0; s < passes; ++s) {
            const int set = set_of(stored);
            if (!ptx::mbar_wait_bounded(&my_written[set], phase_of(stored), abort_flag, args.wait_ns)) {
              fail();
              ok = false;
              break;
            }
            const uint8_t* b = my_bufs + set * C::kPerSet * C::kBufBytes;
            if constexpr (EPI == kDenseGateGrad) {
              ptx::tma_store_3d(&jb.tm_out, b, col, 0, p.m0);
              ptx::tma_store_3d(&jb.tm_out, b + C::kBufBytes, col, 1, p.m0);
              ptx::tma_store_2d(&jb.tm_pre, b + 2 * C::kBufBytes, col, p.m0);
            } else if (s + 1 == passes) {
              ptx::tma_store_2d(&jb.tm_out, b, col, p.m0);
            } else if (EPI == kDenseGate) {
              ptx::tma_store_3d(&jb.tm_pre, b, col, s, p.m0);
            } else {
              ptx::tma_store_2d(&jb.tm_pre, b, col, p.m0);
            }
            ptx::bulk_commit();
            ++stored;
            ptx::bulk_wait_read();
            make_ready();
          }
        }
      }
      // what was asked for lands, what was stored has left, before shared memory is given up
      for (int i = stored; i < asked; ++i)
        ptx::mbar_wait_bounded(&my_ready[set_of(i)], phase_of(i), never, kDrainLimitNs);
      ptx::bulk_wait();
    }
  } else {
    // ------------------------------------------------ epilogue (both CTAs, own TMEM half)
    const int q = warp & 3;
    const int group = (warp - 2) >> 2;
    const int r128 = q * 32 + lane;  // this thread's row of the CTA's 128
    uint8_t* my_bufs = bufs + group * C::kBufs * C::kBufBytes;
    // 16-byte cell j (8 columns) of this thread's row in buffer b
    auto cell = [&](int b, int j) {
      return reinterpret_cast<uint4*>(my_bufs + b * C::kBufBytes + r128 * 128 + ((j ^ (r128 & 7)) << 4));
    };
    int abuf = 0;
    uint32_t aphase = 0;
    int seq = 0;  // passes done
    bool ok = true;
    for (int it = 0, u; ok && (u = unit_at(it)) >= 0; ++it) {
      const Unit t = unit_of(u);
      const Job& jb = args.job[t.job];
      const Place p = place_of(t, group);
      bool bad = false;
      if (lane == 0) bad = !ptx::mbar_wait_cluster_bounded(&tfull[abuf], aphase, abort_flag, args.wait_ns);
      if (__any_sync(0xffffffffu, bad)) {
        fail();
        break;
      }
      __syncwarp();  // orders what lane 0 waited for before the other lanes' reads (a vote orders nothing)
      ptx::tc_fence_after();
      const uint32_t t_acc =
          tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(abuf * BN + p.acc);
      const int passes = passes_of(jb);
      const int n_steps = p.chunks * passes;
#pragma unroll 1
      for (int i2 = 0; i2 < n_steps; ++i2) {
        const int c = passes == 1 ? i2 : passes == 2 ? i2 >> 1 : i2 / 3;
        const int pass = i2 - c * passes;
        const bool last_pass = pass + 1 == passes;
        const int set = set_of(seq);
        const int b = set * C::kPerSet;
        if (lane == 0)
          bad = !ptx::mbar_wait_bounded(&ready[group * 2 + set], phase_of(seq), abort_flag, args.wait_ns);
        if (__any_sync(0xffffffffu, bad)) {
          fail();
          ok = false;
          break;
        }
        __syncwarp();  // the same for the residual, or g and u, that TMA wrote
#pragma unroll 1
        for (int s = 0; s < 2; ++s) {
          const int col = p.col + c * 64 + s * 32;
          const uint32_t at = t_acc + c * 64 + s * 32;
          uint32_t a[32];
          if constexpr (EPI == kDenseLinear) {
            uint4 bias[4];
            if (MAJOR == kMajorKK && jb.bias != nullptr) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (col + 8 * i < jb.N) bias[i] = *reinterpret_cast<const uint4*>(jb.bias + col + 8 * i);
            }
            tmem_ld(at, a);
            ptx::tmem_wait_ld();
            pin(a);
            with_act(MAJOR == kMajorKK && last_pass ? args.act : MOE_EPI_NONE, [&](auto act) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                F2 v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = f2_bits(a[8 * i + 2 * j], a[8 * i + 2 * j + 1]);
                if constexpr (MAJOR == kMajorKK) {
                  if (jb.bias != nullptr) {
                    F2 bv[4];
                    unpack8<kFp16>(bias[i], bv);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] = v[j] + bv[j];
                  }
#pragma unroll
                  for (int j = 0; j < 4; ++j) v[j] = act_value<decltype(act)::value>(v[j]);
                }
                if (jb.residual && last_pass) {
                  F2 r[4];
                  unpack8<kFp16>(*cell(b, s * 4 + i), r);
#pragma unroll
                  for (int j = 0; j < 4; ++j) v[j] = v[j] + r[j];
                }
                *cell(b, s * 4 + i) = pack8<kFp16>(v);
              }
            });
          } else if constexpr (EPI == kDenseGate) {
            const uint32_t u_at = at + (t.part < 0 ? BN / 2 : BN / 4);
            if (!last_pass) {  // g or u as it is
              tmem_ld(pass == 0 ? at : u_at, a);
              ptx::tmem_wait_ld();
              pin(a);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                F2 v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = f2_bits(a[8 * i + 2 * j], a[8 * i + 2 * j + 1]);
                *cell(b, s * 4 + i) = pack8<kFp16>(v);
              }
            } else {
              uint32_t up[32];
              tmem_ld(at, a);
              tmem_ld(u_at, up);
              ptx::tmem_wait_ld();
              pin(a);
              pin(up);
              with_act(args.act, [&](auto act) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  F2 h[4];
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    h[j] = act_value<decltype(act)::value>(f2_bits(a[8 * i + 2 * j], a[8 * i + 2 * j + 1])) *
                           f2_bits(up[8 * i + 2 * j], up[8 * i + 2 * j + 1]);
                  *cell(b, s * 4 + i) = pack8<kFp16>(h);
                }
              });
            }
          } else {
            tmem_ld(at, a);
            ptx::tmem_wait_ld();
            pin(a);
            with_act(args.act, [&](auto act) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                F2 g[4], up[4], h[4], dg[4], du[4];
                unpack8<kFp16>(*cell(b, s * 4 + i), g);
                unpack8<kFp16>(*cell(b + 1, s * 4 + i), up);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const F2 dh = f2_bits(a[8 * i + 2 * j], a[8 * i + 2 * j + 1]);
                  F2 slope;
                  const F2 v = act_value_slope<decltype(act)::value>(g[j], &slope);
                  h[j] = v * up[j];
                  dg[j] = dh * (up[j] * slope);  // dh u alone may overflow where the slope is 0
                  du[j] = dh * v;
                }
                *cell(b, s * 4 + i) = pack8<kFp16>(dg);
                *cell(b + 1, s * 4 + i) = pack8<kFp16>(du);
                *cell(b + 2, s * 4 + i) = pack8<kFp16>(h);
              }
            });
          }
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&written[group * 2 + set]);
        ++seq;
      }
      if (!ok) break;
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_leader_tmem(&tempty[abuf]);
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
    // The odd CTA outlives the last commit's arrival on its own barrier.  The
    // even CTA has seen its half by now: the wait's limit does not run while
    // the tiles are worked on, however long they take together.
    if (rank != 0 && !ptx::mbar_wait_cluster_bounded(mma_done, 0u, never, kDrainLimitNs)) fail();
    __syncwarp();
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

// 2-D map of a row-major [rows, cols] matrix, or 3-D of [rows, 2, cols] halves.
inline bool encode_rows(CUtensorMap* m, bool fp16, const void* p, uint64_t rows, uint64_t cols, uint64_t ld,
                        uint32_t box_cols, uint32_t box_rows) {
  const uint64_t dims[2] = {cols, rows}, st[1] = {ld * 2};
  const uint32_t box[2] = {box_cols, box_rows};
  return encode_16bit(m, fp16, p, 2, dims, st, box);
}
inline bool encode_halves(CUtensorMap* m, bool fp16, const void* p, uint64_t rows, uint64_t cols, uint64_t ld,
                          uint32_t box_rows) {
  const uint64_t dims[3] = {cols, 2, rows}, st[2] = {cols * 2, ld * 2};
  const uint32_t box[3] = {64, 1, box_rows};
  return encode_16bit(m, fp16, p, 3, dims, st, box);
}

// B's rows in two parts of N each (Wg, Wu).
inline bool encode_parts(CUtensorMap* m, bool fp16, const void* p, uint64_t K, uint64_t N, uint64_t ld,
                         uint32_t box_rows) {
  const uint64_t dims[3] = {K, N, 2}, st[2] = {ld * 2, ld * 2 * N};
  const uint32_t box[3] = {64, box_rows, 1};
  return encode_16bit(m, fp16, p, 3, dims, st, box);
}

template <int EPI, int MAJOR, bool kFp16>
bool make_job(const DenseProblem& p, Job* a) {
  using C = Cfg<EPI, MAJOR>;
  const bool a_mn = p.major == kMajorMN, b_mn = p.major != kMajorKK;
  const uint64_t M = p.M, N = p.N, K = p.K;
  bool ok = a_mn ? encode_rows(&a->tm_a, kFp16, p.a, K, M, p.lda, 64, 64)
                 : encode_rows(&a->tm_a, kFp16, p.a, M, K, p.lda, 64, 128);
  if (EPI == kDenseGate) {
    ok = ok && encode_parts(&a->tm_b, kFp16, p.b, K, N, p.ldb, 128) &&
         encode_parts(&a->tm_bh, kFp16, p.b, K, N, p.ldb, 64);
  } else if (b_mn) {
    ok = ok && encode_rows(&a->tm_b, kFp16, p.b, K, N, p.ldb, 64, 64);
    a->tm_bh = a->tm_b;
  } else {
    ok = ok && encode_rows(&a->tm_b, kFp16, p.b, N, K, p.ldb, 64, 128) &&
         encode_rows(&a->tm_bh, kFp16, p.b, N, K, p.ldb, 64, 64);
  }
  if (EPI == kDenseGateGrad) {
    ok = ok && encode_halves(&a->tm_out, kFp16, p.out, M, N, p.ldo, 128) &&
         encode_rows(&a->tm_pre, kFp16, p.out2, M, N, N, 64, 128) &&
         encode_halves(&a->tm_res, kFp16, p.pre, M, N, p.ldp, 128);
  } else {
    ok = ok && encode_rows(&a->tm_out, kFp16, p.out, M, N, p.ldo, 64, 128);
    a->keep_pre = p.pre != nullptr;
    if (p.pre != nullptr)
      ok = ok && (EPI == kDenseGate ? encode_halves(&a->tm_pre, kFp16, p.pre, M, N, p.ldp, 128)
                                    : encode_rows(&a->tm_pre, kFp16, p.pre, M, N, p.ldp, 64, 128));
  }
  a->residual = p.residual != nullptr;
  if (a->residual) ok = ok && encode_rows(&a->tm_res, kFp16, p.residual, M, N, p.ldr, 64, 128);
  a->M = p.M;
  a->N = p.N;
  a->a_mn = a_mn;
  a->b_mn = b_mn;
  a->nk = static_cast<int>((p.K + 63) / 64);
  a->n_mt = static_cast<int>((p.M + 255) / 256);
  a->n_nt = static_cast<int>((p.N + C::kOutCols - 1) / C::kOutCols);
  a->group = group_rows(a->n_mt, a->n_nt);
  a->bias = static_cast<const uint16_t*>(p.bias);
  return ok;
}

template <int EPI, int MAJOR, bool kFp16>
cudaError_t launch_pair(const DenseProblem* p, int n, int num_sms, cudaStream_t stream) {
  using C = Cfg<EPI, MAJOR>;
  auto kern = dense_gemm_kernel<EPI, MAJOR, kFp16>;
  static std::atomic<bool> attr_done[64];
  cudaError_t err = allow_smem(kern, C::kSmemBytes, attr_done);
  if (err != cudaSuccess) return err;
  Args<C::kJobs> a = {};
  int64_t tiles = 0;
  for (int i = 0; i < n; ++i) {
    if (!make_job<EPI, MAJOR, kFp16>(p[i], &a.job[i])) return cudaErrorInvalidValue;
    a.tile0[i] = static_cast<int>(tiles);
    tiles += static_cast<int64_t>(a.job[i].n_mt) * a.job[i].n_nt;
  }
  a.n_jobs = n;
  a.n_tiles = static_cast<int>(tiles);
  a.act = p[0].act;
  a.status = p[0].status;
  a.wait_ns = launch_wait_limit_ns();
  a.tfull_surplus = launch_unreachable_arrivals();
  const int64_t most = num_sms / 2;
  const int64_t rest = tiles % most;  // halves shorten the last round when they fit into one
  a.n_full = static_cast<int>(2 * rest <= most ? tiles - rest : tiles);
  const int64_t units = a.n_full + 2 * (tiles - a.n_full);
  const int pairs = static_cast<int>(units < most ? units : most);
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

}  // namespace moe
