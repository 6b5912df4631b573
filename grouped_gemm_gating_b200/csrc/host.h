// Host-side helpers shared by the files that implement the C ABI: stage
// profiling, TMA tensor-map encoding, per-device queries.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "common.cuh"

namespace moe {

// Records a pair of CUDA events around the launches made during its life,
// when profiling is on (moe_profile_enable) on this host thread.
struct StageScope {
  int stage = 0;
  cudaEvent_t start = nullptr, stop = nullptr;
  cudaStream_t stream;
  bool active;
  StageScope(int stage, cudaStream_t s);
  ~StageScope();
  StageScope(const StageScope&) = delete;
  StageScope& operator=(const StageScope&) = delete;
};

// Launch count of the last successful call on this host thread.
void record_launches(int n);
moe_status finish(cudaError_t err, int launches);

int num_sms_current_device();

// Tiled tensor map of 16-bit elements, 128-byte swizzle, zero fill out of
// bounds; dims and box innermost first, strides in bytes for dims 1..
bool encode_16bit(CUtensorMap* map, bool fp16, const void* base, int rank, const uint64_t* dims,
                  const uint64_t* strides, const uint32_t* box);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
constexpr size_t kWsAlign = 256;

}  // namespace moe
