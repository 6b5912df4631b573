// Activations of the dense operators' epilogues and their derivatives, and
// the 16-bit types they read and write.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <type_traits>

#include "common.cuh"

namespace moe {

// Two 16-bit values of a packed word as fp32, and back (round to nearest even).
template <bool kFp16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (kFp16) return __half22float2(*reinterpret_cast<__half2*>(&v));
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

template <bool kFp16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (kFp16) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  return pack_bf16x2(lo, hi);
}

__device__ __forceinline__ float sigmoid_f(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

constexpr float kSqrtHalf = 0.70710678118654752f;       // 1 / sqrt(2)
constexpr float kInvSqrt2Pi = 0.39894228040143268f;     // 1 / sqrt(2 pi)
constexpr float kTwoSqrt2OverPi = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

// act(z).  __expf and the approximate divide are within a few fp32 ulp (for
// the magnitudes an activation sees); every result is rounded to 8 or 11
// bits right after.  NaN stays NaN.  gelu goes through erfc, which keeps its
// relative precision for negative z; (1 + tanh v) / 2 = sigmoid(2 v).
__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case MOE_EPI_SILU: return __fdividef(z, 1.0f + __expf(-z));
    case MOE_EPI_GELU: return 0.5f * z * erfcf(-kSqrtHalf * z);
    case MOE_EPI_GELU_TANH: return z * sigmoid_f(kTwoSqrt2OverPi * (z + kGeluCubic * z * z * z));
    case MOE_EPI_RELU: return z < 0.0f ? 0.0f : z;
    case MOE_EPI_RELU2: {
      const float p = z < 0.0f ? 0.0f : z;
      return p * p;
    }
    default: return z;
  }
}

// act(z) and act'(z).  The kinks of relu have slope 0.  Where sigmoid is 0 or
// 1 the terms it multiplies by s (1 - s) vanish, so z is clamped there before
// it is squared (an overflow would turn 0 * inf into NaN).
__device__ __forceinline__ float act_value_slope(float z, int act, float* slope) {
  switch (act) {
    case MOE_EPI_SILU: {
      const float s = sigmoid_f(z);
      const float zc = fminf(fmaxf(z, -100.0f), 100.0f);
      *slope = s + zc * s * (1.0f - s);
      return z * s;
    }
    case MOE_EPI_GELU: {
      const float phi = 0.5f * erfcf(-kSqrtHalf * z);
      const float zc = fminf(fmaxf(z, -20.0f), 20.0f);
      *slope = phi + zc * kInvSqrt2Pi * __expf(-0.5f * zc * zc);
      return z * phi;
    }
    case MOE_EPI_GELU_TANH: {
      const float s = sigmoid_f(kTwoSqrt2OverPi * (z + kGeluCubic * z * z * z));
      const float zc = fminf(fmaxf(z, -20.0f), 20.0f);
      *slope = s + zc * s * (1.0f - s) * kTwoSqrt2OverPi * (1.0f + 3.0f * kGeluCubic * zc * zc);
      return z * s;
    }
    case MOE_EPI_RELU:
      *slope = z <= 0.0f ? 0.0f : 1.0f;
      return z < 0.0f ? 0.0f : z;
    case MOE_EPI_RELU2: {
      const float p = z < 0.0f ? 0.0f : z;
      *slope = 2.0f * p;
      return p * p;
    }
    default:
      *slope = 1.0f;
      return z;
  }
}

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

}  // namespace moe
