// Activations of the dense operators' epilogues and their derivatives, on two
// fp32 values at a time, and the 16-bit types they read and write.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <type_traits>

#include "common.cuh"

namespace moe {

// Two fp32 values in a register pair; sm_100a adds, multiplies and fuses both
// in one instruction.  An epilogue has few warps beside the product's own, so
// its instructions count (dz at 8192 x 8192 with tanh-gelu: 120 us one value
// at a time, 91 us two).
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 f2(float both) { return f2(both, both); }
__device__ __forceinline__ F2 f2_bits(uint32_t lo, uint32_t hi) { return f2(__uint_as_float(lo), __uint_as_float(hi)); }
__device__ __forceinline__ float2 split(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
template <class F>
__device__ __forceinline__ F2 each(F2 a, F&& f) {
  const float2 p = split(a);
  return f2(f(p.x), f(p.y));
}

// Two 16-bit values of a packed word as fp32, and back (round to nearest even).
template <bool kFp16>
__device__ __forceinline__ F2 unpack2(uint32_t v) {
  if constexpr (kFp16) {
    const float2 p = __half22float2(*reinterpret_cast<__half2*>(&v));
    return f2(p.x, p.y);
  }
  return f2_bits(v << 16, v & 0xffff0000u);
}

template <bool kFp16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (kFp16) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  return pack_bf16x2(lo, hi);
}
template <bool kFp16>
__device__ __forceinline__ uint32_t pack2(F2 a) {
  const float2 p = split(a);
  return pack2<kFp16>(p.x, p.y);
}

template <bool kFp16>
__device__ __forceinline__ void unpack8(uint4 v, F2 (&f)[4]) {
  f[0] = unpack2<kFp16>(v.x);
  f[1] = unpack2<kFp16>(v.y);
  f[2] = unpack2<kFp16>(v.z);
  f[3] = unpack2<kFp16>(v.w);
}
template <bool kFp16>
__device__ __forceinline__ uint4 pack8(const F2 (&f)[4]) {
  return make_uint4(pack2<kFp16>(f[0]), pack2<kFp16>(f[1]), pack2<kFp16>(f[2]), pack2<kFp16>(f[3]));
}

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kSqrtHalf = 0.70710678118654752f;       // 1 / sqrt(2)
constexpr float kInvSqrt2Pi = 0.39894228040143268f;     // 1 / sqrt(2 pi)
constexpr float kTwoSqrt2OverPi = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

// 1 / (1 + 2^w), by the hardware's approximate 2^x and reciprocal (a few fp32
// ulp; every result is rounded to 8 or 11 bits soon after).  2^w = inf gives
// 0; a sigmoid below the smallest normal number counts as 0.
__device__ __forceinline__ float rcp_1p_exp2(float w) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(w));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}
__device__ __forceinline__ F2 rcp_1p_exp2(F2 w) {
  return each(w, [](float x) { return rcp_1p_exp2(x); });
}

// silu: sigmoid(z).  gelu_tanh: (1 + tanh v) / 2 = sigmoid(2 v), with z^2
// held at 400: beyond |z| = 20 the sigmoid is 0 or 1 either way, and an
// overflowing square would turn 0 * inf into NaN in the slope.
__device__ __forceinline__ F2 silu_gate(F2 z) { return rcp_1p_exp2(z * f2(-kLog2E)); }
__device__ __forceinline__ F2 square_to_400(F2 z) {
  return each(z * z, [](float x) { return fminf(x, 400.0f); });
}
__device__ __forceinline__ F2 gelu_tanh_gate(F2 z, F2 z2) {
  constexpr float c = -kTwoSqrt2OverPi * kLog2E;
  return rcp_1p_exp2(z * fma2(z2, f2(c * kGeluCubic), f2(c)));
}

// gelu: the normal distribution Phi(z), by Abramowitz and Stegun 7.1.26 (a
// polynomial in 1 / (1 + p x) times e^-x^2 with x = |z| / sqrt 2; Phi within
// 7.5e-8), and e^(-z^2 / 2), which its density needs too.
__device__ __forceinline__ F2 normal_cdf(F2 z, F2* e) {
  const F2 x = each(z, [](float v) { return fabsf(v); }) * f2(kSqrtHalf);
  const F2 t = each(fma2(x, f2(0.3275911f), f2(1.0f)), [](float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
  });
  *e = each(z * z * f2(-0.5f * kLog2E), [](float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
  });
  F2 q = fma2(t, f2(0.5f * 1.061405429f), f2(0.5f * -1.453152027f));
  q = fma2(t, q, f2(0.5f * 1.421413741f));
  q = fma2(t, q, f2(0.5f * -0.284496736f));
  q = fma2(t, q, f2(0.5f * 0.254829592f));
  const float2 tail = split(q * t * *e), s = split(z);  // Phi(-|z|)
  return f2(s.x < 0.0f ? tail.x : 1.0f - tail.x, s.y < 0.0f ? tail.y : 1.0f - tail.y);
}

// act(z).  NaN stays NaN.
template <int ACT>
__device__ __forceinline__ F2 act_value(F2 z) {
  if constexpr (ACT == MOE_EPI_SILU) return z * silu_gate(z);
  if constexpr (ACT == MOE_EPI_GELU) {
    F2 e;
    return z * normal_cdf(z, &e);
  }
  if constexpr (ACT == MOE_EPI_GELU_TANH) return z * gelu_tanh_gate(z, square_to_400(z));
  if constexpr (ACT == MOE_EPI_RELU || ACT == MOE_EPI_RELU2) {
    const F2 p = each(z, [](float x) { return x < 0.0f ? 0.0f : x; });
    return ACT == MOE_EPI_RELU ? p : p * p;
  }
  return z;
}

// act(z) and act'(z); the kinks of relu have slope 0.
template <int ACT>
__device__ __forceinline__ F2 act_value_slope(F2 z, F2* slope) {
  if constexpr (ACT == MOE_EPI_SILU) {
    const F2 s = silu_gate(z), v = z * s;
    *slope = fma2(v, fma2(s, f2(-1.0f), f2(1.0f)), s);  // s + z s (1 - s)
    return v;
  }
  if constexpr (ACT == MOE_EPI_GELU) {
    F2 e;
    const F2 phi = normal_cdf(z, &e);
    // z times the density; where e is 0 an infinite z must not meet it
    const F2 zc = each(z, [](float x) { return fminf(fmaxf(x, -20.0f), 20.0f); });
    *slope = fma2(zc * f2(kInvSqrt2Pi), e, phi);
    return z * phi;
  }
  if constexpr (ACT == MOE_EPI_GELU_TANH) {
    const F2 z2 = square_to_400(z), s = gelu_tanh_gate(z, z2), v = z * s;
    const F2 steep = fma2(z2, f2(3.0f * kGeluCubic * kTwoSqrt2OverPi), f2(kTwoSqrt2OverPi));  // (2 v)'
    *slope = fma2(v * fma2(s, f2(-1.0f), f2(1.0f)), steep, s);
    return v;
  }
  if constexpr (ACT == MOE_EPI_RELU) {
    *slope = each(z, [](float x) { return x <= 0.0f ? 0.0f : 1.0f; });
    return act_value<ACT>(z);
  }
  if constexpr (ACT == MOE_EPI_RELU2) {
    const F2 p = act_value<MOE_EPI_RELU>(z);
    *slope = p + p;
    return p * p;
  }
  *slope = f2(1.0f);
  return z;
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
