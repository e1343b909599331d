// activation.cuh -- the activations of the products' epilogues and their slopes.
#pragma once

#include "common.cuh"

namespace moe {

constexpr float kInvSqrt2Pi = 0.39894228040143268f;  // 1 / sqrt(2 pi)
constexpr float kTanhA = 0.79788456080286536f;       // sqrt(2 / pi)
constexpr float kTanhB = 0.044715f;

// 1 / (1 + exp(-v)); exp overflows to inf and the quotient to 0.
__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

// One value, or two in one instruction.
template <typename T>
__device__ __forceinline__ T all_of(float v);
template <>
__device__ __forceinline__ float all_of<float>(float v) { return v; }
template <>
__device__ __forceinline__ float2 all_of<float2>(float v) { return both(v); }
template <typename F>
__device__ __forceinline__ float each(float v, F f) { return f(v); }
template <typename F>
__device__ __forceinline__ float2 each(float2 v, F f) { return make_float2(f(v.x), f(v.y)); }

// Phi(z) = (1 + erf(z / sqrt 2)) / 2 and e = exp(-z^2 / 2), of one value or two.  For
// x >= 0, Phi(-x) = e R(x) with R smooth and falling like 1 / x: a polynomial of
// degree 8 in t = 1 / (1 + 0.305 x), without a constant, fitted for the least
// largest relative error on [0, 14] (1.6 units of 2^-24; 6.4 with fp32's
// roundings, to which the exponential adds about 2 z^2).  So the tail keeps its
// relative precision, where 1 + erf cancels, and one exponential serves gelu's
// slope too.  (With erff and expf the backward pass' kernel was bound by
// instructions.)
template <typename T>
__device__ __forceinline__ T normal_cdf(T z, T& e) {
  auto k = [](float v) { return all_of<T>(v); };
  const T x = each(z, [](float v) { return fabsf(v); });
  const T t = each(fma2(k(0.305f), x, k(1.f)), [](float v) { return __fdividef(1.f, v); });
  e = each(mul2(mul2(x, x), k(-0.72134752044448170f)), exp2_approx);  // 2^(-x^2 / 2 log2 e)
  T q = fma2(k(0.03669917955994606f), t, k(-0.1529882699251175f));
  q = fma2(q, t, k(0.18571682274341583f));
  q = fma2(q, t, k(-0.03797676041722298f));
  q = fma2(q, t, k(0.12102164328098297f));
  q = fma2(q, t, k(0.10342087596654892f));
  q = fma2(q, t, k(0.12246681749820709f));
  q = fma2(q, t, k(0.12163973599672318f));
  q = mul2(q, mul2(t, e));
  if constexpr (sizeof(T) == 8) return make_float2(z.x < 0.f ? q.x : 1.f - q.x, z.y < 0.f ? q.y : 1.f - q.y);
  else return z < 0.f ? q : 1.f - q;
}

__device__ __forceinline__ float activated(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.f ? z : (z != z ? z : 0.f);  // NaN stays
    case MOE_ACT_GELU_TANH: return z * sigmoid(2.f * kTanhA * (z + kTanhB * z * z * z));  // (1 + tanh(u)) / 2 = sigmoid(2u)
    case MOE_ACT_SILU: return z * sigmoid(z);
    default: return z;
  }
}

template <int N>
__device__ __forceinline__ void activate(float* f, int act) {
  switch (act) {  // uniform over the grid; one loop for each, so that the code that runs is short
    case MOE_ACT_RELU:
#pragma unroll
      for (int j = 0; j < N; ++j) f[j] = activated(f[j], MOE_ACT_RELU);
      break;
    case MOE_ACT_GELU:
      if constexpr (N == 1) {
        float e;
        f[0] *= normal_cdf(f[0], e);
      } else {
        // two values an instruction: 16384 x 128 x 4096, bound by this, 136 -> 113 us
#pragma unroll
        for (int j = 0; j < N; j += 2) {
          float2 e;
          const float2 cdf = normal_cdf(make_float2(f[j], f[j + 1]), e);
          f[j] *= cdf.x;
          f[j + 1] *= cdf.y;
        }
      }
      break;
    case MOE_ACT_GELU_TANH:
#pragma unroll
      for (int j = 0; j < N; ++j) f[j] = activated(f[j], MOE_ACT_GELU_TANH);
      break;
    case MOE_ACT_SILU:
#pragma unroll
      for (int j = 0; j < N; ++j) f[j] = activated(f[j], MOE_ACT_SILU);
      break;
    default: break;
  }
}

__device__ __forceinline__ float slope(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case MOE_ACT_GELU: {
      float e;
      const float cdf = normal_cdf(z, e);
      return fmaf(z * kInvSqrt2Pi, e, cdf);
    }
    case MOE_ACT_GELU_TANH: {
      // s + z s' with s = sigmoid(2u); past 16 the slope is 0 or 1 in fp32, and z's
      // square there would overflow beside s (1 - s) = 0
      z = fabsf(z) > 16.f ? copysignf(16.f, z) : z;
      const float s = sigmoid(2.f * kTanhA * (z + kTanhB * z * z * z));
      return fmaf(z * s * (1.f - s), 2.f * kTanhA * (1.f + 3.f * kTanhB * z * z), s);
    }
    case MOE_ACT_SILU: {
      const float s = sigmoid(z);
      return s * (1.f + z * (1.f - s));
    }
    default: return 1.f;
  }
}

// act(z) and its slope at z, sharing the exponential.
__device__ __forceinline__ void act_and_slope(float z, int act, float& value, float& slope) {
  switch (act) {
    case MOE_ACT_RELU:
      value = z > 0.f ? z : (z != z ? z : 0.f);
      slope = z > 0.f ? 1.f : 0.f;
      break;
    case MOE_ACT_GELU: {
      float e;
      const float cdf = normal_cdf(z, e);
      value = z * cdf;
      slope = fmaf(z * kInvSqrt2Pi, e, cdf);
      break;
    }
    case MOE_ACT_GELU_TANH: {
      const float y = fabsf(z) > 16.f ? copysignf(16.f, z) : z;  // as in slope()
      const float s = sigmoid(2.f * kTanhA * (y + kTanhB * y * y * y));
      value = z * s;
      slope = fmaf(y * s * (1.f - s), 2.f * kTanhA * (1.f + 3.f * kTanhB * y * y), s);
      break;
    }
    case MOE_ACT_SILU: {
      const float s = sigmoid(z);
      value = z * s;
      slope = s * (1.f + z * (1.f - s));
      break;
    }
    default:
      value = z;
      slope = 1.f;
      break;
  }
}

}  // namespace moe
