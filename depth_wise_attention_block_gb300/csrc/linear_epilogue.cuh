// Epilogues of the matrix products of attnres_linear and its backward.
#pragma once

#include "attnres.h"
#include "device_common.cuh"

namespace attnres {

// kEpiForward  out = round(act(acc + bias) + res)   (plain products: no bias, no activation)
// kEpiDz       out = round(res * act'(acc + bias)), res the incoming gradient; unrounded column sums to `part`
enum { kEpiForward = 0, kEpiDz = 1 };

struct LinearEpilogue {
  const float* bias;  // [N] or null
  const void* res;    // [M, N] of the storage type, or null
  long long ldr;
  void* out;
  long long ldo;
  int act;
  float* part;  // kEpiDz: partial rows [tiles][N], or null

  // the same for rows r0 .. of the product, whose first partial row is p0
  template <typename T>
  LinearEpilogue rows_from(long long r0, long long p0, int N) const {
    LinearEpilogue e = *this;
    if (e.res) e.res = static_cast<const T*>(e.res) + r0 * ldr;
    e.out = static_cast<T*>(e.out) + r0 * ldo;
    if (e.part) e.part += p0 * N;
    return e;
  }
};

constexpr float kSqrtHalf = 0.70710678f;
constexpr float kInvSqrt2Pi = 0.39894228f;
constexpr float kSqrt2OverPi = 0.79788456f;
constexpr float kGeluCubic = 0.044715f;

// The activations of values that are stored in bf16 (FAST) and in fp32.

// Phi(z), the normal distribution function, and exp(-z^2 / 2).  FAST: erfc by
// the rational-exponential form 7.1.26 of Abramowitz and Stegun (absolute
// error 1.5e-7, relative below half a bf16 step down to z = -5), which shares
// its exponential with the density that the slope of z Phi(z) needs; library
// erfcf and expf, which keep their digits however far out, cost 2048 x 7168 x
// 7168 in bf16 127 us instead of 120, the backward of 2048 x 7168 x 2048 172
// instead of 143.
template <bool FAST>
__device__ __forceinline__ float normal_cdf(float z, float* gauss) {
  if constexpr (FAST) {
    const float x = fabsf(z) * kSqrtHalf;
    const float t = __fdividef(1.f, fmaf(0.3275911f, x, 1.f));
    const float e = __expf(-x * x);
    const float poly = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f), -0.284496736f), 0.254829592f);
    const float tail = 0.5f * poly * e;  // Phi(-|z|)
    *gauss = e;
    return z < 0.f ? tail : 1.f - tail;
  } else {
    *gauss = expf(-0.5f * z * z);
    return 0.5f * erfcf(-z * kSqrtHalf);
  }
}

// s = 1 / (1 + exp(-v)), and 1 - s, both to their last digits (FAST: to a few
// 2^-22, and s = 0 from v = -87 down)
template <bool FAST>
__device__ __forceinline__ float sigmoid(float v, float* rest) {
  if constexpr (FAST) {
    const float s = __fdividef(1.f, 1.f + __expf(-v));
    *rest = 1.f - s;
    return s;
  } else {
    const float e = expf(-fabsf(v)), d = 1.f / (1.f + e);
    *rest = v < 0.f ? d : e * d;
    return v < 0.f ? e * d : d;
  }
}

// (tanh gelu: (1 + tanh u) / 2 = 1 / (1 + exp(-2u)), which does not cancel)
template <int ACT, bool FAST>
__device__ __forceinline__ float act_value(float z) {
  float rest;
  if constexpr (ACT == ATTNRES_ACT_GELU) {
    return z * normal_cdf<FAST>(z, &rest);
  } else if constexpr (ACT == ATTNRES_ACT_GELU_TANH) {
    return z * sigmoid<FAST>(2.f * kSqrt2OverPi * fmaf(kGeluCubic * z * z, z, z), &rest);
  } else if constexpr (ACT == ATTNRES_ACT_SILU) {
    return z * sigmoid<FAST>(z, &rest);
  } else {
    return z;
  }
}

template <int ACT, bool FAST>
__device__ __forceinline__ float act_slope(float z) {
  float rest;
  if constexpr (ACT == ATTNRES_ACT_GELU) {
    const float p = normal_cdf<FAST>(z, &rest);
    return fmaf(z * kInvSqrt2Pi, rest, p);
  } else if constexpr (ACT == ATTNRES_ACT_GELU_TANH) {
    const float s = sigmoid<FAST>(2.f * kSqrt2OverPi * fmaf(kGeluCubic * z * z, z, z), &rest);
    return s * fmaf(z * rest, 2.f * kSqrt2OverPi * fmaf(3.f * kGeluCubic * z, z, 1.f), 1.f);
  } else if constexpr (ACT == ATTNRES_ACT_SILU) {
    const float s = sigmoid<FAST>(z, &rest);
    return s * fmaf(z, rest, 1.f);
  } else {
    return 1.f;
  }
}

// N values at once: v = act(v) + r, or (kEpiDz) v = r act'(v); the choice of
// the activation stays outside the loops.
template <bool FAST, int MODE, int ACT, int N>
__device__ __forceinline__ void act_each(float* v, const float* r) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = MODE == kEpiDz ? r[i] * act_slope<ACT, FAST>(v[i]) : act_value<ACT, FAST>(v[i]) + r[i];
}
template <typename T, int MODE, int N>
__device__ __forceinline__ void act_apply(int act, float* v, const float* r) {
  constexpr bool kFast = sizeof(T) == 2;
  switch (act) {
    case ATTNRES_ACT_GELU: return act_each<kFast, MODE, ATTNRES_ACT_GELU, N>(v, r);
    case ATTNRES_ACT_GELU_TANH: return act_each<kFast, MODE, ATTNRES_ACT_GELU_TANH, N>(v, r);
    case ATTNRES_ACT_SILU: return act_each<kFast, MODE, ATTNRES_ACT_SILU, N>(v, r);
    default: return act_each<kFast, MODE, ATTNRES_ACT_NONE, N>(v, r);
  }
}

// One element; returns the unrounded value (for the column sums).
template <typename T, int MODE>
__device__ __forceinline__ float epilogue_one(const LinearEpilogue& e, long long m, int n, float acc) {
  float v = e.bias ? acc + __ldg(e.bias + n) : acc;
  const float r = e.res ? load_elem(static_cast<const T*>(e.res) + m * e.ldr + n) : 0.f;
  act_apply<T, MODE, 1>(e.act, &v, &r);
  store_elem(static_cast<T*>(e.out) + m * e.ldo + n, v);
  return v;
}

}  // namespace attnres
