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

// Phi(z), the normal distribution function, and exp(-z^2 / 2): erfc by the
// rational-exponential form 7.1.26 of Abramowitz and Stegun (absolute error
// 1.5e-7), which shares its exponential with the density that the slope of
// z Phi(z) needs.  Library erff costs the epilogue about twice as much.
__device__ __forceinline__ float normal_cdf(float z, float* gauss) {
  const float x = fabsf(z) * kSqrtHalf;
  const float t = __fdividef(1.f, fmaf(0.3275911f, x, 1.f));
  const float e = __expf(-x * x);
  const float poly = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f), -0.284496736f), 0.254829592f);
  const float tail = 0.5f * poly * e;  // Phi(-|z|)
  *gauss = e;
  return z < 0.f ? tail : 1.f - tail;
}

// tanh(u) = 1 - 2 / (1 + exp(2u)), absolute error of a few 2^-24
__device__ __forceinline__ float tanh_exp(float u) { return 1.f - __fdividef(2.f, 1.f + __expf(2.f * u)); }

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == ATTNRES_ACT_GELU) {
    float g;
    return z * normal_cdf(z, &g);
  } else if constexpr (ACT == ATTNRES_ACT_GELU_TANH) {
    return 0.5f * z * (1.f + tanh_exp(kSqrt2OverPi * fmaf(kGeluCubic * z * z, z, z)));
  } else if constexpr (ACT == ATTNRES_ACT_SILU) {
    return z * __fdividef(1.f, 1.f + __expf(-z));  // (0 from z = -87 down)
  } else {
    return z;
  }
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == ATTNRES_ACT_GELU) {
    float g;
    const float p = normal_cdf(z, &g);
    return fmaf(z * kInvSqrt2Pi, g, p);
  } else if constexpr (ACT == ATTNRES_ACT_GELU_TANH) {
    const float t = tanh_exp(kSqrt2OverPi * fmaf(kGeluCubic * z * z, z, z));
    return 0.5f * (1.f + t) + 0.5f * z * (1.f - t * t) * kSqrt2OverPi * fmaf(3.f * kGeluCubic * z, z, 1.f);
  } else if constexpr (ACT == ATTNRES_ACT_SILU) {
    const float s = __fdividef(1.f, 1.f + __expf(-z));
    return s * fmaf(z, 1.f - s, 1.f);
  } else {
    return 1.f;
  }
}

// N values at once: v = act(v) + r, or (kEpiDz) v = r act'(v); the choice of
// the activation stays outside the loops.
template <int MODE, int ACT, int N>
__device__ __forceinline__ void act_apply(float* v, const float* r) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = MODE == kEpiDz ? r[i] * act_slope<ACT>(v[i]) : act_value<ACT>(v[i]) + r[i];
}
template <int MODE, int N>
__device__ __forceinline__ void act_apply(int act, float* v, const float* r) {
  switch (act) {
    case ATTNRES_ACT_GELU: return act_apply<MODE, ATTNRES_ACT_GELU, N>(v, r);
    case ATTNRES_ACT_GELU_TANH: return act_apply<MODE, ATTNRES_ACT_GELU_TANH, N>(v, r);
    case ATTNRES_ACT_SILU: return act_apply<MODE, ATTNRES_ACT_SILU, N>(v, r);
    default: return act_apply<MODE, ATTNRES_ACT_NONE, N>(v, r);
  }
}

// One element; returns the unrounded value (for the column sums).
template <typename T, int MODE>
__device__ __forceinline__ float epilogue_one(const LinearEpilogue& e, long long m, int n, float acc) {
  float v = e.bias ? acc + __ldg(e.bias + n) : acc;
  const float r = e.res ? load_elem(static_cast<const T*>(e.res) + m * e.ldr + n) : 0.f;
  act_apply<MODE, 1>(e.act, &v, &r);
  store_elem(static_cast<T*>(e.out) + m * e.ldo + n, v);
  return v;
}

}  // namespace attnres
