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

__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case ATTNRES_ACT_GELU:
      return 0.5f * z * (1.f + erff(z * kSqrtHalf));
    case ATTNRES_ACT_GELU_TANH:
      return 0.5f * z * (1.f + tanhf(kSqrt2OverPi * fmaf(kGeluCubic * z * z, z, z)));
    case ATTNRES_ACT_SILU:
      return z / (1.f + __expf(-z));
    default:
      return z;
  }
}

__device__ __forceinline__ float act_slope(int act, float z) {
  switch (act) {
    case ATTNRES_ACT_GELU:
      return fmaf(z * kInvSqrt2Pi, __expf(-0.5f * z * z), 0.5f * (1.f + erff(z * kSqrtHalf)));
    case ATTNRES_ACT_GELU_TANH: {
      const float t = tanhf(kSqrt2OverPi * fmaf(kGeluCubic * z * z, z, z));
      return 0.5f * (1.f + t) + 0.5f * z * (1.f - t * t) * kSqrt2OverPi * fmaf(3.f * kGeluCubic * z, z, 1.f);
    }
    case ATTNRES_ACT_SILU: {
      const float s = 1.f / (1.f + __expf(-z));
      return s * fmaf(z, 1.f - s, 1.f);
    }
    default:
      return 1.f;
  }
}

// One element; returns the unrounded value (for the column sums).
template <typename T, int MODE>
__device__ __forceinline__ float epilogue_one(const LinearEpilogue& e, long long m, int n, float acc) {
  const float z = e.bias ? acc + __ldg(e.bias + n) : acc;
  float v;
  if constexpr (MODE == kEpiDz) {
    v = load_elem(static_cast<const T*>(e.res) + m * e.ldr + n) * act_slope(e.act, z);
  } else {
    v = act_value(e.act, z);
    if (e.res) v += load_elem(static_cast<const T*>(e.res) + m * e.ldr + n);
  }
  store_elem(static_cast<T*>(e.out) + m * e.ldo + n, v);
  return v;
}

}  // namespace attnres
