// Layer norm of whole rows, and its backward.
//
//   h = (x - m) / sqrt(mean_c (x_c - m)^2 + eps),  y = gain * h + bias.
//   backward: n = gain * dy,  dx = (n - mean(n) - h mean(n h)) / sigma,
//   dgain = sum_t dy h,  dbias = sum_t dy.
//
// The mean is held as the sum of two fp32 numbers: m, the rounded mean, and
// delta, the mean of the differences x - m (exact where m is near x), so rows
// whose mean is far from zero keep their digits.
#include <math.h>

#include "attnres.h"
#include "body.h"
#include "device_common.cuh"
#include "launch.h"
#include "vec16.cuh"

namespace attnres {

namespace {

constexpr int kLnThreads = 256;
constexpr int kLnBlocksPerSm = 4;

struct LnParams {
  const void* x;
  const void* dy;
  void* out;
  long long xs, dys, os;
  const float *gain, *bias;
  long long T;
  int d;
  float eps, inv_d;
  float* part;  // backward: [grid][2][d] partial gain and bias gradients, or null
};

// sums of N values over the CTA, the same in every thread
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float (*red)[N]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  __syncthreads();  // the last sums have been read
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[warp][i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = 0.f;
    for (int w = 0; w < (int)blockDim.x >> 5; ++w) v[i] += red[w][i];
  }
}

// Any width, alignment and stride: one CTA per row, read three times.
template <typename T, bool BWD>
__global__ void __launch_bounds__(kLnThreads) ln_any_kernel(const __grid_constant__ LnParams p) {
  __shared__ float red2[32][2], red3[32][3];
  pdl_wait();
  pdl_trigger();
  float* dg = BWD && p.part ? p.part + (long long)blockIdx.x * 2 * p.d : nullptr;
  float* db = dg ? dg + p.d : nullptr;
  for (int c = threadIdx.x; dg && c < p.d; c += kLnThreads) dg[c] = db[c] = 0.f;
  auto gain = [&](int c) { return p.gain ? __ldg(p.gain + c) : 1.f; };
  for (long long t = blockIdx.x; t < p.T; t += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + t * p.xs;
    const T* dy = BWD ? static_cast<const T*>(p.dy) + t * p.dys : nullptr;
    T* o = static_cast<T*>(p.out) + (p.out ? t * p.os : 0);
    float s1[2] = {0.f, 0.f};  // sum x, sum n
    for (int c = threadIdx.x; c < p.d; c += kLnThreads) {
      s1[0] += load_elem(x + c);
      if (BWD) s1[1] = fmaf(load_elem(dy + c), gain(c), s1[1]);
    }
    block_sums(s1, red2);
    const float m = s1[0] * p.inv_d;
    float s2[3] = {0.f, 0.f, 0.f};  // sum x - m, its squares, sum n (x - m)
    for (int c = threadIdx.x; c < p.d; c += kLnThreads) {
      const float z = load_elem(x + c) - m;
      s2[0] += z;
      s2[1] = fmaf(z, z, s2[1]);
      if (BWD) s2[2] = fmaf(load_elem(dy + c) * gain(c), z, s2[2]);
    }
    block_sums(s2, red3);
    const float delta = s2[0] * p.inv_d;
    const float rstd = rsqrtf(fmaxf(fmaf(-delta, delta, s2[1] * p.inv_d), 0.f) + p.eps);
    if (!BWD) {
      for (int c = threadIdx.x; c < p.d; c += kLnThreads) {
        const float h = ((load_elem(x + c) - m) - delta) * rstd;
        store_elem(o + c, fmaf(h, gain(c), p.bias ? __ldg(p.bias + c) : 0.f));
      }
    } else {
      const float mn = s1[1] * p.inv_d;
      const float mh = (s2[2] * p.inv_d - delta * mn) * rstd;  // mean(n h)
      for (int c = threadIdx.x; c < p.d; c += kLnThreads) {
        const float h = ((load_elem(x + c) - m) - delta) * rstd, g = load_elem(dy + c);
        if (p.out) store_elem(o + c, (fmaf(-h, mh, g * gain(c)) - mn) * rstd);
        if (dg) {
          dg[c] = fmaf(g, h, dg[c]);
          db[c] += g;
        }
      }
    }
  }
}

// gain and bias gradients: the CTAs' partial rows, summed in order (32
// channels x 32 interleaved runs of rows per CTA, whose loads do not wait for
// one another; blockIdx.y: gain or bias)
constexpr int kLnRuns = 32;
__global__ void __launch_bounds__(32 * kLnRuns) ln_dgain_kernel(const float* part, int blocks, int d, float* dgain, float* dbias) {
  __shared__ float sums[kLnRuns][33];
  const int lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane, r = threadIdx.x >> 5;
  float* out = blockIdx.y ? dbias : dgain;
  pdl_wait();
  pdl_trigger();
  if (!out) return;
  float s = 0.f;
  if (c < d) {
#pragma unroll 8
    for (int b = r; b < blocks; b += kLnRuns) s += part[((long long)b * 2 + blockIdx.y) * d + c];
  }
  sums[r][lane] = s;
  __syncthreads();
  s = warp_sum(sums[lane][r]);  // warp r: channel r of the CTA's
  if (lane == 0 && blockIdx.x * 32 + r < d) out[blockIdx.x * 32 + r] = s;
}

}  // namespace

int64_t layer_norm_backward_workspace_bytes(int64_t T, int d) {
  DeviceInfo di;
  if (device_info(&di) != cudaSuccess) return -1;
  (void)T;
  return (int64_t)di.sm_count * kLnBlocksPerSm * 2 * d * 4;
}

cudaError_t launch_layer_norm(const LayerNormArgs& a) {
  const bool dgain = a.backward && (a.dgain || a.dbias);
  if (a.T == 0) {
    for (float* g : {a.dgain, a.dbias})
      if (dgain && g) {
        const cudaError_t e = cudaMemsetAsync(g, 0, (size_t)a.d * 4, a.stream);
        if (e != cudaSuccess) return e;
      }
    return cudaSuccess;
  }
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  LnParams p{a.x, a.dy, a.out, a.xs, a.dys, a.os, a.gain, a.bias, a.T, a.d, a.eps, 1.f / (float)a.d, dgain ? a.workspace : nullptr};
  const long long cap = (long long)di.sm_count * kLnBlocksPerSm;
  const int grid = (int)(a.T < cap ? a.T : cap);
  if (a.dtype == ATTNRES_BF16)
    e = a.backward ? launch_kernel(ln_any_kernel<bf16_t, true>, dim3(grid), dim3(kLnThreads), 0, a.stream, p)
                   : launch_kernel(ln_any_kernel<bf16_t, false>, dim3(grid), dim3(kLnThreads), 0, a.stream, p);
  else
    e = a.backward ? launch_kernel(ln_any_kernel<float, true>, dim3(grid), dim3(kLnThreads), 0, a.stream, p)
                   : launch_kernel(ln_any_kernel<float, false>, dim3(grid), dim3(kLnThreads), 0, a.stream, p);
  if (e != cudaSuccess || !dgain) return e;
  return launch_kernel(ln_dgain_kernel, dim3((a.d + 31) / 32, 2), dim3(32 * kLnRuns), 0, a.stream, (const float*)p.part, grid, a.d,
                       a.dgain, a.dbias);
}

}  // namespace attnres
