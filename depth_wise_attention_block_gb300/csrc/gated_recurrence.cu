// Gated linear recurrence over packed sequences, its backward, and the form
// for single tokens.  Per channel:
//
//   a_t = sigmoid(f_t),  h_t = a_t h_{t-1} + (1 - a_t) x_t,  out_t = h_t silu(g_t)
//   (without an output gate g: out_t = h_t).
//   backward, last token first: dh_t = dy_t silu(g_t) + a_{t+1} dh_{t+1},
//   dx = (1 - a) dh,  df = dh (h_{t-1} - x) a (1 - a),  dg = dy h silu'(g).
#include <math.h>

#include "attnres.h"
#include "body.h"
#include "device_common.cuh"
#include "launch.h"
#include "vec16.cuh"

namespace attnres {

namespace {

constexpr int kGrChunk = 64;  // rows between two kept states
constexpr int kGrThreads = 128;
constexpr int kGsThreads = 256;

// a = 1 / (1 + e^-f) and rest = 1 - a, neither by a difference.  f below -83
// counts as -83 (a = 1e-36), where e^-f would leave fp32; NaN stays NaN.
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void forget(float f, float* a, float* rest) {
  const float e = expf(min_nan(-f, 83.f));
  *a = 1.f / (1.f + e);
  *rest = e * *a;
}
__device__ __forceinline__ float sigmoid(float z) { return 1.f / (1.f + expf(-z)); }

__device__ __forceinline__ int clamp_row(int r, long long T) { return r < 0 ? 0 : r > T ? (int)T : r; }

// One thread per channel and sequence, token after token.
template <typename T>
__global__ void __launch_bounds__(kGrThreads) gr_forward_kernel(const __grid_constant__ RecurrenceArgs p) {
  const int c = blockIdx.x * kGrThreads + threadIdx.x, n = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  if (c >= p.C) return;
  const long long t0 = p.cu ? clamp_row(p.cu[n], p.T) : 0, t1 = p.cu ? clamp_row(p.cu[n + 1], p.T) : p.T;
  float h = p.s0 ? p.s0[(long long)n * p.C + c] : 0.f;
  for (long long t = t0; t < t1; ++t) {
    if (p.chunk && t % kGrChunk == 0) p.chunk[t / kGrChunk * p.C + c] = h;
    float a, rest;
    forget(load_elem(static_cast<const T*>(p.f) + t * p.fs + c), &a, &rest);
    h = fmaf(a, h, rest * load_elem(static_cast<const T*>(p.x) + t * p.xs + c));
    float o = h;
    if (p.g) {
      const float g = load_elem(static_cast<const T*>(p.g) + t * p.gs + c);
      o *= g * sigmoid(g);
    }
    store_elem(static_cast<T*>(p.out) + t * p.os + c, o);
  }
  if (p.s1) p.s1[(long long)n * p.C + c] = h;
}

template <typename T>
__global__ void __launch_bounds__(kGrThreads) gr_backward_kernel(const __grid_constant__ RecurrenceArgs p) {
  const int c = blockIdx.x * kGrThreads + threadIdx.x, n = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  if (c >= p.C) return;
  const long long t0 = p.cu ? clamp_row(p.cu[n], p.T) : 0, t1 = p.cu ? clamp_row(p.cu[n + 1], p.T) : p.T;
  float G = p.ds1 ? p.ds1[(long long)n * p.C + c] : 0.f;  // the gradient at the state behind the token
  float before[kGrChunk];
  for (long long end = t1; end > t0;) {
    long long begin = (end - 1) / kGrChunk * kGrChunk;
    float h;
    if (begin <= t0) {
      begin = t0;
      h = p.s0 ? p.s0[(long long)n * p.C + c] : 0.f;
    } else {
      h = p.chunk[begin / kGrChunk * p.C + c];
    }
    for (long long t = begin; t < end; ++t) {
      float a, rest;
      forget(load_elem(static_cast<const T*>(p.f) + t * p.fs + c), &a, &rest);
      before[t - begin] = h;
      h = fmaf(a, h, rest * load_elem(static_cast<const T*>(p.x) + t * p.xs + c));
    }
    for (long long t = end - 1; t >= begin; --t) {
      float a, rest;
      forget(load_elem(static_cast<const T*>(p.f) + t * p.fs + c), &a, &rest);
      const float x = load_elem(static_cast<const T*>(p.x) + t * p.xs + c), hp = before[t - begin];
      const float dy = load_elem(static_cast<const T*>(p.dout) + t * p.dos + c);
      float d = dy;
      if (p.g) {
        const float g = load_elem(static_cast<const T*>(p.g) + t * p.gs + c), s = sigmoid(g);
        d *= g * s;
        if (p.dg) store_elem(static_cast<T*>(p.dg) + t * p.dgs + c, dy * fmaf(a, hp, rest * x) * fmaf(g * s, 1.f - s, s));
      }
      const float dh = d + G;
      if (p.dx) store_elem(static_cast<T*>(p.dx) + t * p.dxs + c, rest * dh);
      if (p.df) store_elem(static_cast<T*>(p.df) + t * p.dfs + c, dh * (hp - x) * (a * rest));
      G = a * dh;
    }
    end = begin;
  }
  if (p.ds0) p.ds0[(long long)n * p.C + c] = G;
}

// One token per row: a CTA owns a row's channels, and goes on through the
// later rows of the same slot.
template <typename T>
__global__ void __launch_bounds__(kGsThreads) gr_step_kernel(const __grid_constant__ RecurrenceStepArgs p) {
  __shared__ int next_row;
  const int tid = threadIdx.x, c = blockIdx.x * kGsThreads + tid;
  int row = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  const int slot = p.slots ? __ldg(p.slots + row) : row;
  if (slot < 0 || slot >= p.num_slots) return;  // a padding row
  float* st = p.state + (long long)slot * p.C + c;
  const bool in = c < p.C;
  float h = in ? *st : 0.f;
  if (p.slots) {  // rows of one slot belong to the CTA of the first of them
    bool later = false;
    for (int i = tid; i < row; i += kGsThreads) later |= __ldg(p.slots + i) == slot;
    if (__syncthreads_or(later)) return;
  }
  for (;;) {
    if (in) {
      float a, rest;
      forget(load_elem(static_cast<const T*>(p.f) + row * p.fs + c), &a, &rest);
      h = fmaf(a, h, rest * load_elem(static_cast<const T*>(p.x) + row * p.xs + c));
      float o = h;
      if (p.g) {
        const float g = load_elem(static_cast<const T*>(p.g) + row * p.gs + c);
        o *= g * sigmoid(g);
      }
      store_elem(static_cast<T*>(p.out) + row * p.os + c, o);
    }
    if (!p.slots) break;
    if (tid == 0) next_row = p.B;
    __syncthreads();
    for (int i = row + 1 + tid; i < p.B; i += kGsThreads)
      if (__ldg(p.slots + i) == slot) {
        atomicMin(&next_row, i);
        break;
      }
    __syncthreads();
    row = next_row;
    if (row >= p.B) break;
    __syncthreads();  // every thread has read next_row
  }
  if (in) *st = h;
}

}  // namespace

cudaError_t launch_gated_recurrence(const RecurrenceArgs& a) {
  const dim3 grid((a.C + kGrThreads - 1) / kGrThreads, a.N);
  return a.dtype == ATTNRES_BF16 ? launch_kernel(gr_forward_kernel<bf16_t>, grid, dim3(kGrThreads), 0, a.stream, a)
                                 : launch_kernel(gr_forward_kernel<float>, grid, dim3(kGrThreads), 0, a.stream, a);
}

cudaError_t launch_gated_recurrence_backward(const RecurrenceArgs& a) {
  const dim3 grid((a.C + kGrThreads - 1) / kGrThreads, a.N);
  return a.dtype == ATTNRES_BF16 ? launch_kernel(gr_backward_kernel<bf16_t>, grid, dim3(kGrThreads), 0, a.stream, a)
                                 : launch_kernel(gr_backward_kernel<float>, grid, dim3(kGrThreads), 0, a.stream, a);
}

cudaError_t launch_gated_recurrence_step(const RecurrenceStepArgs& a) {
  const dim3 grid((a.C + kGsThreads - 1) / kGsThreads, a.B);
  return a.dtype == ATTNRES_BF16 ? launch_kernel(gr_step_kernel<bf16_t>, grid, dim3(kGsThreads), 0, a.stream, a)
                                 : launch_kernel(gr_step_kernel<float>, grid, dim3(kGsThreads), 0, a.stream, a);
}

}  // namespace attnres
