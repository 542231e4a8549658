// The norm of a list of tensors taken as one vector, and their clipping:
//
//   norm = sqrt(sum g^2),  out = g max_norm / norm where norm > max_norm
//   (out = g otherwise, and where the norm is not finite).
//
// Two launches.  The first forms sums of squares, one fp64 number per CTA;
// in the second every CTA adds these in the same order and scales its part.
// The list travels as a kernel parameter (nothing is copied to the device),
// in groups of tensors.  The tensors are cut into chunks of 1024 16-byte
// vectors, and each CTA owns an even range of them.
//
// Every gradient is read twice and written once: the bound is HBM.  The second
// launch goes through a CTA's range backwards, so what the first one read last
// comes from L2.  822 M elements in 16 bits (1.64 GB), out of place: 766 us with
// eight CTAs to an SM, 95 % of the measured copy bandwidth over the three passes
// (four CTAs: 854; twice the vectors to a thread: no faster).  94 rows of 7168
// in fp32: 12 us on the GPU (10 in place), 8 us in the C call and some 70 in the
// Python binding, which has to look at 188 tensors (in place 94: 63 us a call
// where out of place takes 98).
#include <float.h>
#include <math.h>

#include "attnres.h"
#include "body.h"
#include "device_common.cuh"
#include "launch.h"
#include "vec16.cuh"

namespace attnres {

namespace {

constexpr int kClipThreads = 256;
constexpr int kClipVecs = 4;                            // vectors of a chunk per thread
constexpr int kClipChunk = kClipThreads * kClipVecs;    // vectors
constexpr int kClipBlocksPerSm = 8;
constexpr int kClipFew = 32, kClipSome = 256, kClipMany = 900;  // tensors of one launch (a parameter block holds 32,764 bytes)

// How a tensor is read: `head` elements up to the first 16-byte boundary, the
// vectors behind it, and what is left; or (kScalar: an output lies otherwise
// on those boundaries than its gradient) element by element.
constexpr unsigned char kBf16 = 1, kScalar = 2;

template <int MAX>
struct ClipList {
  const void* in[MAX];
  void* out[MAX];
  long long n[MAX];
  int first[MAX + 1];  // chunks of the tensors before
  unsigned char kind[MAX];
  int count;
};

struct ClipParams {
  double* part;    // [blocks]
  int blocks;
  int add;         // 1: to the sums of the launches before
  float max_norm;
  float* norm;     // or null
};

template <int MAX>
__device__ __forceinline__ int find_tensor(const ClipList<MAX>& l, int chunk) {
  int lo = 0, hi = l.count;  // first[lo] <= chunk < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (l.first[mid] <= chunk) lo = mid; else hi = mid;
  }
  return lo;
}

template <typename T>
__device__ __forceinline__ int head_elems(const void* p, long long n) {
  const int h = (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int)sizeof(T);
  return h < n ? h : (int)n;
}

// f(value) over the elements of chunk c of a tensor that this thread owns
template <typename T, typename F>
__device__ __forceinline__ void each_square(const void* in, long long n, int c, bool scalar, F&& f) {
  constexpr int E = Vec16<T>::kElems;
  const T* x = static_cast<const T*>(in);
  if (scalar) {
    for (int i = threadIdx.x; i < kClipChunk * E; i += kClipThreads) {
      const long long at = (long long)c * kClipChunk * E + i;
      if (at < n) f(load_elem(x + at));
    }
    return;
  }
  const int head = head_elems<T>(in, n);
  const long long nv = (n - head) / E, v0 = (long long)c * kClipChunk + threadIdx.x;
  const uint4* xv = reinterpret_cast<const uint4*>(x + head);
  uint4 v[kClipVecs];
#pragma unroll
  for (int k = 0; k < kClipVecs; ++k) v[k] = v0 + k * kClipThreads < nv ? __ldg(xv + v0 + k * kClipThreads) : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int k = 0; k < kClipVecs; ++k) {
    float e[E];
    Vec16<T>::unpack(v[k], e);
#pragma unroll
    for (int i = 0; i < E; ++i) f(e[i]);
  }
  if (c == 0) {
    if ((int)threadIdx.x < head) f(load_elem(x + threadIdx.x));
    const long long tail = head + nv * E + threadIdx.x;
    if (tail < n) f(load_elem(x + tail));
  }
}

__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < kClipThreads / 32; ++w) v += red[w];
  return v;
}

// A chunk's squares are added in fp32 and then to the thread's fp64 sum.
// Where fp32 does not hold them (a sum above 2^120, or below 2^-90 although
// something is not zero) they are added again in fp64.
template <typename T>
__device__ __forceinline__ double chunk_squares(const void* in, long long n, int c, bool scalar) {
  float s = 0.f;
  uint32_t any = 0;
  each_square<T>(in, n, c, scalar, [&](float v) {
    s = fmaf(v, v, s);
    any |= __float_as_uint(v) << 1;
  });
  if (s <= 0x1p120f && (s >= 0x1p-90f || any == 0)) return (double)s;
  double d = 0.0;
  each_square<T>(in, n, c, scalar, [&](float v) { d = fma((double)v, (double)v, d); });
  return d;
}

template <int MAX>
__global__ void __launch_bounds__(kClipThreads) clip_norm_kernel(const __grid_constant__ ClipList<MAX> l, const __grid_constant__ ClipParams p) {
  __shared__ double red[kClipThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int chunks = l.first[l.count];
  const int c0 = (int)((long long)chunks * blockIdx.x / gridDim.x), c1 = (int)((long long)chunks * (blockIdx.x + 1) / gridDim.x);
  double s = 0.0;
  if (c0 < c1) {
    int i = find_tensor(l, c0);
    for (int c = c0; c < c1; ++c) {
      while (c >= l.first[i + 1]) ++i;
      const bool scalar = l.kind[i] & kScalar;
      s += l.kind[i] & kBf16 ? chunk_squares<bf16_t>(l.in[i], l.n[i], c - l.first[i], scalar)
                             : chunk_squares<float>(l.in[i], l.n[i], c - l.first[i], scalar);
    }
  }
  s = block_sum(s, red);
  if (threadIdx.x == 0) p.part[blockIdx.x] = p.add ? p.part[blockIdx.x] + s : s;
}

// the sums of all CTAs, added in the same order everywhere
__device__ __forceinline__ double total_norm(const ClipParams& p, double* red) {
  double s = 0.0;
  for (int i = threadIdx.x; i < p.blocks; i += kClipThreads) s += p.part[i];
  return sqrt(block_sum(s, red));
}

// what the caller reads: a norm that is finite but above fp32's numbers is the
// largest of them (an infinity says that nothing was scaled)
__device__ __forceinline__ void put_norm(float* to, double norm) {
  *to = isfinite(norm) ? (float)fmin(norm, (double)FLT_MAX) : (float)norm;
}

__global__ void __launch_bounds__(kClipThreads) clip_total_kernel(const __grid_constant__ ClipParams p) {
  __shared__ double red[kClipThreads / 32];
  pdl_wait();
  pdl_trigger();
  const double norm = total_norm(p, red);
  if (threadIdx.x == 0) put_norm(p.norm, norm);
}

// max_norm / norm as a product of two fp32 numbers. Below 2^-126 one would lose
// digits, or be zero, although the results are numbers of fp32: the first is
// then a power of two, by which no value loses anything that its result shows
// (what is rounded away of it, 2^-150 at most, meets a second one below 2^-26).
struct Factor {
  float first, second;
  __device__ __forceinline__ explicit Factor(double ratio)
      : first(ratio >= 0x1p-126 ? 1.f : ratio >= 0x1p-226 ? 0x1p-100f : 0x1p-149f), second((float)(ratio / (double)first)) {}
  __device__ __forceinline__ bool one() const { return second == 1.f; }
  __device__ __forceinline__ float times(float v) const { return v * first * second; }
};

template <typename T>
__device__ __forceinline__ void scale_chunk(const void* in, void* out, long long n, int c, bool scalar, const Factor& factor) {
  constexpr int E = Vec16<T>::kElems;
  const T* x = static_cast<const T*>(in);
  T* y = static_cast<T*>(out);
  if (scalar) {
    for (int i = threadIdx.x; i < kClipChunk * E; i += kClipThreads) {
      const long long at = (long long)c * kClipChunk * E + i;
      if (at < n) store_elem(y + at, factor.times(load_elem(x + at)));
    }
    return;
  }
  const int head = head_elems<T>(in, n);
  const long long nv = (n - head) / E, v0 = (long long)c * kClipChunk + threadIdx.x;
  const uint4* xv = reinterpret_cast<const uint4*>(x + head);
  uint4* yv = reinterpret_cast<uint4*>(y + head);
  uint4 v[kClipVecs];
#pragma unroll
  for (int k = 0; k < kClipVecs; ++k)
    if (v0 + k * kClipThreads < nv) v[k] = xv[v0 + k * kClipThreads];
#pragma unroll
  for (int k = 0; k < kClipVecs; ++k)
    if (v0 + k * kClipThreads < nv) {
      float e[E];
      Vec16<T>::unpack(v[k], e);
#pragma unroll
      for (int i = 0; i < E; ++i) e[i] = factor.times(e[i]);
      yv[v0 + k * kClipThreads] = Vec16<T>::pack(e);
    }
  if (c == 0) {
    if ((int)threadIdx.x < head) store_elem(y + threadIdx.x, factor.times(load_elem(x + threadIdx.x)));
    const long long tail = head + nv * E + threadIdx.x;
    if (tail < n) store_elem(y + tail, factor.times(load_elem(x + tail)));
  }
}

template <int MAX>
__global__ void __launch_bounds__(kClipThreads) clip_scale_kernel(const __grid_constant__ ClipList<MAX> l, const __grid_constant__ ClipParams p) {
  __shared__ double red[kClipThreads / 32];
  pdl_wait();
  pdl_trigger();
  const double norm = total_norm(p, red);
  if (p.norm && blockIdx.x == 0 && threadIdx.x == 0) put_norm(p.norm, norm);
  // (a norm that is not finite scales nothing)
  const Factor factor(norm > (double)p.max_norm && isfinite(norm) ? (double)p.max_norm / norm : 1.0);
  const int chunks = l.first[l.count];
  const int c0 = (int)((long long)chunks * blockIdx.x / gridDim.x), c1 = (int)((long long)chunks * (blockIdx.x + 1) / gridDim.x);
  if (c0 >= c1) return;
  int i = find_tensor(l, c1 - 1);
  for (int c = c1 - 1; c >= c0; --c) {  // what was read last may still be in L2
    while (c < l.first[i]) --i;
    if (factor.one() && l.in[i] == l.out[i]) continue;
    const bool scalar = l.kind[i] & kScalar;
    if (l.kind[i] & kBf16) scale_chunk<bf16_t>(l.in[i], l.out[i], l.n[i], c - l.first[i], scalar, factor);
    else scale_chunk<float>(l.in[i], l.out[i], l.n[i], c - l.first[i], scalar, factor);
  }
}

// the tensors from `at` on that fit one launch; returns the first one that does not
template <int MAX>
int fill_list(ClipList<MAX>& l, const GradClipArgs& a, int at) {
  l.count = 0;
  l.first[0] = 0;
  for (; at < a.n && l.count < MAX; ++at) {
    const int64_t n = a.numels[at];
    if (n == 0) continue;
    const bool bf16 = a.dtypes[at] == ATTNRES_BF16;
    const int es = bf16 ? 2 : 4, E = 16 / es;
    const uintptr_t in = reinterpret_cast<uintptr_t>(a.grads[at]);
    const uintptr_t out = reinterpret_cast<uintptr_t>(a.outs ? a.outs[at] : a.grads[at]);
    const bool scalar = ((in ^ out) & 15) != 0;
    const int64_t chunk = (int64_t)kClipChunk * (scalar ? E : 1);
    const int64_t units = scalar ? n : n / E;
    const int64_t chunks = units < chunk ? 1 : (units + chunk - 1) / chunk;
    if (l.count > 0 && l.first[l.count] + chunks > (1 << 30)) break;
    l.in[l.count] = a.grads[at];
    l.out[l.count] = reinterpret_cast<void*>(out);
    l.n[l.count] = n;
    l.kind[l.count] = (bf16 ? kBf16 : 0) | (scalar ? kScalar : 0);
    l.first[l.count + 1] = l.first[l.count] + (int)chunks;
    ++l.count;
  }
  return at;
}

template <int MAX>
cudaError_t launch_lists(const GradClipArgs& a, int cap) {
  ClipList<MAX> l;
  int at = fill_list(l, a, 0);
  const bool one = at >= a.n;
  auto grid = [&] { return l.first[l.count] < 1 ? 1 : l.first[l.count] < cap ? l.first[l.count] : cap; };
  // (every launch of the sums fills the same ones)
  ClipParams p{a.workspace, one ? grid() : cap, 0, a.max_norm, a.norm};
  for (;;) {
    const cudaError_t e = launch_kernel(clip_norm_kernel<MAX>, dim3(p.blocks), dim3(kClipThreads), 0, a.stream, l, p);
    if (e != cudaSuccess) return e;
    p.add = 1;
    if (at >= a.n) break;
    at = fill_list(l, a, at);
  }
  if (!a.outs) return launch_kernel(clip_total_kernel, dim3(1), dim3(kClipThreads), 0, a.stream, p);
  at = one ? at : fill_list(l, a, 0);
  for (;;) {
    const cudaError_t e = launch_kernel(clip_scale_kernel<MAX>, dim3(grid()), dim3(kClipThreads), 0, a.stream, l, p);
    if (e != cudaSuccess) return e;
    p.norm = nullptr;  // (written by the first)
    if (at >= a.n) return cudaSuccess;
    at = fill_list(l, a, at);
  }
}

}  // namespace

int64_t grad_clip_workspace_bytes() {
  DeviceInfo di;
  if (device_info(&di) != cudaSuccess) return -1;
  return (int64_t)di.sm_count * kClipBlocksPerSm * sizeof(double);
}

cudaError_t launch_grad_clip(const GradClipArgs& a) {
  DeviceInfo di;
  const cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  const int cap = di.sm_count * kClipBlocksPerSm;
  return a.n <= kClipFew    ? launch_lists<kClipFew>(a, cap)
         : a.n <= kClipSome ? launch_lists<kClipSome>(a, cap)
                            : launch_lists<kClipMany>(a, cap);
}

}  // namespace attnres
